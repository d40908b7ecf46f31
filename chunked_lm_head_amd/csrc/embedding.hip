// embedding.hip — rows of the vocabulary matrix by token, and their gradient.
//
// Mathematics. out[i] = scale W[id_i]. dW[v] (+)= scale sum_{i: id_i = v}
// dout[i]: a sum over the tokens of each id, in fp32, in an order that depends
// on the ids alone.
//
// Both are bound by memory. The gradient runs in three launches:
//   1. group: tokens in the order (bucket, id, place). A workgroup owns the ids
//      of one bucket (id mod B, so that common ids spread over the buckets) and
//      reads all n ids, twice: once to count, once to place. It needs nothing
//      from the others: its first place is the number of ids of lower buckets,
//      which it counts along. Where the whole gradient is written, the
//      workgroup also writes the zeros of its ids without a token.
//   2. sum: a workgroup adds kSumRows tokens of that order over 2048 columns.
//      A run of one id within them is finished there; a run that passes a
//      border leaves fp32 partial sums.
//   3. join: partial sums of such runs, in order.
#include "host_util.h"
#include "train_kernels.h"
#include "vec8.h"

namespace lmhead {

namespace {

// ------------------------------------------------------------------ forward

// A row is taken by 8 .. 64 lanes of a wave (all that its vectors of 8 can
// use), eight vectors per lane in flight; wider rows in segments (grid y).
template <int TYPE, bool OUT32>
__global__ __launch_bounds__(256) void embedding_kernel(EmbedArgs a, int log_lanes) {
    const int lanes = 1 << log_lanes, lane = threadIdx.x & 63;
    const int sub = lane & (lanes - 1);
    const int per_group = 256 >> log_lanes;   // rows of a workgroup
    const int nv = a.hidden >> 3;
    for (int64_t row0 = (int64_t)blockIdx.x * per_group; row0 < a.n; row0 += (int64_t)gridDim.x * per_group) {
        const int64_t row = row0 + (threadIdx.x >> log_lanes);
        if (row >= a.n) continue;
        const int64_t id = a.ids[row];
        const bool live = id >= 0 && id < a.vocab;
        const float fill = id >= a.vocab ? __builtin_nanf("") : 0.0f;
        if (a.hdr != nullptr && id >= a.vocab && sub == 0 && blockIdx.y == 0) {
            atomicOr(&a.hdr[kHdrErrCode], kDevErrToken);
            atomicMin(&a.hdr[kHdrErrRow], (int)row);
        }
        const int64_t from = (live ? id : 0) * nv, to = row * nv;
        V8 f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int v = sub + (((int)blockIdx.y * 8 + k) << log_lanes);
            f[k] = V8{{fill, fill, fill, fill, fill, fill, fill, fill}};
            if (live && v < nv) {
                if (TYPE == kEmbedE4m3) {
                    f[k] = e4m3_to8(reinterpret_cast<const uint2*>(a.weight)[from + v]);
                    const float s = a.weight_scale[(id >> 7) * (nv >> 4) + (v >> 4)];
#pragma unroll
                    for (int c = 0; c < 8; ++c) f[k].v[c] *= s;
                } else {
                    f[k] = load8<TYPE == kEmbedF32>(a.weight, from + v);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int v = sub + (((int)blockIdx.y * 8 + k) << log_lanes);
            if (v >= nv) continue;
            if (live)
#pragma unroll
                for (int c = 0; c < 8; ++c) f[k].v[c] *= a.scale;
            store8<OUT32>(a.out, to + v, f[k]);
        }
    }
}

// ----------------------------------------------------------------- backward

constexpr int kLocals = 512;   // ids of one bucket
constexpr int kWaves = 16;     // of a grouping workgroup
constexpr int kSumCols = 2048; // columns of a summing workgroup
constexpr int kJoinCols = 256;

int buckets_log(int64_t vocab) {
    int b = 8;
    while ((int64_t(kLocals) << b) < vocab) ++b;
    return b;
}

struct GroupArgs {
    const int32_t* ids;
    int64_t n, vocab;
    int log_buckets;
    int32_t *hdr, *order, *keys;
    uint4* zero_into;     // dweight where untouched rows are written, else null
    int64_t row_vectors;  // 16-byte vectors of its rows
};

__global__ __launch_bounds__(1024) void group_tokens_kernel(GroupArgs a) {
    // places of (id, wave): an id's tokens stand in the order of the waves' segments
    __shared__ int place[kLocals * kWaves];
    __shared__ int total[kLocals];
    __shared__ int wave_sum[kWaves], wave_low[kWaves], wave_bad[kWaves];
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
    const int bucket = blockIdx.x, mask = (1 << a.log_buckets) - 1;
    for (int i = t; i < kLocals * kWaves; i += 1024) place[i] = 0;
    __syncthreads();
    const int64_t segment = (a.n + kWaves * 64 - 1) / (kWaves * 64) * 64;
    const int64_t from = wave * segment, to = from + segment < a.n ? from + segment : a.n;
    int low = 0, bad = 0x7fffffff;
#pragma unroll 8
    for (int64_t i = from + lane; i < to; i += 64) {
        const int id = a.ids[i];
        if (id < 0) continue;
        if (id >= a.vocab) {
            bad = bad < (int)i ? bad : (int)i;
            continue;
        }
        const int b = id & mask;
        low += b < bucket;
        if (b == bucket) atomicAdd(&place[(id >> a.log_buckets) * kWaves + wave], 1);
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        low += __shfl_xor(low, m);
        const int other = __shfl_xor(bad, m);
        bad = bad < other ? bad : other;
    }
    if (lane == 0) {
        wave_low[wave] = low;
        wave_bad[wave] = bad;
    }
    __syncthreads();
    // exclusive sums over (id, wave): eight entries per thread, two threads per id
    int own[8], sum = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        own[k] = place[t * 8 + k];
        sum += own[k];
    }
    const int both = sum + __shfl_xor(sum, 1);
    if ((t & 1) == 0) total[t >> 1] = both;
    int run = sum;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int v = __shfl_up(run, m);
        if (lane >= m) run += v;
    }
    if (lane == 63) wave_sum[wave] = run;
    __syncthreads();
    int base = 0, all = 0;
    for (int w = 0; w < kWaves; ++w) {
        base += wave_low[w];
        if (w < wave) run += wave_sum[w];
        all += wave_sum[w];
    }
    run += base - sum;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        place[t * 8 + k] = run;
        run += own[k];
    }
    if (t == 0) {
        if (bucket == 0) {   // has seen every id
            int row = 0x7fffffff;
            for (int w = 0; w < kWaves; ++w) row = row < wave_bad[w] ? row : wave_bad[w];
            a.hdr[kHdrErrRow] = row;
            a.hdr[kHdrErrCode] = row != 0x7fffffff ? kDevErrToken : 0;
        }
        if (bucket == mask) a.hdr[kHdrCount] = base + all;
    }
    __syncthreads();
    if (all > 0) {
        volatile int* at = place + wave;   // this wave's column
        for (int64_t i0 = from; i0 < to; i0 += 64) {
            const int64_t i = i0 + lane;
            const int id = i < to ? a.ids[i] : -1;
            const bool mine = id >= 0 && id < a.vocab && (id & mask) == bucket;
            unsigned long long left = __ballot(mine);
            while (left != 0) {   // one id a turn, its lanes in order
                const int lead = __ffsll((long long)left) - 1;
                const int one = __shfl(id, lead);
                const unsigned long long same = __ballot(mine && id == one);
                const int slot = (one >> a.log_buckets) * kWaves;
                const int first = at[slot];
                if (mine && id == one) {
                    const int p = first + __popcll(same & ((1ull << lane) - 1));
                    a.order[p] = (int)i;
                    a.keys[p] = id;
                }
                if (lane == lead) at[slot] = first + __popcll(same);
                left &= ~same;
            }
        }
    }
    if (a.zero_into == nullptr) return;
    for (int l = wave; l < kLocals; l += kWaves) {
        const int64_t id = ((int64_t)l << a.log_buckets) + bucket;
        if (id >= a.vocab) break;
        if (total[l] != 0) continue;
        uint4* row = a.zero_into + id * a.row_vectors;
        for (int64_t v = lane; v < a.row_vectors; v += 64) row[v] = make_uint4(0u, 0u, 0u, 0u);
    }
}

struct SumArgs {
    EmbedBwdArgs e;
    const int32_t *hdr, *order, *keys;
    float* partial;   // [blocks][2][hidden]: a block's first run, if it began before; its last, if it goes on
    int slices;
};

// dweight's vector i of a row from the id's finished sum
template <bool W32>
__device__ __forceinline__ void finish(const EmbedBwdArgs& e, int64_t id, int vec, const V8& sum) {
    const int64_t at = id * (e.hidden >> 3) + vec;
    V8 f;
#pragma unroll
    for (int c = 0; c < 8; ++c) f.v[c] = sum.v[c] * e.scale;
    if (e.accumulate) {
        const V8 old = load8<W32>(e.dweight, at);
#pragma unroll
        for (int c = 0; c < 8; ++c) f.v[c] += old.v[c];
    }
    store8<W32>(e.dweight, at, f);
}

template <bool D32, bool W32>
__global__ __launch_bounds__(256) void embedding_sum_kernel(SumArgs a) {
    __shared__ int token[kSumRows], key[kSumRows + 2];
    const int64_t block = blockIdx.x / a.slices;
    const int slice = (int)(blockIdx.x - block * a.slices);
    const int64_t count = a.hdr[kHdrCount], i0 = block * kSumRows;
    if (i0 >= count) return;
    const int rows = (int)(count - i0 < kSumRows ? count - i0 : kSumRows);
    const int t = threadIdx.x;
    if (t < kSumRows + 2) {   // key[1 + j]: row j's; -1 before the first and behind the last row of all
        const int64_t i = i0 + t - 1;
        key[t] = i >= 0 && i < count ? a.keys[i] : -1;
    }
    if (t < rows) token[t] = a.order[i0 + t];
    __syncthreads();
    const int nv = a.e.hidden >> 3, vec = slice * (kSumCols / 8) + t;
    if (vec >= nv) return;
    V8 sum = zeros8();
    bool first = true;
    for (int j0 = 0; j0 < rows; j0 += 8) {
        V8 f[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (j0 + u < rows) f[u] = load8<D32>(a.e.dout, (int64_t)token[j0 + u] * nv + vec);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int j = j0 + u;
            if (j >= rows) break;
#pragma unroll
            for (int c = 0; c < 8; ++c) sum.v[c] += f[u].v[c];
            const int k = key[1 + j];
            const bool last = j == rows - 1;
            if (!last && key[2 + j] == k) continue;
            const bool before = first && key[0] == k, after = last && key[2 + j] == k;
            if (before || after) {
                float* out = a.partial + (block * 2 + (before ? 0 : 1)) * a.e.hidden;
                store8<true>(out, vec, sum);
            } else {
                finish<W32>(a.e, k, vec, sum);
            }
            sum = zeros8();
            first = false;
        }
    }
}

// The runs that begin in a block and pass its end: that block's last partial
// sum and the following blocks' first ones. Sixteen waves take every 16th of
// the latter and are added in order. Four columns per lane.
template <bool W32>
__global__ __launch_bounds__(1024) void embedding_join_kernel(SumArgs a) {
    __shared__ float4 part[16][64];
    const int64_t block = blockIdx.x;
    const int64_t count = a.hdr[kHdrCount], next = (block + 1) * kSumRows;
    if (next >= count) return;
    const int k = a.keys[next - 1];
    if (a.keys[next] != k) return;
    if (block > 0 && a.keys[block * kSumRows] == k && a.keys[block * kSumRows - 1] == k) return;   // began before
    int64_t lo = block + 1, hi = (count - 1) / kSumRows;   // the last block that begins with k
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) / 2;
        if (a.keys[mid * kSumRows] == k) lo = mid;
        else hi = mid - 1;
    }
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int col = (int)blockIdx.y * kJoinCols + lane * 4;
    const bool in = col < a.e.hidden;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (in) {
#pragma unroll 8
        for (int64_t b = block + 1 + wave; b <= lo; b += 16) {
            const float4 v = *reinterpret_cast<const float4*>(a.partial + b * 2 * a.e.hidden + col);
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || !in) return;
    s = *reinterpret_cast<const float4*>(a.partial + (block * 2 + 1) * a.e.hidden + col);
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        const float4 v = part[w][lane];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    const int64_t at = (int64_t)k * a.e.hidden + col;
    float f[4] = {s.x * a.e.scale, s.y * a.e.scale, s.z * a.e.scale, s.w * a.e.scale};
    if (W32) {
        float4* out = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.e.dweight) + at);
        if (a.e.accumulate) {
            const float4 old = *out;
            f[0] += old.x;
            f[1] += old.y;
            f[2] += old.z;
            f[3] += old.w;
        }
        *out = make_float4(f[0], f[1], f[2], f[3]);
    } else {
        uint2* out = reinterpret_cast<uint2*>(reinterpret_cast<bf16_bits*>(a.e.dweight) + at);
        if (a.e.accumulate) {
            const uint2 old = *out;
            f[0] += __builtin_bit_cast(float, old.x << 16);
            f[1] += __builtin_bit_cast(float, old.x & 0xffff0000u);
            f[2] += __builtin_bit_cast(float, old.y << 16);
            f[3] += __builtin_bit_cast(float, old.y & 0xffff0000u);
        }
        *out = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    }
}

template <bool D32, bool W32>
void sum_and_join(const SumArgs& a, hipStream_t s) {
    const int64_t blocks = cdiv(a.e.n, kSumRows);
    embedding_sum_kernel<D32, W32><<<(unsigned)(blocks * a.slices), 256, 0, s>>>(a);
    if (blocks > 1)
        embedding_join_kernel<W32>
            <<<dim3((unsigned)blocks, (unsigned)cdiv(a.e.hidden, kJoinCols)), 1024, 0, s>>>(a);
}

}  // namespace

void launch_embedding(const EmbedArgs& a, hipStream_t s) {
    const int nv = a.hidden >> 3;
    int log_lanes = 3;
    while (log_lanes < 6 && (1 << log_lanes) < nv) ++log_lanes;
    const dim3 grid((unsigned)grid_1d(a.n, 256 >> log_lanes, 1 << 20), (unsigned)cdiv(nv, 8 << log_lanes));
    if (a.hdr != nullptr) init_header_kernel<<<1, 64, 0, s>>>(a.hdr);
    if (a.weight_type == kEmbedE4m3) {
        if (a.out_f32) embedding_kernel<kEmbedE4m3, true><<<grid, 256, 0, s>>>(a, log_lanes);
        else embedding_kernel<kEmbedE4m3, false><<<grid, 256, 0, s>>>(a, log_lanes);
    } else if (a.weight_type == kEmbedF32) {
        if (a.out_f32) embedding_kernel<kEmbedF32, true><<<grid, 256, 0, s>>>(a, log_lanes);
        else embedding_kernel<kEmbedF32, false><<<grid, 256, 0, s>>>(a, log_lanes);
    } else {
        if (a.out_f32) embedding_kernel<kEmbedBf16, true><<<grid, 256, 0, s>>>(a, log_lanes);
        else embedding_kernel<kEmbedBf16, false><<<grid, 256, 0, s>>>(a, log_lanes);
    }
}

namespace {
struct EmbedPlan {
    int64_t order, keys, partial, bytes;
};
EmbedPlan plan_bwd(int64_t n, int hidden) {
    EmbedPlan p;
    p.order = 256;
    p.keys = p.order + round_up(4 * n, 256);
    p.partial = p.keys + round_up(4 * n, 256);
    const int64_t blocks = cdiv(n, kSumRows);
    p.bytes = p.partial + (blocks > 1 ? round_up(blocks * 2 * hidden * 4, 256) : 0);
    return p;
}
}  // namespace

size_t embedding_bwd_workspace(int64_t n, int hidden) { return (size_t)plan_bwd(n, hidden).bytes; }

void launch_embedding_bwd(const EmbedBwdArgs& a, void* workspace, hipStream_t s) {
    const EmbedPlan p = plan_bwd(a.n, a.hidden);
    char* w = (char*)workspace;
    GroupArgs g;
    g.ids = a.ids;
    g.n = a.n;
    g.vocab = a.vocab;
    g.log_buckets = buckets_log(a.vocab);
    g.hdr = (int32_t*)w;
    g.order = (int32_t*)(w + p.order);
    g.keys = (int32_t*)(w + p.keys);
    g.zero_into = a.accumulate ? nullptr : (uint4*)a.dweight;
    g.row_vectors = (int64_t)a.hidden * (a.dweight_f32 ? 4 : 2) / 16;
    group_tokens_kernel<<<1u << g.log_buckets, 1024, 0, s>>>(g);
    if (a.n == 0) return;
    SumArgs u;
    u.e = a;
    u.hdr = g.hdr;
    u.order = g.order;
    u.keys = g.keys;
    u.partial = (float*)(w + p.partial);
    u.slices = (int)cdiv(a.hidden, kSumCols);
    if (a.dout_f32) {
        if (a.dweight_f32) sum_and_join<true, true>(u, s);
        else sum_and_join<true, false>(u, s);
    } else {
        if (a.dweight_f32) sum_and_join<false, true>(u, s);
        else sum_and_join<false, false>(u, s);
    }
}

}  // namespace lmhead
