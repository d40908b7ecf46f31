// embedding.hip — rows of the vocabulary matrix by token, and their gradient.
//
// Mathematics. out[i] = scale W[id_i]. dW[v] (+)= scale sum_{i: id_i = v}
// dout[i]: a sum over the tokens of each id, in fp32, in the order of their places,
// by pieces whose length depends on n alone.
//
// Both are bound by memory. The gradient runs in three launches:
//   1. group: tokens in the order (bucket, id, place). A workgroup owns the ids
//      of one bucket (id mod B, so that common ids spread over the buckets) and
//      reads all n ids, twice: once to count, once to place. It needs nothing
//      from the others: its first place is the number of ids of lower buckets,
//      which it counts along. Where the whole gradient is written, further
//      workgroups of this launch write its zeros meanwhile, 8 KB each.
//   2. sum: a run of tokens of one id is cut into pieces of R (16, or 64 above
//      8192 tokens); 16 .. 64 lanes add a piece over up to 1024 columns. A run
//      of one piece is finished there, longer ones leave fp32 partial sums.
//   3. join: the pieces of the longer runs, in order.
// 16,384 tokens of Zipf ids, 152 k x 4096 bf16 written whole: 190 us (1.25 GB, 6.5
// TB/s), 68 (while the zeros drain to memory) and 6.5. 4096 tokens added to fp32: 9.5,
// 16 (78 MB, 4.8 TB/s) and 6.5; to bf16 9.4, 13 and 6.5. 64 tokens: written whole 190,
// 8 and 4.5, added 6.6, 7 and 4.4 (latency; 16 in a graph).
#include "host_util.h"
#include "train_kernels.h"
#include "vec8.h"

namespace lmhead {

namespace {

// ------------------------------------------------------------------ forward

// A row is taken by 8 .. 64 lanes of a wave (all that its vectors of 8 can
// use), four vectors per lane in flight; wider rows in segments (grid y). 16,384
// rows of 4096 bf16, through the caches: 37.7 us, eight vectors 41.5, two 45.2.
// STREAM: the output past the caches, from twice the eight L2s' 32 MB on. Rows of
// 4096 and 2048 bf16, common and uniform ids, with the norm behind them, through the
// caches / past them: 32 MB of output 25.1 / 26.6 and 26.3 / 28.1 us, 64 MB 42.0 /
// 42.5, 50.3 / 49.1, 40.2 / 41.5 and 49.1 / 47.4, 128 MB 86 / 89, 105 / 104, 86 / 91 and
// 105 / 99, 192 MB 131 / 130, 153 / 148, 140 / 137 and 149 / 147, 512 MB 353 / 340 and 383 / 375.
// The lookup alone gains at every size: 64 MB 18.5 / 15.8, 128 MB 35.3 / 30.7, 512 MB
// 168 / 107.
constexpr int kVectors = 4;
constexpr int64_t kStreamBytes = int64_t(64) << 20;

template <int TYPE, bool OUT32, bool STREAM>
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
        V8 f[kVectors];
#pragma unroll
        for (int k = 0; k < kVectors; ++k) {
            const int v = sub + (((int)blockIdx.y * kVectors + k) << log_lanes);
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
        for (int k = 0; k < kVectors; ++k) {
            const int v = sub + (((int)blockIdx.y * kVectors + k) << log_lanes);
            if (v >= nv) continue;
            if (live)
#pragma unroll
                for (int c = 0; c < 8; ++c) f[k].v[c] *= a.scale;
            store8<OUT32, STREAM>(a.out, to + v, f[k]);
        }
    }
}

// ----------------------------------------------------------------- backward

constexpr int kLocals = 512;       // ids of one bucket
// Tokens of a piece: short ones spread few tokens over the chip, long ones leave
// fewer partial sums. Zipf ids, 100 k x 4096, added to fp32, pieces of 16 and 64:
// 1024 tokens 18.4 and 26.3 us, 4096 28.9 and 37.0, 16,384 91.9 and 89.1, 65,536
// 295 and 266.
constexpr int kLogPiece = 4, kLogPieceMany = 6;
constexpr int64_t kManyTokens = 8192;
constexpr int64_t kMaxFill = int64_t(1) << 21;   // workgroups that write zeros
// 4096 tokens, 90 % of them one id: 30.5 us for the whole gradient, with 4 waves
// 38.4, with one 60; Zipf ids 31.1 and 30.5 us
constexpr int kJoinWaves = 8;
constexpr int kJoinCols = 256;

// An item is a piece's first token in the order: .x its length and flags, .y the
// whole run's length. Other tokens have .x 0.
constexpr int kItemLength = 0xff, kItemFirst = 0x100, kItemLong = 0x200;

int buckets_log(int64_t vocab) {
    int b = 8;
    while ((int64_t(kLocals) << b) < vocab) ++b;
    return b;
}

struct GroupArgs {
    const int32_t* ids;
    int64_t n, vocab;
    int log_buckets;
    int log_piece;
    int32_t *hdr, *order, *keys;
    int2* items;
    uint4* zeros;     // dweight where all of it is written, else null
    int64_t vectors;  // 16-byte vectors of it
};

// 16 waves with 8 ids per lane in registers; 8 waves with 16 where zeros are
// written too, whose workgroups do best at 512 threads (16,384 tokens, 152 k x 4096
// bf16: 258 us for all three launches, with 1024 threads 270; added to fp32
// instead 101 and 94).
template <int kWaves, int kHeld>
__global__ __launch_bounds__(64 * kWaves, kWaves / 2) void group_tokens_kernel(GroupArgs a) {
    constexpr int kGroupThreads = 64 * kWaves;
    // places of (id, wave): an id's tokens stand in the order of the waves' segments
    __shared__ int place[kLocals * kWaves];
    __shared__ int total[kLocals], start[kLocals];
    __shared__ int wave_sum[kWaves], wave_low[kWaves], wave_bad[kWaves];
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
    if ((int)blockIdx.x >> a.log_buckets != 0) {
        const unsigned first = 1u << a.log_buckets;
        for (int64_t v = (int64_t)(blockIdx.x - first) * kGroupThreads + t; v < a.vectors;
             v += (int64_t)(gridDim.x - first) * kGroupThreads)
            a.zeros[v] = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const int bucket = blockIdx.x, mask = (1 << a.log_buckets) - 1;
    for (int i = t; i < kLocals * kWaves; i += kGroupThreads) place[i] = 0;
    __syncthreads();
    const int64_t segment = (a.n + kWaves * 64 - 1) / (kWaves * 64) * 64;
    const int64_t from = wave * segment, to = from + segment < a.n ? from + segment : a.n;
    volatile int* at = place + wave;   // this wave's column
    int low = 0, bad = 0x7fffffff;
    int ids[kHeld];
    const auto fetch = [&](int64_t i0) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const int64_t i = i0 + k * 64 + lane;
            ids[k] = i < to ? a.ids[i] : -1;
        }
    };
    for (int64_t i0 = from; i0 < to; i0 += 64 * kHeld) {
        fetch(i0);
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const int id = ids[k], i = (int)(i0 + k * 64 + lane);
            const bool valid = id >= 0 && id < a.vocab;
            if (id >= a.vocab) bad = bad < i ? bad : i;
            low += valid && (id & mask) < bucket;
            const bool mine = valid && (id & mask) == bucket;
            unsigned long long left = __ballot(mine);
            while (left != 0) {   // as below: atomics of 64 lanes on one common id would wait for one another
                const int lead = __ffsll((long long)left) - 1;
                const int one = __shfl(id, lead);
                const unsigned long long same = __ballot(mine && id == one);
                if (lane == lead) at[(one >> a.log_buckets) * kWaves] += __popcll(same);
                left &= ~same;
            }
        }
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
    // exclusive sums over (id, wave): eight entries per thread, kWaves / 8 threads per id
    int own[8], sum = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        own[k] = place[t * 8 + k];
        sum += own[k];
    }
    const int whole = kWaves == 16 ? sum + __shfl_xor(sum, 1) : sum;
    const bool leads = kWaves == 8 || (t & 1) == 0;
    const int local = kWaves == 16 ? t >> 1 : t;
    if (leads) total[local] = whole;
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
    if (leads) start[local] = run;
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
        for (int64_t i0 = from; i0 < to; i0 += 64 * kHeld) {
            if (to - from > 64 * kHeld) fetch(i0);   // else they are still held
#pragma unroll
            for (int k = 0; k < kHeld; ++k) {
                const int id = ids[k];
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
                        const int l = one >> a.log_buckets, q = p - start[l], c = total[l], piece = 1 << a.log_piece;
                        int2 item = make_int2(0, c);
                        if ((q & (piece - 1)) == 0)
                            item.x = (c - q < piece ? c - q : piece) | (q == 0 ? kItemFirst : 0) |
                                     (c > piece ? kItemLong : 0);
                        a.order[p] = (int)(i0 + k * 64 + lane);
                        a.keys[p] = id;
                        a.items[p] = item;
                    }
                    if (lane == lead) at[slot] = first + __popcll(same);
                    left &= ~same;
                }
            }
        }
    }
}

struct SumArgs {
    EmbedBwdArgs e;
    const int32_t *hdr, *order, *keys;
    const int2* items;
    float* partial;    // [2 windows][hidden], see partial_row
    int log_piece, log_lanes;
    unsigned parts;
};

// A window is as many places of the order as a piece is long. A run's pieces
// begin a window apart, so a window holds at most one later piece of a long run
// and, behind it, at most one first piece of another.
__device__ __forceinline__ int64_t partial_row(int64_t place, int log_piece, bool first) {
    return 2 * (place >> log_piece) + (first ? 1 : 0);
}

// A workgroup takes the items among 16 places of the order, over 64 VPL vectors of
// 8 columns (a part of the row). All that says where its operands stand is
// loaded at once; then 16 .. 64 lanes each take every 4th .. 16th item.
template <bool D32, bool W32, int VPL>
__global__ __launch_bounds__(256) void embedding_sum_kernel(SumArgs a) {
    const int lanes = 1 << a.log_lanes, sub = threadIdx.x & (lanes - 1), near = threadIdx.x & 15;
    const unsigned group = blockIdx.x / a.parts, part = blockIdx.x - group * a.parts;
    const int64_t place0 = (int64_t)group * 16, place = place0 + near, end = a.e.n - 1;
    const int64_t at = place < end ? place : end, at16 = place + 16 < end ? place + 16 : end;
    int2 item = a.items[at];
    const int key = a.keys[at], token_lo = a.order[at], token_hi = a.order[at16];
    if (place >= a.hdr[kHdrCount]) item.x = 0;
    // of these 16 lanes (every 16 of the wave hold the same)
    unsigned live = (unsigned)(__ballot(item.x != 0) >> (threadIdx.x & 48)) & 0xffffu;
    for (int skip = threadIdx.x >> a.log_lanes; skip > 0 && live != 0; --skip) live &= live - 1;
    const int nv = a.e.hidden >> 3, v0 = (int)part * 64 * VPL + sub;
    while (live != 0) {
        const int o = __ffs((int)live) - 1;
        const int flags = __shfl(item.x, o, 16), length = flags & kItemLength;
        const bool whole = (flags & kItemLong) == 0, add = whole && a.e.accumulate;
        const int64_t row = (int64_t)__shfl(key, o, 16) * nv;
        V8 sum[VPL];
        Raw8<W32> old[VPL];
        if (add)   // under way while the tokens are summed
#pragma unroll
            for (int k = 0; k < VPL; ++k)
                if (v0 + k * lanes < nv) old[k] = load_raw8<W32>(a.e.dweight, row + v0 + k * lanes);
#pragma unroll
        for (int k = 0; k < VPL; ++k) sum[k] = zeros8();
        constexpr int U = 4;   // tokens in flight
        for (int j0 = 0; j0 < length; j0 += 16) {
            const int stop = length - j0 < 16 ? length - j0 : 16;
            const int later = j0 > 0 && near < stop ? a.order[place0 + o + j0 + near] : 0;
            for (int j = 0; j < stop; j += U) {
                Raw8<D32> f[U][VPL];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = o + j + u;
                    const int lo = __shfl(token_lo, i, 16), hi = __shfl(token_hi, i, 16), on = __shfl(later, j + u, 16);
                    const int64_t from = (int64_t)(j0 > 0 ? on : i < 16 ? lo : hi) * nv;
                    if (j + u < stop)
#pragma unroll
                        for (int k = 0; k < VPL; ++k)
                            if (v0 + k * lanes < nv) f[u][k] = load_raw8<D32>(a.e.dout, from + v0 + k * lanes);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (j + u < stop)
#pragma unroll
                        for (int k = 0; k < VPL; ++k) {
                            const V8 x = to8<D32>(f[u][k]);
#pragma unroll
                            for (int c = 0; c < 8; ++c) sum[k].v[c] += x.v[c];
                        }
            }
        }
        float* out = a.partial + partial_row(place0 + o, a.log_piece, (flags & kItemFirst) != 0) * a.e.hidden;
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
            const int v = v0 + k * lanes;
            if (v >= nv) continue;
            if (!whole) {
                store8<true>(out, v, sum[k]);
                continue;
            }
            const V8 before = add ? to8<W32>(old[k]) : zeros8();
#pragma unroll
            for (int c = 0; c < 8; ++c) sum[k].v[c] = sum[k].v[c] * a.e.scale + before.v[c];
            store8<W32>(a.e.dweight, row + v, sum[k]);
        }
        for (int skip = 256 >> a.log_lanes; skip > 0 && live != 0; --skip) live &= live - 1;
    }
}

// The long run whose first piece lies in this workgroup's window, if there is
// one. Four columns per lane; each wave takes every eighth piece, then their
// sums are added in order.
template <bool W32>
__global__ __launch_bounds__(64 * kJoinWaves) void embedding_join_kernel(SumArgs a) {
    __shared__ float4 part_sum[kJoinWaves][64];
    const int64_t count = a.hdr[kHdrCount], window = blockIdx.x, from = window << a.log_piece;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t place = from + lane;
    const bool in = lane < 1 << a.log_piece && place < count;
    const int2 item = in ? a.items[place] : make_int2(0, 0);
    const unsigned long long heads = __ballot((item.x & kItemFirst) != 0 && (item.x & kItemLong) != 0);
    if (heads == 0) return;
    const int lead = __ffsll((long long)heads) - 1;
    const int length = __shfl(item.y, lead);
    const int64_t pieces = ((int64_t)length + (1 << a.log_piece) - 1) >> a.log_piece;
    const int64_t id = a.keys[from + lead];
    const int col = (int)blockIdx.y * kJoinCols + lane * 4;
    const bool live = col < a.e.hidden;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (live) {
#pragma unroll 8
        for (int64_t j = wave; j < pieces; j += kJoinWaves) {
            const float4 v = *reinterpret_cast<const float4*>(a.partial + (2 * (window + j) + (j == 0)) * a.e.hidden + col);
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
    }
    part_sum[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || !live) return;
#pragma unroll
    for (int w = 1; w < kJoinWaves; ++w) {
        const float4 v = part_sum[w][lane];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    const int64_t at = id * a.e.hidden + col;
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
void sum_and_join(SumArgs a, hipStream_t s) {
    const int nv = a.e.hidden >> 3;
    a.log_lanes = nv <= 16 ? 4 : nv <= 32 ? 5 : 6;
    a.parts = nv <= 64 ? 1u : (unsigned)cdiv(nv, 128);
    const unsigned x = (unsigned)cdiv(a.e.n, 16) * a.parts;
    if (nv <= 64) embedding_sum_kernel<D32, W32, 1><<<x, 256, 0, s>>>(a);
    else embedding_sum_kernel<D32, W32, 2><<<x, 256, 0, s>>>(a);
    if (a.e.n > 1 << a.log_piece)
        embedding_join_kernel<W32><<<dim3((unsigned)cdiv(a.e.n, 1 << a.log_piece), (unsigned)cdiv(a.e.hidden, kJoinCols)),
                                     64 * kJoinWaves, 0, s>>>(a);
}

}  // namespace

namespace {
template <int TYPE, bool OUT32>
void embedding(const EmbedArgs& a, hipStream_t s) {
    const int nv = a.hidden >> 3;
    int log_lanes = 3;
    while (log_lanes < 6 && (1 << log_lanes) < nv) ++log_lanes;
    const dim3 grid((unsigned)grid_1d(a.n, 256 >> log_lanes, 1 << 20), (unsigned)cdiv(nv, kVectors << log_lanes));
    if (a.n * a.hidden * (OUT32 ? 4 : 2) >= kStreamBytes) embedding_kernel<TYPE, OUT32, true><<<grid, 256, 0, s>>>(a, log_lanes);
    else embedding_kernel<TYPE, OUT32, false><<<grid, 256, 0, s>>>(a, log_lanes);
}
}  // namespace

void launch_embedding(const EmbedArgs& a, hipStream_t s) {
    if (a.hdr != nullptr) init_header_kernel<<<1, 64, 0, s>>>(a.hdr);
    if (a.weight_type == kEmbedE4m3) {
        if (a.out_f32) embedding<kEmbedE4m3, true>(a, s);
        else embedding<kEmbedE4m3, false>(a, s);
    } else if (a.weight_type == kEmbedF32) {
        if (a.out_f32) embedding<kEmbedF32, true>(a, s);
        else embedding<kEmbedF32, false>(a, s);
    } else {
        if (a.out_f32) embedding<kEmbedBf16, true>(a, s);
        else embedding<kEmbedBf16, false>(a, s);
    }
}

namespace {
struct EmbedPlan {
    int log_buckets, log_piece;
    int64_t order, keys, items, partial, bytes;
};
EmbedPlan plan_bwd(int64_t n, int64_t vocab, int hidden) {
    EmbedPlan p;
    p.log_buckets = buckets_log(vocab);
    p.log_piece = n > kManyTokens ? kLogPieceMany : kLogPiece;
    p.order = 256;
    p.keys = p.order + round_up(4 * n, 256);
    p.items = p.keys + round_up(4 * n, 256);
    p.partial = p.items + round_up(8 * n, 256);
    const int64_t piece = 1 << p.log_piece;
    p.bytes = p.partial + (n > piece ? round_up(cdiv(n, piece) * 2 * hidden * 4, 256) : 0);
    return p;
}
}  // namespace

size_t embedding_bwd_workspace(int64_t n, int64_t vocab, int hidden) {
    return (size_t)plan_bwd(n, vocab, hidden).bytes;
}

void launch_embedding_bwd(const EmbedBwdArgs& a, void* workspace, hipStream_t s) {
    const EmbedPlan p = plan_bwd(a.n, a.vocab, a.hidden);
    char* w = (char*)workspace;
    GroupArgs g;
    g.ids = a.ids;
    g.n = a.n;
    g.vocab = a.vocab;
    g.log_buckets = p.log_buckets;
    g.log_piece = p.log_piece;
    g.hdr = (int32_t*)w;
    g.order = (int32_t*)(w + p.order);
    g.keys = (int32_t*)(w + p.keys);
    g.items = (int2*)(w + p.items);
    g.zeros = (uint4*)a.dweight;
    g.vectors = a.accumulate ? 0 : a.vocab * (a.hidden * (a.dweight_f32 ? 4 : 2) / 16);
    const unsigned buckets = 1u << g.log_buckets;
    const int64_t fills = cdiv(g.vectors, 512);
    if (a.accumulate) group_tokens_kernel<16, 8><<<buckets, 1024, 0, s>>>(g);
    else group_tokens_kernel<8, 16><<<buckets + (unsigned)(fills < kMaxFill ? fills : kMaxFill), 512, 0, s>>>(g);
    if (a.n == 0) return;
    SumArgs u;
    u.e = a;
    u.hdr = g.hdr;
    u.order = g.order;
    u.keys = g.keys;
    u.items = g.items;
    u.partial = (float*)(w + p.partial);
    u.log_piece = p.log_piece;
    if (a.dout_f32) {
        if (a.dweight_f32) sum_and_join<true, true>(u, s);
        else sum_and_join<true, false>(u, s);
    } else {
        if (a.dweight_f32) sum_and_join<false, true>(u, s);
        else sum_and_join<false, false>(u, s);
    }
}

}  // namespace lmhead
