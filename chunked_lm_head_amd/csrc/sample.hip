// sample.hip — one token per row from a row of logits and one uniform number:
// temperature, top-k, top-p, min-p, then the inverse of the cumulated kept
// weight in index order (include/lmhead_decode.h states the rule).
//
// Exactness. Which token a row gets is decided by comparisons of sums of
// weights w = exp((x - max) / tau), so the weights are made once, in 64 bits
// (2^d by a degree-10 polynomial on |r| <= 1/2, relative error 6e-16), and
// rounded to integers of 2^-shift (shift = 44 up to 262,144 tokens). Their sums
// are exact in 64-bit integers whatever the order, so histograms may be
// filled with integer atomics and the result still repeats bit for bit.
#include "decode_kernels.h"
#include "host_util.h"

#include <limits.h>

namespace lmhead {

namespace {

constexpr int kRowThreads = 1024;
constexpr int kRowWaves = kRowThreads / 64;
constexpr int kBins = 2048;
constexpr int kSegs = 2048;
constexpr uint32_t kMaskedKey = 0x007fffffu;   // key of -infinity

// Order-preserving map of floats to integers; -0 and +0 share a key.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// 2^(d + shift), d <= 0: 2^n (1 + r q(r)), r = d - n, |r| <= 1/2. q
// interpolates (2^r - 1) / r at the ten Chebyshev nodes of the interval.
__device__ __forceinline__ double exp2_scaled(double d, int shift) {
    const double n = __builtin_rint(d);
    const double r = d - n;
    double q = 0x1.e5e9f548e5725p-28;
    q = __builtin_fma(q, r, 0x1.b6571de2f2351p-24);
    q = __builtin_fma(q, r, 0x1.62bfe46117445p-20);
    q = __builtin_fma(q, r, 0x1.ffcb76789860fp-17);
    q = __builtin_fma(q, r, 0x1.4309130378460p-13);
    q = __builtin_fma(q, r, 0x1.5d87fe908f88ap-10);
    q = __builtin_fma(q, r, 0x1.3b2ab6fba385fp-7);
    q = __builtin_fma(q, r, 0x1.c6b08d7044119p-5);
    q = __builtin_fma(q, r, 0x1.ebfbdff82c590p-3);
    q = __builtin_fma(q, r, 0x1.62e42fefa39f7p-1);
    q = __builtin_fma(q, r, 1.0);
    return __builtin_amdgcn_ldexp(q, (int)n + shift);
}

// The row's weights: scaled(x) = 2^shift exp((x - top) / tau), and its integer.
struct Weights {
    double top, scale;   // scale = log2(e) / tau
    int shift;
    __device__ __forceinline__ double scaled(float x) const {
        const double d = ((double)x - top) * scale;
        return d > -64.0 ? exp2_scaled(d, shift) : 0.0;   // -infinity included
    }
    // nearest integer of a value below 2^51: the low bits of 2^52 + it
    static __device__ __forceinline__ uint64_t whole(double s) {
        return __builtin_bit_cast(uint64_t, s + 0x1.0p52) & 0xfffffffffffffull;
    }
};

// A row of logits as 16-byte vectors: the first and last may reach past it
// (rows start at any element); positions outside read as -infinity.
template <bool F32>
struct Row {
    static constexpr int kPer = F32 ? 4 : 8;
    const char* base;    // 16-byte aligned, at or before the row
    int64_t off, end;    // the row is positions off .. end - 1
    __device__ __forceinline__ Row(const void* logits, int64_t row, int64_t ld, int64_t vocab) {
        const char* p = reinterpret_cast<const char*>(logits) + row * ld * (F32 ? 4 : 2);
        const uintptr_t a = reinterpret_cast<uintptr_t>(p);
        base = p - (a & 15);
        off = (int64_t)(a & 15) / (F32 ? 4 : 2);
        end = off + vocab;
    }
    __device__ __forceinline__ int64_t vectors() const { return (end + kPer - 1) / kPer; }
    __device__ __forceinline__ float at(int64_t pos) const {
        if (F32) return reinterpret_cast<const float*>(base)[pos];
        return __builtin_bit_cast(float, (uint32_t) reinterpret_cast<const uint16_t*>(base)[pos] << 16);
    }
    __device__ __forceinline__ void load(int64_t k, float (&x)[kPer]) const {
        const int64_t p0 = k * kPer;
        if (p0 >= off && p0 + kPer <= end) {
            const uint4 v = *reinterpret_cast<const uint4*>(base + k * 16);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (F32) {
                    x[i] = __builtin_bit_cast(float, w[i]);
                } else {
                    x[2 * i] = __builtin_bit_cast(float, w[i] << 16);
                    x[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                x[i] = p0 + i >= off && p0 + i < end ? at(p0 + i) : -__builtin_huge_valf();
        }
    }
};

__device__ __forceinline__ uint64_t wave_scan(uint64_t v, int lane) {   // inclusive
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint64_t o = __shfl_up(v, m);
        if (lane >= m) v += o;
    }
    return v;
}
__device__ __forceinline__ uint64_t wave_total(uint64_t v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

struct Shared {
    uint64_t hist[kBins];
    uint32_t ties[kSegs];
    uint64_t part[kRowWaves + 1];
    uint64_t found_above;
    uint32_t found_bin, flags;
    uint32_t top;
};

// Exclusive prefix of v over the workgroup's threads; total to all.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, Shared& S, uint64_t& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t inc = wave_scan(v, lane);
    __syncthreads();
    if (lane == 63) S.part[wave] = inc;
    __syncthreads();
    uint64_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kRowWaves; ++i) {
        const uint64_t p = S.part[i];
        before += i < wave ? p : 0;
        all += p;
    }
    total = all;
    return before + inc - v;
}

// From the highest bin down: the bin in which the running sum, started at
// `above`, reaches `target` (it is reached); its running sum before it.
__device__ __forceinline__ void find_bin(Shared& S, uint64_t above, uint64_t target, uint32_t& bin,
                                         uint64_t& before) {
    const int b1 = kBins - 1 - 2 * (int)threadIdx.x, b0 = b1 - 1;
    const uint64_t h1 = S.hist[b1], h0 = S.hist[b0];
    uint64_t total;
    const uint64_t ex = above + block_scan(h1 + h0, S, total);
    if (ex < target && ex + h1 + h0 >= target) {
        const bool first = ex + h1 >= target;
        S.found_bin = first ? b1 : b0;
        S.found_above = first ? ex : ex + h1;
    }
    __syncthreads();
    bin = S.found_bin;
    before = S.found_above;
    __syncthreads();
}

// What is kept: keys above `key`, and the first `ties` (by index) equal to it.
struct Threshold {
    uint32_t key;
    uint64_t ties;
};

// The threshold at which the descending running sum of counts (WEIGHTED
// false) or weights reaches `target`, among the members of `in`. Three
// histograms of 11, 11 and 10 key bits.
template <bool F32, bool WEIGHTED>
__device__ Threshold descend(const Row<F32>& row, const Weights& W, Shared& S, uint64_t target,
                             const Threshold& in) {
    constexpr int kPer = Row<F32>::kPer;
    const int64_t nvec = row.vectors();
    uint32_t prefix = 0, mask = 0;
    uint64_t above = 0;
    const uint64_t w_in = WEIGHTED ? Weights::whole(W.scaled(value_of(in.key))) : 0;
    for (int level = 0; level < 3; ++level) {
        const int sh = level == 0 ? 21 : level == 1 ? 10 : 0;
        const uint32_t field = level == 2 ? 1023u : 2047u;
        for (int i = threadIdx.x; i < kBins; i += kRowThreads) S.hist[i] = 0;
        __syncthreads();
        for (int64_t k = threadIdx.x; k < nvec; k += kRowThreads) {
            float x[kPer];
            row.load(k, x);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const uint32_t key = key_of(x[i]);
                if (key > in.key && (key & mask) == prefix)
                    atomicAdd((unsigned long long*)&S.hist[(key >> sh) & field],
                              (unsigned long long)(WEIGHTED ? Weights::whole(W.scaled(x[i])) : 1));
            }
        }
        __syncthreads();
        if (threadIdx.x == 0 && in.ties > 0 && (in.key & mask) == prefix)
            S.hist[(in.key >> sh) & field] += WEIGHTED ? in.ties * w_in : in.ties;
        __syncthreads();
        uint32_t bin;
        find_bin(S, above, target, bin, above);
        prefix |= bin << sh;
        mask |= field << sh;
    }
    const uint64_t w = WEIGHTED ? Weights::whole(W.scaled(value_of(prefix))) : 1;
    return {prefix, (target - above + w - 1) / w};
}

template <bool F32>
__global__ __launch_bounds__(kRowThreads) void sample_rows_kernel(SampleArgs a) {
    constexpr int kPer = Row<F32>::kPer;
    __shared__ Shared S;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
        const Row<F32> row(a.logits, r, a.ld, a.vocab);
        const int64_t nvec = row.vectors();
        const float tau = row_tau(a.T, r);
        const float u = a.u[r];
        const float top_p = a.row_top_p != nullptr ? a.row_top_p[r] : (a.top_p == 0.0f ? 1.0f : a.top_p);
        const float min_p = a.row_min_p != nullptr ? a.row_min_p[r] : a.min_p;
        const int64_t top_k = a.row_top_k != nullptr ? a.row_top_k[r] : a.top_k;
        // largest logit, unmasked tokens, bad logits
        __syncthreads();
        if (tid == 0) S.flags = S.top = 0;
        __syncthreads();
        uint32_t top = 0, bad = 0;
        uint64_t valid = 0;
        for (int64_t k = tid; k < nvec; k += kRowThreads) {
            float x[kPer];
            row.load(k, x);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                bad |= !(x[i] < __builtin_huge_valf());   // NaN, +infinity
                const uint32_t key = key_of(x[i]);
                top = key > top ? key : top;
                valid += key > kMaskedKey;
            }
        }
        atomicMax(&S.top, top);
        if (bad) atomicOr(&S.flags, 1u);
        uint64_t n_valid;
        block_scan(valid, S, n_valid);
        const int code = (S.flags ? kDevErrLogit : 0) | (tau_ok(tau) ? 0 : kDevErrTemperature) |
                         (u >= 0.0f && u < 1.0f && top_p > 0.0f && top_p <= 1.0f && min_p >= 0.0f && min_p <= 1.0f
                              ? 0 : kDevErrSampling);
        if (code != 0 || n_valid == 0) {
            if (tid == 0) {
                a.token[r] = -1;
                if (a.logprob != nullptr) a.logprob[r] = code != 0 ? __builtin_nanf("") : 0.0f;
                if (code != 0) {
                    atomicOr(a.hdr + kHdrErrCode, code);
                    atomicMin(a.hdr + kHdrErrRow, (int32_t)r);
                }
            }
            continue;
        }
        Weights W;
        W.top = (double)value_of(S.top);
        W.scale = 1.4426950408889634 / (double)tau;
        W.shift = a.shift;
        // filters: the threshold of top-k, then that of top-p within it
        Threshold T{kMaskedKey, 0};
        if (top_k > 0 && (uint64_t)top_k < n_valid) T = descend<F32, false>(row, W, S, (uint64_t)top_k, T);
        // the weight of everything (for the log-probability) and of what top-k kept
        uint64_t all, kept;
        {
            uint64_t s_all = 0, s_kept = 0;
            for (int64_t k = tid; k < nvec; k += kRowThreads) {
                float x[kPer];
                row.load(k, x);
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const uint64_t w = Weights::whole(W.scaled(x[i]));
                    s_all += w;
                    s_kept += key_of(x[i]) > T.key ? w : 0;
                }
            }
            block_scan(s_all, S, all);
            block_scan(s_kept, S, kept);
            kept += T.ties * Weights::whole(W.scaled(value_of(T.key)));
        }
        if (top_p < 1.0f) {
            uint64_t target = (uint64_t)__builtin_ceil((double)top_p * (double)kept);
            target = target < 1 ? 1 : (target > kept ? kept : target);
            T = descend<F32, true>(row, W, S, target, T);
        }
        const double floor_p = (double)min_p * __builtin_amdgcn_ldexp(1.0, a.shift);
        const double edge = W.scaled(value_of(T.key));
        const uint64_t w_tie = T.ties > 0 && edge >= floor_p ? Weights::whole(edge) : 0;
        // kept weight and ties per segment of 64 m vectors, a wave each
        const int64_t m = (nvec + 64 * kSegs - 1) / (64 * kSegs);
        const int nseg = (int)((nvec + 64 * m - 1) / (64 * m));
        __syncthreads();
        for (int sg = tid; sg < kSegs; sg += kRowThreads) S.hist[sg] = 0, S.ties[sg] = 0;
        __syncthreads();
        for (int sg = wave; sg < nseg; sg += kRowWaves) {
            uint64_t w = 0, t = 0;
            for (int64_t j = 0; j < m; ++j) {
                const int64_t k = ((int64_t)sg * m + j) * 64 + lane;
                if (k >= nvec) break;
                float x[kPer];
                row.load(k, x);
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const uint32_t key = key_of(x[i]);
                    const double s = W.scaled(x[i]);
                    w += key > T.key && s >= floor_p ? Weights::whole(s) : 0;
                    t += key == T.key;
                }
            }
            w = wave_total(w);
            t = wave_total(t);
            if (lane == 0) S.hist[sg] = w, S.ties[sg] = (uint32_t)t;
        }
        __syncthreads();
        // prefix over the segments (two per thread): ties first, then weight
        const uint64_t t0 = S.ties[2 * tid], t1 = S.ties[2 * tid + 1];
        uint64_t n_ties, total;
        const uint64_t tb = block_scan(t0 + t1, S, n_ties);
        auto kept_ties = [&](uint64_t before, uint64_t here) {
            const uint64_t left = before < T.ties ? T.ties - before : 0;
            return left < here ? left : here;
        };
        const uint64_t w0 = S.hist[2 * tid] + kept_ties(tb, t0) * w_tie;
        const uint64_t w1 = S.hist[2 * tid + 1] + kept_ties(tb + t0, t1) * w_tie;
        const uint64_t wb = block_scan(w0 + w1, S, total);
        uint64_t goal = (uint64_t)((double)u * (double)total);
        goal = goal < total ? goal : total - 1;
        // the segment where the running weight passes the goal: its index, the
        // weight and the ties before it
        __syncthreads();
        if (wb <= goal && wb + w0 + w1 > goal) {
            const bool first = wb + w0 > goal;
            S.found_bin = 2 * tid + (first ? 0 : 1);
            S.found_above = first ? wb : wb + w0;
            S.part[kRowWaves] = first ? tb : tb + t0;
        }
        __syncthreads();
        if (wave == 0) {
            uint64_t run = S.found_above, ties = S.part[kRowWaves];
            const int64_t sg = S.found_bin;
            bool done = false;
            for (int64_t j = 0; j < m && !done; ++j) {
                const int64_t k = (sg * m + j) * 64 + lane;
                float x[kPer];
                uint64_t w[kPer], lane_w = 0, lane_t = 0;
                if (k < nvec) {
                    row.load(k, x);
                } else {
#pragma unroll
                    for (int i = 0; i < kPer; ++i) x[i] = -__builtin_huge_valf();
                }
#pragma unroll
                for (int i = 0; i < kPer; ++i) lane_t += key_of(x[i]) == T.key;
                const uint64_t t_inc = wave_scan(lane_t, lane);
                uint64_t rank = ties + t_inc - lane_t;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const uint32_t key = key_of(x[i]);
                    const double s = W.scaled(x[i]);
                    const bool tie = key == T.key;
                    w[i] = tie ? (rank < T.ties ? w_tie : 0) : (key > T.key && s >= floor_p ? Weights::whole(s) : 0);
                    rank += tie;
                    lane_w += w[i];
                }
                const uint64_t w_inc = wave_scan(lane_w, lane);
                const uint64_t before = run + w_inc - lane_w;
                const bool mine = before <= goal && before + lane_w > goal;
                if (mine) {
                    uint64_t c = before;
                    int pick = 0;
                    bool got = false;
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        c += w[i];
                        if (!got && c > goal) pick = i, got = true;
                    }
                    const int64_t pos = k * kPer + pick;
                    a.token[r] = (int32_t)(pos - row.off);
                    if (a.logprob != nullptr)
                        a.logprob[r] = (float)(((double)row.at(pos) - W.top) / (double)tau -
                                               log((double)all * __builtin_amdgcn_ldexp(1.0, -a.shift)));
                }
                done = __any(mine);
                run += __shfl(w_inc, 63);
                ties += __shfl(t_inc, 63);
            }
        }
    }
}

}  // namespace

void launch_sample(const SampleArgs& a, hipStream_t s) {
    const int grid = grid_1d(a.n, 1, 1 << 20);
    if (a.logits_f32)
        sample_rows_kernel<true><<<grid, kRowThreads, 0, s>>>(a);
    else
        sample_rows_kernel<false><<<grid, kRowThreads, 0, s>>>(a);
}

}  // namespace lmhead
