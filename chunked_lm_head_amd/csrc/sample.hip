// sample.hip — one token per row from a row of logits and one uniform number:
// temperature, top-k, top-p, min-p, then the inverse of the cumulated kept
// weight in index order (include/lmhead_decode.h states the rule).
//
// Exactness. Which token a row gets is decided by comparisons of sums of
// weights w = exp((x - max) / tau), so the weights are made in 64 bits (2^d by
// a degree-9 polynomial on |r| <= 1/2, relative error 4e-14) and rounded to
// integers of 2^-shift (shift = 44 up to 262,144 tokens). Their sums are exact
// in 64-bit integers whatever the order, so histograms may be filled with
// integer atomics and the result still repeats bit for bit. What the rounding
// leaves of each weight is summed beside them where the step is coarser (larger
// vocabularies), in integers of 2^-30 of it, for the log-probability: millions
// of tokens below half a step weigh something together.
//
// Plan. In the order of descending logit (equal logits by index) each filter
// keeps a prefix, so all of them together keep the shortest of the prefixes.
// Rows are cut into slices, a workgroup each, and go through five launches
// (three without filters):
//   scan    largest and smallest logit of the slice, bad values;
//   hist    weight (and count, for top-k) of the slice's tokens in 2048 bins
//           of equal width below the row's largest logit;
//   border  (a workgroup per row) the bins in which the prefixes end;
//   gather  the row's tokens in those bins (some hundred) are listed;
//   pick    the list sorted, the end of the prefix found exactly; the kept
//           weight of each slice from its histogram; the slice in which u
//           falls, and the token in it.
// So each logit is read three times (from memory once, the rest from the
// caches: rows are taken 256 at a time) and its weight is computed once. What
// the list cannot hold (thousands of equal logits at the border) is resolved
// by a radix descent over the row, in the pick kernel.
#include "decode_kernels.h"
#include "host_util.h"

#include <limits.h>

namespace lmhead {

namespace {

constexpr int kRowThreads = 1024;
constexpr int kRowWaves = kRowThreads / 64;
constexpr int kBins = 2048;
constexpr int kSegs = 2048;
constexpr int kList = 4096;        // listed border tokens per row
constexpr int kMaxSlices = 16;
constexpr int kChunkRows = 256;    // rows per set of launches
constexpr uint32_t kMaskedKey = 0x007fffffu;   // key of -infinity

// Order-preserving map of floats to integers; -0 and +0 share a key.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// a * b + c with the constant c in scalar registers. Given as a builtin, the
// compiler copies every constant into vector registers before each use, one
// move per multiply-add.
__device__ __forceinline__ double fma_s(double a, double b, double c) {
    double d;
    asm("v_fma_f64 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "s"(c));
    return d;
}

// The row's weights: scaled(x) = 2^shift exp((x - top) / tau) as a double.
// 2^d = 2^n (1 + r q(r)), r = d - n, |r| <= 1/2; q interpolates (2^r - 1) / r
// at the nine Chebyshev nodes of the interval. The nearest integer n comes from
// adding 1.5 * 2^52, whose low word then holds it; 2^n goes into the exponent
// field. d is kept at -64 or above (-infinity included): a weight of 0.
struct Weights {
    double top, scale;   // scale = log2(e) / tau
    int shift;
    __device__ __forceinline__ double scaled(float x) const {
        const double d = __builtin_fmax(((double)x - top) * scale, -64.0);
        const double t = d + 0x1.8p52;
        const double r = d - (t - 0x1.8p52);
        double q = 0x1.b63880a30e9ffp-24;
        q = fma_s(q, r, 0x1.63d136366db24p-20);
        q = fma_s(q, r, 0x1.ffcb9515a8016p-17);
        q = fma_s(q, r, 0x1.4308ac85aa947p-13);
        q = fma_s(q, r, 0x1.5d87fe86fe88ep-10);
        q = fma_s(q, r, 0x1.3b2ab7181b755p-7);
        q = fma_s(q, r, 0x1.c6b08d7047e52p-5);
        q = fma_s(q, r, 0x1.ebfbdff823cedp-3);
        q = fma_s(q, r, 0x1.62e42fefa39efp-1);
        q = __builtin_fma(q, r, 1.0);
        const int n = (int)(uint32_t)__builtin_bit_cast(uint64_t, t) + shift;
        return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, q) + ((uint64_t)(uint32_t)n << 52));
    }
    // nearest integer of a value below 2^51: the low bits of 2^52 + it
    static __device__ __forceinline__ uint64_t whole(double s) {
        return __builtin_bit_cast(uint64_t, s + 0x1.0p52) & 0xfffffffffffffull;
    }
    __device__ __forceinline__ uint64_t of(float x) const { return whole(scaled(x)); }
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
    // the vectors that lie inside the row: whole_from() .. whole_to() - 1 (none when not below)
    __device__ __forceinline__ int64_t whole_from() const { return off > 0 ? 1 : 0; }
    __device__ __forceinline__ int64_t whole_to() const { return end / kPer; }
    // vectors k, k + 64, k + 128, k + 192; as -infinity those from k1 on and the row's ragged ones
    __device__ __forceinline__ void load4(int64_t k, int64_t k1, float (&x)[4][kPer]) const {
        const int64_t a0 = whole_from(), a1 = whole_to();
        uint4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t kq = k + q * 64;
            v[q] = *reinterpret_cast<const uint4*>(base + (kq < a0 ? a0 : kq < a1 ? kq : a1 - 1) * 16);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t kq = k + q * 64;
            const bool in = kq < k1 && kq >= a0 && kq < a1;
            const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (F32) {
                    x[q][i] = in ? __builtin_bit_cast(float, w[i]) : -__builtin_huge_valf();
                } else {
                    x[q][2 * i] = in ? __builtin_bit_cast(float, w[i] << 16) : -__builtin_huge_valf();
                    x[q][2 * i + 1] = in ? __builtin_bit_cast(float, w[i] & 0xffff0000u) : -__builtin_huge_valf();
                }
            }
        }
    }
    // f(values, first position) for this thread's share of vectors k0 .. k1 - 1 (arrays of kPer values;
    // of one at the row's ragged ends). One vector at a time: the waves of the other workgroups cover its
    // load (256 rows of 151,936, histogram: 45 us; two or four at a time, or the next ones fetched ahead,
    // 56 to 59 us)
    template <class F>
    __device__ __forceinline__ void each(int64_t k0, int64_t k1, F f) const {
        const int64_t a0 = k0 == 0 && off > 0 ? 1 : k0;               // the vectors inside the row
        const int64_t a1 = k1 * kPer > end ? end / kPer : k1;
        for (int64_t k = a0 + threadIdx.x; k < a1; k += kRowThreads) {
            const uint4 v = *reinterpret_cast<const uint4*>(base + k * 16);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            float x[kPer];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (F32) {
                    x[i] = __builtin_bit_cast(float, w[i]);
                } else {
                    x[2 * i] = __builtin_bit_cast(float, w[i] << 16);
                    x[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
                }
            }
            f(x, k * kPer);
        }
        // the row's first and last positions outside whole vectors, one a thread
        const int64_t h1 = end < kPer ? end : kPer;
        if (k0 == 0 && k1 > 0 && off > 0 && threadIdx.x < h1 - off) one(f, off + threadIdx.x);
        const int64_t t0 = end / kPer * kPer;
        if (k1 * kPer > end && (t0 > 0 || off == 0) && threadIdx.x < end - t0) one(f, t0 + threadIdx.x);
    }
    template <class F>
    __device__ __forceinline__ void one(F f, int64_t pos) const {
        const float x[1] = {at(pos)};
        f(x, pos);
    }
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

// v plus the value that the DPP move CTRL brings from another lane (0 where it brings none)
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t add_dpp(uint64_t v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xf, false);
    return v + ((uint64_t)hi << 32 | lo);
}
// Inclusive prefix over the wave: within rows of 16 lanes (row_shr 1, 2, 4, 8),
// then lane 15 of a row to the next (row_bcast 15), lane 31 to the upper half.
__device__ __forceinline__ uint64_t wave_scan(uint64_t v) {
    v = add_dpp<0x111, 0xf>(v);
    v = add_dpp<0x112, 0xf>(v);
    v = add_dpp<0x114, 0xf>(v);
    v = add_dpp<0x118, 0xf>(v);
    v = add_dpp<0x142, 0xa>(v);
    return add_dpp<0x143, 0xc>(v);
}
__device__ __forceinline__ uint64_t last_lane(uint64_t v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, 63);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), 63);
    return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ uint64_t wave_total(uint64_t v) { return last_lane(wave_scan(v)); }

// The lane at which the running sum of v passes the goal (it does), and the goal less the sum before it.
__device__ __forceinline__ int lane_of(uint64_t v, uint64_t& goal) {
    const uint64_t inc = wave_scan(v), before = inc - v;
    const int at = __builtin_ctzll(__ballot(inc > goal));
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)before, at);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(before >> 32), at);
    goal -= (uint64_t)hi << 32 | lo;
    return at;
}

struct Shared {
    uint64_t hist[kBins];
    uint32_t ties[kSegs];
    uint64_t part[kRowWaves + 1];
    uint64_t found_above;
    uint32_t found_bin;
};

// Exclusive prefix of v over the workgroup's threads; total to all.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, Shared& S, uint64_t& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t inc = wave_scan(v);
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
    const uint64_t w_in = WEIGHTED && in.ties > 0 ? W.of(value_of(in.key)) : 0;
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
                              (unsigned long long)(WEIGHTED ? W.of(x[i]) : 1));
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
    const uint64_t w = WEIGHTED ? W.of(value_of(prefix)) : 1;
    return {prefix, (target - above + w - 1) / w};
}

struct Params {
    float tau, u, top_p, min_p;
    int64_t top_k;
    int code;   // data errors of the row's own numbers
};

__device__ __forceinline__ Params row_params(const SampleArgs& a, int64_t r) {
    Params P;
    P.tau = row_tau(a.T, r);
    P.u = a.u[r];
    P.top_p = a.row_top_p != nullptr ? a.row_top_p[r] : (a.top_p == 0.0f ? 1.0f : a.top_p);
    P.min_p = a.row_min_p != nullptr ? a.row_min_p[r] : a.min_p;
    P.top_k = a.row_top_k != nullptr ? a.row_top_k[r] : a.top_k;
    P.code = (tau_ok(P.tau) ? 0 : kDevErrTemperature) |
             (P.u >= 0.0f && P.u < 1.0f && P.top_p > 0.0f && P.top_p <= 1.0f && P.min_p >= 0.0f && P.min_p <= 1.0f
                  ? 0 : kDevErrSampling);
    return P;
}

// smallest integer weight that min-p keeps
__device__ __forceinline__ uint64_t weight_floor(float min_p, int shift) {
    return (uint64_t)__builtin_ceil((double)min_p * (double)(1ull << shift));
}
// integer weight that top-p has to reach, of `kept`
__device__ __forceinline__ uint64_t nucleus(float top_p, uint64_t kept) {
    const uint64_t t = (uint64_t)__builtin_ceil((double)top_p * (double)kept);
    return t < 1 ? 1 : (t > kept ? kept : t);
}

template <bool F32>
__device__ __forceinline__ void write_token(const SampleArgs& a, int64_t r, const Row<F32>& row, int64_t pos, float x,
                                            const Weights& W, float tau, double all) {
    a.token[r] = (int32_t)(pos - row.off);
    if (a.logprob != nullptr)
        a.logprob[r] = (float)(((double)x - W.top) / (double)tau -
                               log(all * __builtin_amdgcn_ldexp(1.0, -W.shift)));
}

// A whole row by radix descent: what the listed border tokens cannot resolve, in
// two to eight passes of one workgroup over the row (151,936 tokens, most of them
// in ties of thousands: top-p 427 us for one row, 560 us for 256; with top-k 595 and
// 765 us; the list takes 47 and 137 us).
// rest: what its integer weights leave out.
template <bool F32>
__device__ __attribute__((noinline)) void whole_row(const SampleArgs& a, int64_t r, const Row<F32>& row, const Params& P, const Weights& W,
                          double rest, Shared& S) {
    constexpr int kPer = Row<F32>::kPer;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t nvec = row.vectors();
    // filters: the threshold of top-k, then that of top-p within it
    Threshold T{kMaskedKey, 0};
    if (P.top_k > 0) T = descend<F32, false>(row, W, S, (uint64_t)P.top_k, T);
    // the weight of everything (for the log-probability) and of what top-k kept
    uint64_t all, kept;
    {
        uint64_t s_all = 0, s_kept = 0;
        for (int64_t k = tid; k < nvec; k += kRowThreads) {
            float x[kPer];
            row.load(k, x);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const uint64_t w = W.of(x[i]);
                s_all += w;
                s_kept += key_of(x[i]) > T.key ? w : 0;
            }
        }
        block_scan(s_all, S, all);
        block_scan(s_kept, S, kept);
        if (T.ties > 0) kept += T.ties * W.of(value_of(T.key));
    }
    if (P.top_p < 1.0f) T = descend<F32, true>(row, W, S, nucleus(P.top_p, kept), T);
    const uint64_t floor_w = weight_floor(P.min_p, W.shift);
    const uint64_t edge = T.ties > 0 ? W.of(value_of(T.key)) : 0;
    const uint64_t w_tie = T.ties > 0 && edge >= floor_w ? edge : 0;
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
                const uint64_t wx = W.of(x[i]);
                w += key > T.key && wx >= floor_w ? wx : 0;
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
    uint64_t goal = (uint64_t)((double)P.u * (double)total);
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
            const uint64_t t_inc = wave_scan(lane_t);
            uint64_t rank = ties + t_inc - lane_t;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const uint32_t key = key_of(x[i]);
                const uint64_t wx = W.of(x[i]);
                const bool tie = key == T.key;
                w[i] = tie ? (rank < T.ties ? w_tie : 0) : (key > T.key && wx >= floor_w ? wx : 0);
                rank += tie;
                lane_w += w[i];
            }
            const uint64_t w_inc = wave_scan(lane_w);
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
                write_token(a, r, row, pos, row.at(pos), W, P.tau, (double)all + rest);
            }
            done = __any(mine);
            run += last_lane(w_inc);
            ties += last_lane(t_inc);
        }
    }
}

// ------------------------------------------------------------ the five launches

struct SliceStat {
    uint32_t top, low, bad, valid;   // keys of the unmasked logits
};

// Workspace of one set of launches: [rows][slices] throughout.
struct SampleSpace {
    SliceStat* stat;
    uint64_t* weight;    // [kBins] a slice
    uint64_t* total;     // one a slice
    uint64_t* rest;      // one a slice, with a coarser step: see kRestStep
    uint32_t* count;     // [kBins] a slice
    uint32_t* listed;    // one a row
    uint64_t* list;      // [kList] a row: ~key << 32 | token
    uint64_t* run_weight;   // [kBins] a row: weight before the bin
    uint32_t* run_count;    // [kBins] a row: tokens before the bin (with top-k)
    struct Borders* borders;   // one a row
};

// What every kernel after the scan derives from the row's scan.
struct RowPlan {
    Weights W;
    Params P;
    float top, c;      // largest logit; bins per unit of logit below it
    uint64_t valid;
    bool bad, filtered;
    bool capped;       // the last bin holds tokens of weight 0 only
    __device__ __forceinline__ int bin(float x) const {
        return (int)__builtin_fminf((top - x) * c, (float)(kBins - 1));   // a NaN (0 times infinity) gives the last
    }
};

// Maximum (0), or (1), sum (2) over the 16 lanes of a row, as a uniform value.
template <int OP>
__device__ __forceinline__ uint32_t row_join(uint32_t v) {
    auto join = [](uint32_t x, uint32_t y) { return OP == 0 ? (x > y ? x : y) : OP == 1 ? x | y : x + y; };
    v = join(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false));   // row_ror 8, 4, 2, 1
    v = join(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, false));
    v = join(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, false));
    v = join(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, false));
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}

__device__ __forceinline__ RowPlan row_plan(const SampleArgs& a, const SampleSpace& w, int64_t r, int local, int slices) {
    RowPlan R;
    R.P = row_params(a, r);
    // a lane a slice, joined over the 16 lanes of a DPP row
    const int lane = threadIdx.x & 15;
    const SliceStat t = w.stat[local * slices + (lane < slices ? lane : 0)];
    const uint32_t top = row_join<0>(t.top), low = ~row_join<0>(~t.low), bad = row_join<1>(t.bad);
    R.valid = row_join<2>(lane < slices ? t.valid : 0);
    R.bad = bad != 0 || R.P.code != 0 || R.valid == 0;
    if (bad) R.P.code |= kDevErrLogit;
    R.top = value_of(top);
    R.W.top = (double)R.top;
    R.W.scale = 1.4426950408889634 / (double)R.P.tau;
    R.W.shift = a.shift;
    if (R.P.top_k <= 0 || (uint64_t)R.P.top_k >= R.valid) R.P.top_k = 0;
    R.filtered = R.P.top_k > 0 || R.P.top_p < 1.0f || R.P.min_p > 0.0f;
    // bins over the row's range, or over the 47 binary orders below the top that weights can tell apart
    const double whole = R.W.top - (double)value_of(low), most = 47.0 / R.W.scale;
    R.capped = whole > most;
    const double range = R.capped ? most : whole;
    R.c = range > 0.0 ? (float)__builtin_fmin((kBins - 1) / range, 1e38) : 0.0f;
    return R;
}

template <bool F32>
__global__ __launch_bounds__(kRowThreads) void sample_scan_kernel(SampleArgs a, SampleSpace w, int64_t r0) {
    __shared__ uint32_t s_top, s_low, s_bad, s_valid;
    const int s = blockIdx.x, slices = gridDim.x, local = blockIdx.y;
    if (threadIdx.x == 0) {
        s_top = s_bad = s_valid = 0;
        s_low = 0xffffffffu;
        if (s == 0) w.listed[local] = 0;
        if (s == 0 && local == 0 && r0 == 0) {
            a.hdr[kHdrErrCode] = 0;
            a.hdr[kHdrErrRow] = INT_MAX;
            a.hdr[kHdrCount] = 0;
        }
    }
    __syncthreads();
    const Row<F32> row(a.logits, r0 + local, a.ld, a.vocab);
    const int64_t nvec = row.vectors();
    uint32_t top = 0, low = 0xffffffffu, bad = 0, valid = 0;
    row.each(nvec * s / slices, nvec * (s + 1) / slices, [&](auto& x, int64_t) {
#pragma unroll
        for (float v : x) {
            bad |= !(v < __builtin_huge_valf());   // NaN, +infinity
            const uint32_t key = key_of(v);
            const bool in = key > kMaskedKey;
            top = in && key > top ? key : top;
            low = in && key < low ? key : low;
            valid += in;
        }
    });
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint32_t t = __shfl_xor(top, m), l = __shfl_xor(low, m);
        top = t > top ? t : top;
        low = l < low ? l : low;
        bad |= __shfl_xor(bad, m);
        valid += __shfl_xor(valid, m);
    }
    if ((threadIdx.x & 63) == 0) {
        atomicMax(&s_top, top);
        atomicMin(&s_low, low);
        atomicOr(&s_bad, bad);
        atomicAdd(&s_valid, valid);
    }
    __syncthreads();
    if (threadIdx.x == 0) w.stat[local * slices + s] = SliceStat{s_top, s_low, s_bad, s_valid};
}

// What the integer weights leave out, in integers of 2^-30: at most 2^29 for each
// of up to 2^30 tokens. A masked token and one 64 binary orders below the most
// likely one count as 2^-64 of it here, 2^-34 in all. (64 rows of 300,000 tokens,
// bf16, top-p: 105 us without, 119 us with it.)
constexpr double kRestStep = 0x1p-30;

template <bool F32, bool REST>
__global__ __launch_bounds__(kRowThreads) void sample_hist_kernel(SampleArgs a, SampleSpace w, int64_t r0) {
    __shared__ uint64_t hist[kBins];
    __shared__ uint32_t count[kBins];
    __shared__ uint64_t part[kRowWaves], part_rest[REST ? kRowWaves : 1];
    const int s = blockIdx.x, slices = gridDim.x, local = blockIdx.y;
    const RowPlan R = row_plan(a, w, r0 + local, local, slices);
    if (R.bad) return;
    const bool counted = R.P.top_k > 0;
    for (int i = threadIdx.x; i < kBins; i += kRowThreads) hist[i] = 0, count[i] = 0;
    __syncthreads();
    const Row<F32> row(a.logits, r0 + local, a.ld, a.vocab);
    const int64_t nvec = row.vectors();
    uint64_t total = 0, rest = 0;
    row.each(nvec * s / slices, nvec * (s + 1) / slices, [&](auto& x, int64_t) {
        constexpr int N = sizeof(x) / 4;
        uint64_t v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const double scaled = R.W.scaled(x[i]);
            v[i] = R.W.whole(scaled);   // 0 for a masked token
            total += v[i];
            if (REST) rest += (uint64_t)(int64_t)((scaled - (double)v[i]) * (1.0 / kRestStep));
        }
        if (!R.filtered) return;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int b = R.bin(x[i]);
            if (v[i] == 0) continue;
            atomicAdd((unsigned long long*)&hist[b], (unsigned long long)v[i]);
            if (counted) atomicAdd(&count[b], 1u);
        }
    });
    total = wave_total(total);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = total;
    if (REST) {
        rest = wave_total(rest);
        if ((threadIdx.x & 63) == 0) part_rest[threadIdx.x >> 6] = rest;
    }
    __syncthreads();
    const int64_t at = (int64_t)local * slices + s;
    if (threadIdx.x == 0) {
        uint64_t t = 0;
        for (int i = 0; i < kRowWaves; ++i) t += part[i];
        w.total[at] = t;
        if (REST) {
            uint64_t e = 0;
            for (int i = 0; i < kRowWaves; ++i) e += part_rest[i];
            w.rest[at] = e;
        }
    }
    if (!R.filtered) return;
    for (int i = threadIdx.x; i < kBins; i += kRowThreads) {
        w.weight[at * kBins + i] = hist[i];
        if (counted) w.count[at * kBins + i] = count[i];
    }
}

// The bins in which the kept prefix may end: lo .. lim, and bk, top-k's own
// (-1: none; needed beyond lim where top-p refers to what top-k keeps). Every
// token in a bin below lo is kept, none above lim (lo > lim: none is undecided). Leaves the row's exclusive
// running weight in S.hist and, with top-k, its running count in S.ties.
struct Borders {
    int lo, lim, bk;
    uint64_t all;
};

// The bins 2 t and 2 t + 1 of thread t, over the row's slices.
struct BinSums {
    uint64_t h0 = 0, h1 = 0, c0 = 0, c1 = 0;
};
__device__ __forceinline__ BinSums bin_sums(const SampleSpace& w, int local, int slices, bool counted) {
    BinSums s;
#pragma unroll 8
    for (int q = 0; q < slices; ++q) {
        const int64_t at = ((int64_t)local * slices + q) * kBins + 2 * threadIdx.x;
        const ulonglong2 h = *reinterpret_cast<const ulonglong2*>(w.weight + at);
        s.h0 += h.x, s.h1 += h.y;
        if (counted) {
            const uint2 c = *reinterpret_cast<const uint2*>(w.count + at);
            s.c0 += c.x, s.c1 += c.y;
        }
    }
    return s;
}

__device__ Borders borders(const RowPlan& R, const BinSums& sums, Shared& S) {
    const int b = 2 * threadIdx.x;
    const bool counted = R.P.top_k > 0;
    const uint64_t h0 = sums.h0, h1 = sums.h1, c0 = sums.c0, c1 = sums.c1;
    Borders B;
    uint64_t n;
    const uint64_t ew = block_scan(h0 + h1, S, B.all);
    __syncthreads();
    S.hist[b] = ew, S.hist[b + 1] = ew + h0;
    if (threadIdx.x == 0) S.found_bin = kBins;
    __syncthreads();
    B.bk = -1;
    uint64_t w_lo = B.all, w_hi = B.all;
    if (counted) {
        const uint64_t k = (uint64_t)R.P.top_k;
        const uint64_t ec = block_scan(c0 + c1, S, n);
        S.ties[b] = (uint32_t)ec, S.ties[b + 1] = (uint32_t)(ec + c0);
        if (ec < k && ec + c0 + c1 >= k) S.found_bin = ec + c0 >= k ? b : b + 1;
        __syncthreads();
        B.bk = (int)S.found_bin;
        // only tokens that weigh something are counted: with fewer of them than k, top-k decides nothing
        if (B.bk == kBins) B.bk = -1;
        if (B.bk >= 0) {
            w_lo = S.hist[B.bk];
            w_hi = B.bk + 1 < kBins ? S.hist[B.bk + 1] : B.all;
        }
    }
    B.lo = B.lim = kBins - 1;
    if (B.bk >= 0) B.lo = B.lim = B.bk;
    if (R.P.top_p < 1.0f) {
        // the target lies between those of top-k's weight without and with its border bin
        const uint64_t t0 = nucleus(R.P.top_p, w_lo > 0 ? w_lo : 1), t1 = nucleus(R.P.top_p, w_hi);
        __syncthreads();
        if (ew < t0 && ew + h0 + h1 >= t0) S.part[0] = ew + h0 >= t0 ? b : b + 1;
        if (ew < t1 && ew + h0 + h1 >= t1) S.part[1] = ew + h0 >= t1 ? b : b + 1;
        __syncthreads();
        const int p0 = (int)S.part[0], p1 = (int)S.part[1];
        B.lo = p0 < B.lo ? p0 : B.lo;
        B.lim = p1 < B.lim ? p1 : B.lim;
    }
    if (R.P.min_p > 0.0f) {
        // Of weights that round to the floor: a bin more than those of floor + 1/2 and floor - 1/2 (float
        // rounding of bin()). Where the row's range passes the largest float, bin() puts what lies farther
        // from the top into the last bin.
        const double f = (double)weight_floor(R.P.min_p, R.W.shift), one = (double)(1ull << R.W.shift);
        const double per = (double)R.c / R.W.scale;   // bins per binary order
        const double d0 = -log2((f + 0.5) / one) * per, d1 = -log2((f - 0.5) / one) * per;
        const int m0 = d0 < (double)kBins ? (int)d0 - 1 : kBins, m1 = d1 < (double)kBins ? (int)d1 + 1 : kBins;
        const bool far = (double)R.c * 3.4028234663852886e38 < (double)(kBins - 1);
        B.lo = m0 < B.lo ? (m0 > 0 ? m0 : 0) : B.lo;
        B.lim = m1 < B.lim && !far ? m1 : B.lim;
    }
    if (R.capped && B.lim == kBins - 1) B.lim = kBins - 2;
    __syncthreads();
    return B;
}

__global__ __launch_bounds__(kRowThreads) void sample_border_kernel(SampleArgs a, SampleSpace w, int64_t r0, int slices) {
    __shared__ Shared S;
    const int local = blockIdx.x;
    // the sums' loads go out with those of the row's scan (an unfiltered or bad row has no histogram: unused)
    const BinSums sums = bin_sums(w, local, slices, row_params(a, r0 + local).top_k > 0);
    const RowPlan R = row_plan(a, w, r0 + local, local, slices);
    if (R.bad || !R.filtered) return;
    const Borders B = borders(R, sums, S);
    for (int i = threadIdx.x; i < kBins; i += kRowThreads) {
        w.run_weight[(int64_t)local * kBins + i] = S.hist[i];
        if (R.P.top_k > 0) w.run_count[(int64_t)local * kBins + i] = S.ties[i];
    }
    if (threadIdx.x == 0) w.borders[local] = B;
}

template <bool F32>
__global__ __launch_bounds__(kRowThreads) void sample_gather_kernel(SampleArgs a, SampleSpace w, int64_t r0) {
    __shared__ uint64_t found[kList], below[kRowWaves];
    __shared__ uint32_t n_found, at0;
    const int s = blockIdx.x, slices = gridDim.x, local = blockIdx.y;
    const RowPlan R = row_plan(a, w, r0 + local, local, slices);
    if (R.bad || !R.filtered) return;
    if (threadIdx.x == 0) n_found = 0;
    const Borders B = w.borders[local];
    // the slice's weight in the bins below lo, for the pick kernel
    const int64_t at = (int64_t)local * slices + s;
    {
        uint64_t t = 0;
        for (int b = threadIdx.x; b < B.lo; b += kRowThreads) t += w.weight[at * kBins + b];
        t = wave_total(t);
        if ((threadIdx.x & 63) == 0) below[threadIdx.x >> 6] = t;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        uint64_t t = 0;
#pragma unroll
        for (int i = 0; i < kRowWaves; ++i) t += below[i];
        w.total[at] = t;   // in the place of the slice's whole weight, which the border kernel has summed
    }
    const int extra = R.P.top_p < 1.0f ? B.bk : -1;
    const Row<F32> row(a.logits, r0 + local, a.ld, a.vocab);
    const int64_t nvec = row.vectors();
    // the bins' tokens go to LDS first: one global atomic a workgroup
    row.each(nvec * s / slices, nvec * (s + 1) / slices, [&](auto& x, int64_t pos) {
        constexpr int N = sizeof(x) / 4;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int b = R.bin(x[i]);
            if (!((b >= B.lo && b <= B.lim) || b == extra) || !(x[i] > -__builtin_huge_valf())) continue;
            const uint32_t at = atomicAdd(&n_found, 1u);
            if (at < kList) found[at] = (uint64_t)(~key_of(x[i])) << 32 | (uint32_t)(pos + i - row.off);
        }
    });
    __syncthreads();
    const uint32_t n = n_found;
    if (n == 0) return;
    if (threadIdx.x == 0) at0 = atomicAdd(&w.listed[local], n);
    __syncthreads();
    uint64_t* list = w.list + (int64_t)local * kList;
    const uint32_t first = at0;
    for (uint32_t i = threadIdx.x; i < n && i < kList && first + i < kList; i += kRowThreads) list[first + i] = found[i];
}

struct PickShared {
    Shared S;
    uint64_t list[kList];     // sorted: descending logit, ascending token
    uint64_t before[kList];   // running weight of the list
    int first[kBins];         // first list position of a bin
    int rank[512];
    uint64_t slice[kMaxSlices];   // kept weight
    uint64_t end;
    int last, lim;
};

// Slice of a token.
template <bool F32>
__device__ __forceinline__ int slice_of(const Row<F32>& row, int64_t token, int slices) {
    const int64_t nvec = row.vectors(), vec = (token + row.off) / Row<F32>::kPer;
    int s = (int)(vec * slices / nvec);
    while (s + 1 < slices && vec >= nvec * (s + 1) / slices) ++s;
    while (s > 0 && vec < nvec * s / slices) --s;
    return s;
}

// The end of the kept prefix by one wave, a listed token a lane: lim and end
// (see the kernel), and the slices' kept weight.
template <bool F32>
__device__ __forceinline__ void short_list(const RowPlan& R, const Borders& B, const SampleSpace& w, const Row<F32>& row,
                                           int local, int slices, uint64_t entry, int listed, uint64_t slice_total,
                                           uint64_t all, PickShared& L) {
    const Shared& S = L.S;
    const int lane = threadIdx.x & 63;
    // sorted: lane p gets the entry of rank p
    int rank = 0;
    for (int i = 0; i < listed; ++i) {
        const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)entry, i);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(entry >> 32), i);
        rank += ((uint64_t)hi << 32 | lo) < entry;
    }
    if (lane >= listed) rank = lane;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_permute(4 * rank, (int)(uint32_t)entry);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_ds_permute(4 * rank, (int)(uint32_t)(entry >> 32));
    const uint64_t mine = (uint64_t)hi << 32 | lo;
    const bool in = lane < listed;
    const float x = value_of(~hi);
    const uint64_t v = in ? R.W.of(x) : 0;
    const int bin = in ? R.bin(x) : -1;
    const uint64_t before = wave_scan(v) - v;
    // the first entry of the lane's bin
    const int left = __shfl_up(bin, 1);   // by every lane: an idle one gives nothing
    const bool head = lane == 0 || left != bin;
    const uint64_t heads = __ballot(head) & (~0ull >> (63 - lane));
    const int first = 63 - __builtin_clzll(heads);
    const uint64_t in_bin = before - __shfl(before, first);
    const uint64_t k = (uint64_t)R.P.top_k;
    const uint64_t place = in && B.bk >= 0 ? S.ties[bin] + (uint64_t)(lane - first) : 0;
    const uint64_t bk_kept = wave_total(in && bin == B.bk && place < k ? v : 0);
    const uint64_t zk = B.bk >= 0 ? S.hist[B.bk] + bk_kept : all;
    const uint64_t target = R.P.top_p < 1.0f ? nucleus(R.P.top_p, zk) : ~0ull;
    const bool kept = in && (B.bk < 0 || place < k) && S.hist[in ? bin : 0] + in_bin < target &&
                      v >= weight_floor(R.P.min_p, R.W.shift);
    const uint64_t keep = __ballot(kept);
    const int last = keep != 0 ? 63 - __builtin_clzll(keep) : -1;
    const int lim = last >= 0 ? __builtin_amdgcn_readlane(bin, last) : B.lo;
    if (lane < slices) {
        uint64_t t = slice_total;
        for (int b = B.lo; b < lim; ++b) t += w.weight[((int64_t)local * slices + lane) * kBins + b];
        L.slice[lane] = t;
    }
    if (bin == lim && lane <= last)
        atomicAdd((unsigned long long*)&L.slice[slice_of(row, (int64_t)lo, slices)], (unsigned long long)v);
    if (lane == last) L.end = mine;
    if (lane == 0) {
        if (last < 0) L.end = 0;
        L.lim = lim;
    }
}

// Ascending bitonic sort in LDS; size a power of two.
__device__ __forceinline__ void sort_list(uint64_t* list, int size) {
    for (int k = 2; k <= size; k <<= 1)
        for (int j = k >> 1; j > 0; j >>= 1) {
            for (int i = threadIdx.x; i < size / 2; i += kRowThreads) {
                const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
                const uint64_t x = list[lo], y = list[hi];
                if ((x > y) == ((lo & k) == 0)) list[lo] = y, list[hi] = x;
            }
            __syncthreads();
        }
}

template <bool F32>
__global__ __launch_bounds__(kRowThreads) void sample_pick_kernel(SampleArgs a, SampleSpace w, int64_t r0, int slices) {
    constexpr int kPer = Row<F32>::kPer;
    __shared__ PickShared L;
    Shared& S = L.S;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, local = blockIdx.x;
    const int64_t r = r0 + local;
    // what the other kernels left, loaded at once with the row's scan (unused where the row has no filter)
    const uint32_t listed = w.listed[local];
    const Borders B = w.borders[local];
    const uint64_t run0 = w.run_weight[(int64_t)local * kBins + tid];
    const uint64_t run1 = w.run_weight[(int64_t)local * kBins + kRowThreads + tid];
    const uint32_t cnt0 = w.run_count[(int64_t)local * kBins + tid];
    const uint32_t cnt1 = w.run_count[(int64_t)local * kBins + kRowThreads + tid];
    const uint64_t entry = w.list[(int64_t)local * kList + tid];
    const uint64_t slice_total = w.total[(int64_t)local * slices + (lane < slices ? lane : 0)];
    const RowPlan R = row_plan(a, w, r, local, slices);
    // keeps the loads above the branches
    asm volatile("" ::"v"(run0), "v"(run1), "v"(cnt0), "v"(cnt1), "v"(entry), "v"(slice_total), "s"(listed));
    if (R.bad) {
        if (tid == 0) {
            a.token[r] = -1;
            if (a.logprob != nullptr) a.logprob[r] = R.P.code != 0 ? __builtin_nanf("") : 0.0f;
            if (R.P.code != 0) {
                atomicOr(a.hdr + kHdrErrCode, R.P.code);
                atomicMin(a.hdr + kHdrErrRow, (int32_t)r);
            }
        }
        return;
    }
    double rest = 0.0;
    if (a.shift < kWeightBits)
        rest = (double)(int64_t)wave_total(lane < slices ? w.rest[(int64_t)local * slices + lane] : 0) * kRestStep;
    const Row<F32> row(a.logits, r, a.ld, a.vocab);
    const int64_t nvec = row.vectors();
    const uint64_t floor_w = weight_floor(R.P.min_p, R.W.shift);
    // a token is kept in bins below `lim`, and in `lim` up to `end` in the list's order
    int lim = kBins;
    uint64_t end = 0, all = 0;
    if (R.filtered) {
        if (listed > kList) {
            whole_row<F32>(a, r, row, R.P, R.W, rest, S);
            return;
        }
        all = B.all;
        S.hist[tid] = run0, S.hist[kRowThreads + tid] = run1;
        if (R.P.top_k > 0) S.ties[tid] = cnt0, S.ties[kRowThreads + tid] = cnt1;
        if (listed <= 64) {
            // a wave holds the list: no workgroup-wide step until the answer
            __syncthreads();
            if (wave == 0) short_list<F32>(R, B, w, row, local, slices, entry, (int)listed, slice_total, all, L);
            __syncthreads();
            lim = L.lim;
            end = L.end;
        } else {
            int size = 64;
            while (size < (int)listed) size <<= 1;
            for (int i = tid; i < size; i += kRowThreads)
                L.before[i] = i >= (int)listed ? ~0ull : i == tid ? entry : w.list[(int64_t)local * kList + i];
            if (tid == 0) L.last = -1;
            __syncthreads();
            if (listed <= 512) {
                // an entry's rank is the number of entries before it (all differ); 1024 / size threads share the count
                for (int i = tid; i < size; i += kRowThreads) L.rank[i] = 0;
                __syncthreads();
                const int e = tid & (size - 1), parts = kRowThreads / size;
                const int each = ((int)listed + parts - 1) / parts, i0 = tid / size * each;
                const int i1 = i0 + each < (int)listed ? i0 + each : (int)listed;
                if (e < (int)listed) {
                    int rank = 0;
                    const uint64_t mine = L.before[e];
#pragma unroll 8
                    for (int i = i0; i < i1; ++i) rank += L.before[i] < mine;
                    atomicAdd(&L.rank[e], rank);
                }
                __syncthreads();
                if (tid < (int)listed) L.list[L.rank[tid]] = L.before[tid];
                __syncthreads();
            } else {
                for (int i = tid; i < size; i += kRowThreads) L.list[i] = L.before[i];
                __syncthreads();
                sort_list(L.list, size);
            }
            // running weight of the list: four consecutive entries a thread
            const int p0 = 4 * tid;
            uint64_t v[4], sum = 0;
            int bin[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool in = p0 + i < (int)listed;
                const float x = value_of(~(uint32_t)((in ? L.list[p0 + i] : 0) >> 32));
                v[i] = in ? R.W.of(x) : 0;
                bin[i] = in ? R.bin(x) : -1;
                sum += v[i];
            }
            uint64_t total;
            uint64_t run = block_scan(sum, S, total);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (bin[i] >= 0) {
                    const int p = p0 + i;
                    L.before[p] = run;
                    run += v[i];
                    const float px = p > 0 ? value_of(~(uint32_t)(L.list[p - 1] >> 32)) : 0.0f;
                    if (p == 0 || R.bin(px) != bin[i]) L.first[bin[i]] = p;
                }
            __syncthreads();
            // what top-k keeps, then the three rules for each listed token
            uint64_t in_bk = 0;
            const uint64_t k = (uint64_t)R.P.top_k;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (bin[i] >= 0 && bin[i] == B.bk && S.ties[B.bk] + (uint64_t)(p0 + i - L.first[B.bk]) < k) in_bk += v[i];
            block_scan(in_bk, S, total);
            const uint64_t zk = B.bk >= 0 ? S.hist[B.bk] + total : all;
            const uint64_t target = R.P.top_p < 1.0f ? nucleus(R.P.top_p, zk) : ~0ull;
            int last = -1;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (bin[i] >= 0) {
                    const int p = p0 + i, f = L.first[bin[i]];
                    const bool rank_ok = B.bk < 0 || S.ties[bin[i]] + (uint64_t)(p - f) < k;
                    const bool sum_ok = S.hist[bin[i]] + (L.before[p] - L.before[f]) < target;
                    if (rank_ok && sum_ok && v[i] >= floor_w) last = p;
                }
            if (last >= 0) atomicMax(&L.last, last);
            __syncthreads();
            last = L.last;
            lim = B.lo;   // nothing listed is kept: the prefix ends before the listed bins
            if (last >= 0) {
                end = L.list[last];
                lim = R.bin(value_of(~(uint32_t)(end >> 32)));
            }
            // kept weight of each slice: its bins below lo (from the gather kernel) and on to lim, and the
            // listed tokens of lim
            for (int s = wave; s < slices; s += kRowWaves) {
                const int64_t at = (int64_t)local * slices + s;
                uint64_t t = 0;
                for (int b = B.lo + lane; b < lim; b += 64) t += w.weight[at * kBins + b];
                t = wave_total(t);
                if (lane == s) L.slice[s] = slice_total + t;
            }
            __syncthreads();
            if (last >= 0)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (bin[i] == lim && p0 + i <= last) {
                        const int s = slice_of(row, (int64_t)(uint32_t)L.list[p0 + i], slices);
                        atomicAdd((unsigned long long*)&L.slice[s], (unsigned long long)v[i]);
                    }
            __syncthreads();
        }
    }
    // the slice in which the goal lies, and the goal within it
    const uint64_t sv = lane < slices ? (R.filtered ? L.slice[lane] : slice_total) : 0;
    const uint64_t total = wave_total(sv);
    if (!R.filtered) all = total;
    uint64_t goal = (uint64_t)((double)R.P.u * (double)total);
    goal = goal < total ? goal : total - 1;
    const int s = lane_of(sv, goal);
    const int64_t k0 = nvec * s / slices, k1 = nvec * (s + 1) / slices;
    // Weights of a vector's kept tokens (0 for the others and for masked ones).
    // With a last kept token in the list, the kept ones are those at or before
    // it in the list's order: a larger logit, or an equal one and no larger an
    // index (the bins need not be made again). Without one, the bins below lim.
    const bool by_end = lim == kBins || end != 0;
    const float x_end = lim == kBins ? -__builtin_huge_valf() : value_of(~(uint32_t)(end >> 32));
    const int64_t p_end = lim == kBins ? -1 : (int64_t)(uint32_t)end + row.off;
    auto weigh = [&](const float (&x)[kPer], int64_t pos, uint64_t (&v)[kPer]) {
        bool in[kPer], any = false;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            in[i] = by_end ? x[i] > x_end || (x[i] == x_end && pos + i <= p_end) : R.bin(x[i]) < lim;
            any |= in[i];
            v[i] = 0;
        }
        if (any)
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const uint64_t w1 = R.W.of(x[i]);
                v[i] = in[i] ? w1 : 0;
            }
    };
    // Narrow the slice down: its vectors in 16 runs, a wave each, the run in
    // which the goal lies, again until a vector a thread is left.
    int64_t lo = k0, hi = k1;
    while (hi - lo > kRowThreads) {
        const int64_t run = (hi - lo + kRowWaves - 1) / kRowWaves;
        const int64_t e0 = lo + run * wave, e1 = e0 + run < hi ? e0 + run : hi;
        uint64_t t = 0;
        if (row.whole_from() < row.whole_to())
            for (int64_t k = e0 + lane; k < e1; k += 4 * 64) {
                float x[4][kPer];
                row.load4(k, e1, x);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (k - lane + 64 * q >= e1) break;
                    uint64_t v[kPer];
                    weigh(x[q], (k + 64 * q) * kPer, v);
#pragma unroll
                    for (int i = 0; i < kPer; ++i) t += v[i];
                }
            }
        // the run's ragged vectors, a position a lane
        for (int64_t k = e0; k < e1; k = k + 1 < row.whole_to() ? row.whole_to() : k + 1) {
            const int64_t pos = k * kPer + lane;
            if ((k < row.whole_from() || k >= row.whole_to()) && lane < kPer && pos >= row.off && pos < row.end) {
                float x[kPer];
                uint64_t v[kPer];
#pragma unroll
                for (int i = 0; i < kPer; ++i) x[i] = -__builtin_huge_valf();
                x[0] = row.at(pos);
                weigh(x, pos, v);
                t += v[0];
            }
        }
        t = wave_total(t);
        if (lane == 0) S.part[wave] = t;
        __syncthreads();
        lo += run * lane_of(lane < kRowWaves ? S.part[lane] : 0, goal);
        hi = lo + run < hi ? lo + run : hi;
        __syncthreads();
    }
    const int64_t k = lo + tid;
    float x[kPer];
    uint64_t v[kPer], mine = 0;
    if (k < hi) {
        row.load(k, x);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] = -__builtin_huge_valf();
    }
    weigh(x, k * kPer, v);
#pragma unroll
    for (int i = 0; i < kPer; ++i) mine += v[i];
    const uint64_t inc = wave_scan(mine);
    if (lane == 63) S.part[wave] = inc;
    __syncthreads();
    if (wave != lane_of(lane < kRowWaves ? S.part[lane] : 0, goal)) return;
    uint64_t c = inc - mine;
    if (c <= goal && c + mine > goal) {
        int pick = kPer;
        float logit = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            c += v[i];
            if (pick == kPer && c > goal) pick = i, logit = x[i];
        }
        write_token(a, r, row, k * kPer + pick, logit, R.W, R.P.tau, (double)all + rest);
    }
}

// Workgroups a row: four to a compute unit over all rows, each with some
// kSliceTokens tokens at least (a slice costs its histogram's traffic and its
// share of the row's; 64 rows of 128,256: 8 slices 72 us, 16 slices 82 us; 256
// rows of 151,936: 4 slices 153 us, 2 slices 171 us, 8 slices 164 us).
constexpr int64_t kSliceTokens = 16384;
int slices_of(int64_t rows, int64_t vocab) {
    int64_t s = 4 * 256 / rows;
    const int64_t most = cdiv(vocab, kSliceTokens);
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : (s < kMaxSlices ? s : kMaxSlices));
}

template <bool F32>
void sample_rows(const SampleArgs& a, const SampleSpace& w, hipStream_t s) {
    const bool filters = a.row_top_k != nullptr || a.row_top_p != nullptr || a.row_min_p != nullptr || a.top_k > 0 ||
                         (a.top_p > 0.0f && a.top_p < 1.0f) || a.min_p > 0.0f;
    for (int64_t r0 = 0; r0 < a.n; r0 += kChunkRows) {
        const int rows = (int)(a.n - r0 < kChunkRows ? a.n - r0 : kChunkRows);
        const int slices = slices_of(rows, a.vocab);
        const dim3 grid(slices, rows);
        sample_scan_kernel<F32><<<grid, kRowThreads, 0, s>>>(a, w, r0);
        if (a.shift < kWeightBits)
            sample_hist_kernel<F32, true><<<grid, kRowThreads, 0, s>>>(a, w, r0);
        else
            sample_hist_kernel<F32, false><<<grid, kRowThreads, 0, s>>>(a, w, r0);
        if (filters) sample_border_kernel<<<rows, kRowThreads, 0, s>>>(a, w, r0, slices);
        if (filters) sample_gather_kernel<F32><<<grid, kRowThreads, 0, s>>>(a, w, r0);
        sample_pick_kernel<F32><<<rows, kRowThreads, 0, s>>>(a, w, r0, slices);
    }
}

// Regions after the header; returns the size.
size_t carve(int64_t n, int64_t vocab, char* base, SampleSpace& w) {
    const int64_t rows = n < 1 ? 1 : (n < kChunkRows ? n : kChunkRows);
    // the most slices any set of up to `rows` rows has
    int64_t parts = 0;
    for (int64_t r = 1; r <= rows; ++r) parts = r * slices_of(r, vocab) > parts ? r * slices_of(r, vocab) : parts;
    size_t off = 256;
    auto take = [&](int64_t bytes) {
        char* p = base + off;
        off += (size_t)round_up(bytes, 256);
        return p;
    };
    w.stat = (SliceStat*)take(parts * (int64_t)sizeof(SliceStat));
    w.weight = (uint64_t*)take(8 * parts * kBins);
    w.total = (uint64_t*)take(8 * parts);
    w.rest = (uint64_t*)take(8 * parts);
    w.count = (uint32_t*)take(4 * parts * kBins);
    w.listed = (uint32_t*)take(4 * rows);
    w.list = (uint64_t*)take(8 * rows * kList);
    w.run_weight = (uint64_t*)take(8 * rows * kBins);
    w.run_count = (uint32_t*)take(4 * rows * kBins);
    w.borders = (Borders*)take(rows * (int64_t)sizeof(Borders));
    return off;
}

}  // namespace

size_t sample_workspace(int64_t n, int64_t vocab) {
    SampleSpace w;
    return carve(n, vocab, nullptr, w);
}

void launch_sample(const SampleArgs& a, void* workspace, hipStream_t s) {
    SampleSpace w;
    carve(a.n, a.vocab, (char*)workspace, w);
    if (a.logits_f32)
        sample_rows<true>(a, w, s);
    else
        sample_rows<false>(a, w, s);
}

}  // namespace lmhead
