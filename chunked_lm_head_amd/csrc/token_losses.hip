// token_losses.hip — the clipped policy loss and the preference loss on packed
// per-token log-probabilities, forward and backward.
//
// Mathematics (lmhead_train.h). Policy: L = -A rho + b KL, loss = sum_t w_s L_t,
// dlogp_t = g w_s (-A r [not clipped] + b KL'). The border of rho is compared as
// logp - old against log(1 + eps) in 64 bits: near it the fp32 ratio could fall
// on either side. Preference: s_q = sum or mean of logp - ref over a sequence, h
// = beta (s_chosen - s_rejected) - margin; dlogp_t = g coef_q.
//
// 12 to 24 bytes per token and direction and few operations: small batches are
// bound by launches, large ones by memory. So up to 8192 tokens are one launch
// of one workgroup; above, tiles of 2048 tokens leave 64-bit partial sums and a
// second launch (a third for the sequence mean) adds them in order.
//
// Sequences and tiles. A tile's partial of sequence s stands at slot tile + s:
// along the packed tokens either the tile or the sequence moves on, so no two
// meeting pairs share a slot, and tiles + sequences slots hold them all.
#include "host_util.h"
#include "train_kernels.h"

namespace lmhead {

namespace {

constexpr int kTileThreads = 256, kWholeThreads = 1024;
constexpr int kEach = 8;   // tokens per thread
constexpr int64_t kWholeTokens = kWholeThreads * kEach;
constexpr int64_t kTileTokens = kTileThreads * kEach;

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

// Sum over the workgroup, for every thread, in the order of lanes and waves. red: a
// double per wave.
template <int THREADS>
__device__ __forceinline__ double group_sum(double v, double* red) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
    for (int w = 0; w < THREADS / 64; ++w) s += red[w];
    return s;
}

__device__ __forceinline__ int64_t border(const Tokens& t, int64_t s) {
    if (t.cu == nullptr) return s <= 0 ? 0 : t.n;
    const int64_t v = t.cu[s];
    return v < 0 ? 0 : v < t.n ? v : t.n;
}

// The last sequence whose first token is at or before i (-1: none), searched by
// a wave: 64 places at once, so two steps find one of 4096 borders.
__device__ __forceinline__ int64_t sequence_at(const Tokens& t, int64_t i) {
    if (t.cu == nullptr) return 0;
    int64_t lo = 0, hi = t.sequences + 1;   // number of borders <= i
    const int lane = threadIdx.x & 63;
    while (lo < hi) {
        const int64_t step = (hi - lo + 63) >> 6, at = lo + lane * step;
        const int c = __popcll(__ballot(at < hi && border(t, at) <= i));
        if (c == 0) break;
        const int64_t end = lo + c * step;
        lo = lo + (c - 1) * step + 1;
        hi = end < hi ? end : hi;
    }
    return lo - 1;
}
// The same for one token between two known answers.
__device__ __forceinline__ int64_t sequence_between(const Tokens& t, int64_t lo, int64_t hi, int64_t i) {
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (border(t, mid) <= i) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

struct Term {
    float loss, slope, kl, ratio, back;
    bool clipped;
};

// exp(-x) - 1 + x; for |x| <= 1/2, where the difference would cancel, its
// series x^2 sum_k (-x)^k / (k + 2)!, whose first term left out is below 2^-24
// of the sum
__device__ __forceinline__ float k3_of(float x) {
    if (!(fabsf(x) <= 0.5f)) return expf(-x) - 1.0f + x;
    const float y = -x;
    float s = 1.0f / 40320.0f;
    s = __builtin_fmaf(y, s, 1.0f / 5040.0f);
    s = __builtin_fmaf(y, s, 1.0f / 720.0f);
    s = __builtin_fmaf(y, s, 1.0f / 120.0f);
    s = __builtin_fmaf(y, s, 1.0f / 24.0f);
    s = __builtin_fmaf(y, s, 1.0f / 6.0f);
    s = __builtin_fmaf(y, s, 0.5f);
    return x * x * s;
}

__device__ __forceinline__ Term policy_term(const PolicyArgs& a, float logp, float old, float ref, float adv) {
    Term o;
    const double gap = (double)logp - (double)old;
    const float d = (float)gap;
    o.ratio = expf(d);
    float rho;
    if (adv >= 0.0f) {
        o.clipped = gap > a.log_high;
        rho = o.clipped ? a.high : o.ratio;
    } else {
        o.clipped = gap < a.log_low;
        rho = o.clipped ? a.low : o.ratio;
        if (gap > a.log_dual) {
            o.clipped = true;
            rho = a.dual;
        }
    }
    o.loss = -adv * rho;
    o.slope = o.clipped ? 0.0f : -adv * o.ratio;
    o.back = k3_of(d);
    o.kl = 0.0f;
    if (a.ref_logp != nullptr) {
        const float x = logp - ref;
        float dk;
        if (a.kl_kind == 1) {
            o.kl = x;
            dk = 1.0f;
        } else if (a.kl_kind == 2) {
            o.kl = 0.5f * x * x;
            dk = x;
        } else {
            o.kl = k3_of(x);
            dk = -expm1f(-x);
        }
        o.loss = __builtin_fmaf(a.kl_weight, o.kl, o.loss);
        o.slope = __builtin_fmaf(a.kl_weight, dk, o.slope);
    }
    return o;
}

// ------------------------------------------------------------------- policy

struct Sums {
    double loss, count, kl, clipped, ratio, back;
};
struct Part {
    double sum, count;
};

struct Tile {
    int64_t t0, t1, first, last;   // tokens; sequences at the first and last one
};
template <int THREADS>
__device__ __forceinline__ Tile tile_at(const Tokens& t, int64_t index) {
    Tile o;
    o.t0 = index * THREADS * kEach;
    o.t1 = o.t0 + THREADS * kEach < t.n ? o.t0 + THREADS * kEach : t.n;
    o.first = sequence_at(t, o.t0);
    o.last = o.t1 - o.t0 > 1 ? sequence_at(t, o.t1 - 1) : o.first;
    return o;
}

// A tile's terms, summed; per token kept in LDS where sequences are summed apart.
template <int THREADS, bool SEQ>
__device__ __forceinline__ Sums policy_tile(const PolicyArgs& a, const Tile& tile, float* kept, uint8_t* counts,
                                            double* red) {
    Sums s = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
    float logp[kEach], old[kEach], ref[kEach], adv[kEach];
    bool valid[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int64_t i = tile.t0 + k * THREADS + threadIdx.x;
        valid[k] = false;
        logp[k] = old[k] = ref[k] = adv[k] = 0.0f;
        if (i >= tile.t1) continue;
        const int64_t q = sequence_between(a.t, tile.first, tile.last, i);
        valid[k] = q >= 0 && q < a.t.sequences && (a.t.targets == nullptr || a.t.targets[i] >= 0);
        logp[k] = a.logp[i];
        old[k] = a.old_logp != nullptr ? a.old_logp[i] : logp[k];
        if (a.ref_logp != nullptr) ref[k] = a.ref_logp[i];
        if (!a.per_sequence) adv[k] = a.advantage[i];
        else if (valid[k]) adv[k] = a.advantage[q];
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const Term o = policy_term(a, logp[k], old[k], ref[k], adv[k]);
        if (valid[k]) {   // whatever stands in the other places takes no part
            s.loss += (double)o.loss;
            s.count += 1.0;
            s.kl += (double)o.kl;
            s.clipped += o.clipped ? 1.0 : 0.0;
            s.ratio += (double)o.ratio;
            s.back += (double)o.back;
        }
        if (SEQ) {
            kept[k * THREADS + threadIdx.x] = o.loss;
            counts[k * THREADS + threadIdx.x] = valid[k];
        }
    }
    if (!SEQ) s.loss = group_sum<THREADS>(s.loss, red);
    s.count = group_sum<THREADS>(s.count, red);
    s.kl = group_sum<THREADS>(s.kl, red);
    s.clipped = group_sum<THREADS>(s.clipped, red);
    s.ratio = group_sum<THREADS>(s.ratio, red);
    s.back = group_sum<THREADS>(s.back, red);   // also: kept and counts are written
    return s;
}

// One sequence's part of a tile, from LDS, by one wave.
__device__ __forceinline__ Part part_of(const Tokens& t, const Tile& tile, int64_t q, const float* kept,
                                        const uint8_t* counts) {
    int64_t from = border(t, q), to = border(t, q + 1);
    from = from > tile.t0 ? from : tile.t0;
    to = to < tile.t1 ? to : tile.t1;
    Part p = {0.0, 0.0};
    for (int64_t i = from + (threadIdx.x & 63); i < to; i += 64)
        if (counts[i - tile.t0]) {
            p.sum += (double)kept[i - tile.t0];
            p.count += 1.0;
        }
    p.sum = wave_sum(p.sum);
    p.count = wave_sum(p.count);
    return p;
}

// The same over the tiles that a sequence touches, from their slots.
__device__ __forceinline__ Part part_of(const Tokens& t, int64_t q, const Part* slots) {
    const int64_t from = border(t, q), to = border(t, q + 1);
    Part p = {0.0, 0.0};
    if (from < to)
        for (int64_t tile = from / kTileTokens + (threadIdx.x & 63); tile <= (to - 1) / kTileTokens; tile += 64) {
            const Part o = slots[tile + q];
            p.sum += o.sum;
            p.count += o.count;
        }
    p.sum = wave_sum(p.sum);
    p.count = wave_sum(p.count);
    return p;
}

__device__ __forceinline__ double share(int64_t given, double counted) {
    const double d = given >= 0 ? (double)given : counted;
    return d > 0.0 ? 1.0 / d : 0.0;
}

// A sequence's weight in the sequence mean; returns its mean times its share.
__device__ __forceinline__ double weigh(const PolicyArgs& a, int64_t q, const Part& p) {
    const double w = p.count > 0.0 ? share(a.num_valid, (double)a.t.sequences) / p.count : 0.0;
    if ((threadIdx.x & 63) == 0) a.weights[q] = (float)w;
    return w > 0.0 ? w * p.sum : 0.0;
}

// What is left once the totals are known: called by every thread of the last workgroup.
__device__ __forceinline__ void policy_end(const PolicyArgs& a, const Sums& s, double sequence_means, int threads) {
    const bool seq = a.reduction == 2;
    const double w = a.reduction == 0 ? share(a.num_valid, s.count) : 1.0;
    if (!seq)   // one weight for all
        for (int64_t q = threadIdx.x; q < a.t.sequences; q += threads) a.weights[q] = (float)w;
    if (threadIdx.x != 0) return;
    a.loss[0] = (float)(seq ? sequence_means : w > 0.0 ? w * s.loss : 0.0);
    if (a.stats == nullptr) return;
    const double each = s.count > 0.0 ? 1.0 / s.count : 0.0;
    a.stats[0] = (float)(s.kl * each);
    a.stats[1] = (float)(s.clipped * each);
    a.stats[2] = (float)(s.ratio * each);
    a.stats[3] = (float)(s.back * each);
}

template <bool SEQ>
__global__ __launch_bounds__(kWholeThreads) void policy_whole_kernel(PolicyArgs a) {
    __shared__ double red[kWholeThreads / 64];
    __shared__ float kept[SEQ ? kWholeTokens : 1];
    __shared__ uint8_t counts[SEQ ? kWholeTokens : 1];
    const Tile tile = tile_at<kWholeThreads>(a.t, 0);
    const Sums s = policy_tile<kWholeThreads, SEQ>(a, tile, kept, counts, red);
    double means = 0.0;
    if (SEQ) {
        for (int64_t q = threadIdx.x >> 6; q < a.t.sequences; q += kWholeThreads / 64)
            means += weigh(a, q, part_of(a.t, tile, q, kept, counts));
        means = group_sum<kWholeThreads>((threadIdx.x & 63) == 0 ? means : 0.0, red);
    }
    policy_end(a, s, means, kWholeThreads);
}

template <bool SEQ>
__global__ __launch_bounds__(kTileThreads) void policy_tiles_kernel(PolicyArgs a, Sums* tiles, Part* slots) {
    __shared__ double red[kTileThreads / 64];
    __shared__ float kept[SEQ ? kTileTokens : 1];
    __shared__ uint8_t counts[SEQ ? kTileTokens : 1];
    const Tile tile = tile_at<kTileThreads>(a.t, blockIdx.x);
    const Sums s = policy_tile<kTileThreads, SEQ>(a, tile, kept, counts, red);
    if (threadIdx.x == 0) tiles[blockIdx.x] = s;
    if (!SEQ) return;
    for (int64_t q = (tile.first > 0 ? tile.first : 0) + (threadIdx.x >> 6); q <= tile.last && q < a.t.sequences;
         q += kTileThreads / 64) {
        const Part p = part_of(a.t, tile, q, kept, counts);
        if ((threadIdx.x & 63) == 0) slots[blockIdx.x + q] = p;
    }
}

__global__ __launch_bounds__(kTileThreads) void policy_sequences_kernel(PolicyArgs a, const Part* slots, double* means) {
    const int64_t q = (int64_t)blockIdx.x * (kTileThreads / 64) + (threadIdx.x >> 6);
    if (q >= a.t.sequences) return;
    const double m = weigh(a, q, part_of(a.t, q, slots));
    if ((threadIdx.x & 63) == 0) means[q] = m;
}

__global__ __launch_bounds__(kWholeThreads) void policy_join_kernel(PolicyArgs a, const Sums* tiles, int64_t count,
                                                                    const double* means) {
    __shared__ double red[kWholeThreads / 64];
    Sums s = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < count; i += kWholeThreads) {
        const Sums o = tiles[i];
        s.loss += o.loss;
        s.count += o.count;
        s.kl += o.kl;
        s.clipped += o.clipped;
        s.ratio += o.ratio;
        s.back += o.back;
    }
    double m = 0.0;
    if (a.reduction == 2)
#pragma unroll 4
        for (int64_t q = threadIdx.x; q < a.t.sequences; q += kWholeThreads) m += means[q];
    s.loss = group_sum<kWholeThreads>(a.reduction == 2 ? m : s.loss, red);
    s.count = group_sum<kWholeThreads>(s.count, red);
    s.kl = group_sum<kWholeThreads>(s.kl, red);
    s.clipped = group_sum<kWholeThreads>(s.clipped, red);
    s.ratio = group_sum<kWholeThreads>(s.ratio, red);
    s.back = group_sum<kWholeThreads>(s.back, red);
    policy_end(a, s, s.loss, kWholeThreads);
}

constexpr int kBackEach = 4;
constexpr int64_t kBackTile = kTileThreads * kBackEach;

// The tile of a backward workgroup: kBackEach tokens per thread.
__device__ __forceinline__ Tile back_tile(const Tokens& t) {
    Tile o;
    o.t0 = (int64_t)blockIdx.x * kBackTile;
    o.t1 = o.t0 + kBackTile < t.n ? o.t0 + kBackTile : t.n;
    o.first = sequence_at(t, o.t0);
    o.last = sequence_at(t, o.t1 - 1);
    return o;
}

__global__ __launch_bounds__(kTileThreads) void policy_bwd_kernel(PolicyArgs a, const float* grad, float* dlogp) {
    const Tile tile = back_tile(a.t);
    const float g = grad[0];
#pragma unroll
    for (int k = 0; k < kBackEach; ++k) {
        const int64_t i = tile.t0 + k * kTileThreads + threadIdx.x;
        if (i >= tile.t1) continue;
        const int64_t q = sequence_between(a.t, tile.first, tile.last, i);
        float d = 0.0f;
        if (q >= 0 && q < a.t.sequences && (a.t.targets == nullptr || a.t.targets[i] >= 0)) {
            const float logp = a.logp[i];
            const Term o = policy_term(a, logp, a.old_logp != nullptr ? a.old_logp[i] : logp,
                                       a.ref_logp != nullptr ? a.ref_logp[i] : 0.0f,
                                       a.advantage[a.per_sequence ? q : i]);
            d = g * (a.weights[q] * o.slope);
        }
        dlogp[i] = d;
    }
}

// --------------------------------------------------------------- preference

template <int THREADS>
__device__ __forceinline__ void preference_tile(const PreferenceArgs& a, const Tile& tile, float* kept, uint8_t* counts) {
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int64_t i = tile.t0 + k * THREADS + threadIdx.x;
        float gain = 0.0f;
        bool valid = false;
        if (i < tile.t1) {
            gain = a.logp[i] - (a.ref_logp != nullptr ? a.ref_logp[i] : 0.0f);
            valid = a.t.targets == nullptr || a.t.targets[i] >= 0;
        }
        kept[k * THREADS + threadIdx.x] = gain;
        counts[k * THREADS + threadIdx.x] = valid;
    }
    __syncthreads();
}

// One pair from its sequences' sums: writes the rewards and coefficients, returns its share of the loss.
__device__ __forceinline__ double pair_loss(const PreferenceArgs& a, int64_t pair, Part c, Part r) {
    const int64_t pairs = a.t.sequences / 2;
    const double one = share(a.num_pairs, (double)pairs);
    const double fc = a.average && c.count > 0.0 ? 1.0 / c.count : 1.0;
    const double fr = a.average && r.count > 0.0 ? 1.0 / r.count : 1.0;
    const double sc = c.sum * fc, sr = r.sum * fr;
    const double h = a.beta * (sc - sr) - a.margin;
    double loss, slope;
    if (a.kind == 0) {
        // softplus(x) = max(x, 0) + log(1 + e^-|x|)
        const double tail = log1p(exp(-fabs(h)));
        const double minus = (h < 0.0 ? -h : 0.0) + tail, plus = (h > 0.0 ? h : 0.0) + tail;
        loss = (1.0 - a.smoothing) * minus + a.smoothing * plus;
        slope = a.smoothing / (1.0 + exp(-h)) - (1.0 - a.smoothing) / (1.0 + exp(h));
        if (h != h) loss = slope = h;
    } else if (a.kind == 1) {
        loss = h < 1.0 ? 1.0 - h : h != h ? h : 0.0;
        slope = h < 1.0 ? -1.0 : h != h ? h : 0.0;
    } else {
        const double d = (h - 0.5) / a.beta;
        loss = d * d;
        slope = 2.0 * d / a.beta;
    }
    if ((threadIdx.x & 63) == 0) {
        const double k = one > 0.0 ? a.beta * slope * one : 0.0;
        a.coef[pair] = (float)(k * fc);
        a.coef[pairs + pair] = (float)(-k * fr);
        if (a.rewards != nullptr) {
            a.rewards[pair] = (float)(a.beta * sc);
            a.rewards[pairs + pair] = (float)(a.beta * sr);
        }
    }
    return one > 0.0 ? loss * one : 0.0;
}

__global__ __launch_bounds__(kWholeThreads) void preference_whole_kernel(PreferenceArgs a) {
    __shared__ double red[kWholeThreads / 64];
    __shared__ float kept[kWholeTokens];
    __shared__ uint8_t counts[kWholeTokens];
    Tile tile = {0, a.t.n, 0, 0};
    preference_tile<kWholeThreads>(a, tile, kept, counts);
    const int64_t pairs = a.t.sequences / 2;
    double loss = 0.0;
    for (int64_t j = threadIdx.x >> 6; j < pairs; j += kWholeThreads / 64)
        loss += pair_loss(a, j, part_of(a.t, tile, j, kept, counts), part_of(a.t, tile, pairs + j, kept, counts));
    loss = group_sum<kWholeThreads>((threadIdx.x & 63) == 0 ? loss : 0.0, red);
    if (threadIdx.x == 0) a.loss[0] = (float)loss;
}

__global__ __launch_bounds__(kTileThreads) void preference_tiles_kernel(PreferenceArgs a, Part* slots) {
    __shared__ float kept[kTileTokens];
    __shared__ uint8_t counts[kTileTokens];
    const Tile tile = tile_at<kTileThreads>(a.t, blockIdx.x);
    preference_tile<kTileThreads>(a, tile, kept, counts);
    for (int64_t q = (tile.first > 0 ? tile.first : 0) + (threadIdx.x >> 6); q <= tile.last && q < a.t.sequences;
         q += kTileThreads / 64) {
        const Part p = part_of(a.t, tile, q, kept, counts);
        if ((threadIdx.x & 63) == 0) slots[blockIdx.x + q] = p;
    }
}

__global__ __launch_bounds__(kTileThreads) void preference_pairs_kernel(PreferenceArgs a, const Part* slots, double* each) {
    const int64_t j = (int64_t)blockIdx.x * (kTileThreads / 64) + (threadIdx.x >> 6), pairs = a.t.sequences / 2;
    if (j >= pairs) return;
    const double l = pair_loss(a, j, part_of(a.t, j, slots), part_of(a.t, pairs + j, slots));
    if ((threadIdx.x & 63) == 0) each[j] = l;
}

__global__ __launch_bounds__(kWholeThreads) void preference_join_kernel(const double* each, int64_t count, float* loss) {
    __shared__ double red[kWholeThreads / 64];
    double s = 0.0;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < count; i += kWholeThreads) s += each[i];
    s = group_sum<kWholeThreads>(s, red);
    if (threadIdx.x == 0) loss[0] = (float)s;
}

__global__ __launch_bounds__(kTileThreads) void preference_bwd_kernel(Tokens t, const float* grad, const float* coef,
                                                                      float* dlogp) {
    const Tile tile = back_tile(t);
    const float g = grad[0];
#pragma unroll
    for (int k = 0; k < kBackEach; ++k) {
        const int64_t i = tile.t0 + k * kTileThreads + threadIdx.x;
        if (i >= tile.t1) continue;
        const int64_t q = sequence_between(t, tile.first, tile.last, i);
        const bool valid = q >= 0 && q < t.sequences && (t.targets == nullptr || t.targets[i] >= 0);
        dlogp[i] = valid ? g * coef[q] : 0.0f;
    }
}

}  // namespace

size_t policy_workspace(int64_t n, int64_t sequences, int reduction) {
    if (n <= kWholeTokens) return 256;
    const int64_t tiles = cdiv(n, kTileTokens);
    int64_t bytes = round_up(tiles * (int64_t)sizeof(Sums), 256);
    if (reduction == 2)
        bytes += round_up((tiles + sequences) * (int64_t)sizeof(Part), 256) + round_up(sequences * 8, 256);
    return (size_t)bytes;
}

void launch_policy(const PolicyArgs& a, void* workspace, hipStream_t s) {
    const bool seq = a.reduction == 2;
    if (a.t.n <= kWholeTokens) {
        if (seq) policy_whole_kernel<true><<<1, kWholeThreads, 0, s>>>(a);
        else policy_whole_kernel<false><<<1, kWholeThreads, 0, s>>>(a);
        return;
    }
    const int64_t tiles = cdiv(a.t.n, kTileTokens);
    char* w = (char*)workspace;
    Sums* sums = (Sums*)w;
    Part* slots = (Part*)(w + round_up(tiles * (int64_t)sizeof(Sums), 256));
    double* means = (double*)((char*)slots + round_up((tiles + a.t.sequences) * (int64_t)sizeof(Part), 256));
    if (seq) {
        policy_tiles_kernel<true><<<(unsigned)tiles, kTileThreads, 0, s>>>(a, sums, slots);
        policy_sequences_kernel<<<(unsigned)cdiv(a.t.sequences, kTileThreads / 64), kTileThreads, 0, s>>>(a, slots, means);
    } else {
        policy_tiles_kernel<false><<<(unsigned)tiles, kTileThreads, 0, s>>>(a, sums, nullptr);
    }
    policy_join_kernel<<<1, kWholeThreads, 0, s>>>(a, sums, tiles, means);
}

void launch_policy_bwd(const PolicyArgs& a, const float* grad, float* dlogp, hipStream_t s) {
    policy_bwd_kernel<<<(unsigned)cdiv(a.t.n, kBackTile), kTileThreads, 0, s>>>(a, grad, dlogp);
}

size_t preference_workspace(int64_t n, int64_t pairs) {
    if (n <= kWholeTokens) return 256;
    return (size_t)(round_up((cdiv(n, kTileTokens) + 2 * pairs) * (int64_t)sizeof(Part), 256) + round_up(pairs * 8, 256));
}

void launch_preference(const PreferenceArgs& a, void* workspace, hipStream_t s) {
    if (a.t.n <= kWholeTokens) {
        preference_whole_kernel<<<1, kWholeThreads, 0, s>>>(a);
        return;
    }
    const int64_t tiles = cdiv(a.t.n, kTileTokens), pairs = a.t.sequences / 2;
    Part* slots = (Part*)workspace;
    double* each = (double*)((char*)workspace + round_up((tiles + a.t.sequences) * (int64_t)sizeof(Part), 256));
    preference_tiles_kernel<<<(unsigned)tiles, kTileThreads, 0, s>>>(a, slots);
    preference_pairs_kernel<<<(unsigned)cdiv(pairs, kTileThreads / 64), kTileThreads, 0, s>>>(a, slots, each);
    preference_join_kernel<<<1, kWholeThreads, 0, s>>>(each, pairs, a.loss);
}

void launch_preference_bwd(const Tokens& t, const float* grad, const float* coef, float* dlogp, hipStream_t s) {
    preference_bwd_kernel<<<(unsigned)cdiv(t.n, kBackTile), kTileThreads, 0, s>>>(t, grad, coef, dlogp);
}

}  // namespace lmhead
