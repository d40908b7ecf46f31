// token_losses.hip — the clipped policy loss and the preference loss on packed
// per-token log-probabilities, forward and backward.
//
// Mathematics (lmhead_train.h). Policy: L = -A rho + b KL, loss = sum_t w_s L_t,
// dlogp_t = g w_s (-A r [not clipped] + b KL'). The border of rho is compared as
// logp - old against log(1 + eps) in 64 bits: near it the fp32 ratio could fall
// on either side. Preference: s_q = sum or mean of logp - ref over a sequence, h
// = beta (s_chosen - s_rejected) - margin; dlogp_t = g coef_q.
//
// 12 to 24 bytes per token and direction and some 100 operations: small batches
// are bound by launches and by the latency of loads that wait for one another,
// large ones by memory. So few tokens are one launch of one workgroup; above,
// tiles of 1024 tokens leave 64-bit partial sums and a second launch adds them in
// order (over more sequences or tiles than a workgroup can take at once, a
// third). A tile's tokens are loaded before its sequences are looked up, and all
// its sums cross the workgroup behind one barrier. 1 M tokens: tiles 12.4 us, their
// sums 7, backward 7; the bytes alone would take 10 us of the 26. With sequence means
// 16, 8.5 and 8.5 (30 in a graph).
//
// Sequences and tiles. A tile's partial of sequence s stands at slot tile + s:
// along the packed tokens either the tile or the sequence moves on, so no two
// meeting pairs share a slot, and tiles + sequences slots hold them all.
#include "host_util.h"
#include "train_kernels.h"

namespace lmhead {

namespace {

constexpr int kTileThreads = 256, kTileEach = 4;     // tokens per thread
constexpr int64_t kTileTokens = kTileThreads * kTileEach;
// Forward and backward of the policy loss with sequence means, in a graph. Up to
// 512 tokens by 256 threads: 11.3 us, by 1024 12.9 (1024 tokens 18.8 and 17.5).
// One launch for up to 4096 tokens in up to 64 sequences: 30.2 us, as tiles 31.8 (128
// sequences 36.3 and 33.9; 4096 tokens in 8 sequences 21.1 and 23.4). The preference
// loss: 512 tokens 8.1 us by 256 threads and by 1024 (1024 tokens in 64 sequences 25.1
// and 17.5); 4096 tokens in 64 sequences 18.0 us in one launch, as tiles 21.4 (128
// sequences 26.6 and 23.3).
constexpr int kFewThreads = 256, kWholeThreads = 1024, kWholeEach = 4;
constexpr int64_t kFewTokens = 512, kWholeTokens = kWholeThreads * kWholeEach, kWholeSequences = 64;

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

// Sums over the workgroup of N values per thread, for every thread: lanes, then
// waves, each in a fixed tree. red: N doubles per wave, used once.
template <int N, int THREADS>
__device__ __forceinline__ void group_sums(double (&v)[N], double* red) {
    constexpr int WAVES = THREADS / 64;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = wave_sum(v[k]);
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) red[k * WAVES + (threadIdx.x >> 6)] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] = red[k * WAVES + (lane & (WAVES - 1))];
#pragma unroll
        for (int m = 1; m < WAVES; m <<= 1) v[k] += __shfl_xor(v[k], m);
    }
}

__device__ __forceinline__ int64_t border(const Tokens& t, int64_t s) {
    if (t.cu == nullptr) return s <= 0 ? 0 : t.n;
    const int64_t v = t.cu[s];
    return v < 0 ? 0 : v < t.n ? v : t.n;
}

// The last sequences whose first tokens are at or before i and j >= i (-1: none),
// searched by a wave: 64 borders at once, the first look for both, so that two
// looks find any of 4096.
struct Span {
    int64_t first, last;
};
__device__ __forceinline__ void narrow(int64_t& lo, int64_t& hi, int64_t step, int c) {
    if (c == 0) {
        hi = lo;
        return;
    }
    const int64_t end = lo + c * step;
    lo = lo + (c - 1) * step + 1;
    hi = end < hi ? end : hi;
}
__device__ __forceinline__ Span sequences_at(const Tokens& t, int64_t i, int64_t j) {
    if (t.cu == nullptr) return Span{0, 0};
    const int lane = threadIdx.x & 63;
    int64_t lo = 0, hi = t.sequences + 1, lo2 = 0, hi2 = hi;   // the number of borders <= i, <= j
    const int64_t step0 = (hi + 63) >> 6, at0 = lane * step0;
    const int64_t b0 = at0 < hi ? border(t, at0) : t.n + 1;
    narrow(lo, hi, step0, __popcll(__ballot(b0 <= i)));
    narrow(lo2, hi2, step0, __popcll(__ballot(b0 <= j)));
    while (lo < hi || lo2 < hi2) {
        const int64_t step = (hi - lo + 63) >> 6, at = lo + lane * step;
        const int64_t step2 = (hi2 - lo2 + 63) >> 6, at2 = lo2 + lane * step2;
        const int64_t b = at < hi ? border(t, at) : t.n + 1, b2 = at2 < hi2 ? border(t, at2) : t.n + 1;
        if (lo < hi) narrow(lo, hi, step, __popcll(__ballot(b <= i)));
        if (lo2 < hi2) narrow(lo2, hi2, step2, __popcll(__ballot(b2 <= j)));
    }
    return Span{lo - 1, lo2 - 1};
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

// k = exp(-x) - 1 + x and m = exp(-x) - 1, from power = exp(-x). For |x| <= 1/2, where
// the differences would cancel, k is its series x^2 sum_i (-x)^i / (i + 2)!, whose
// first term left out is below 2^-24 of the sum, and m = k - x.
struct K3 {
    float k, m;
};
__device__ __forceinline__ K3 k3_of(float x, float power) {
    const float y = -x;
    float s = 1.0f / 40320.0f;
    s = __builtin_fmaf(y, s, 1.0f / 5040.0f);
    s = __builtin_fmaf(y, s, 1.0f / 720.0f);
    s = __builtin_fmaf(y, s, 1.0f / 120.0f);
    s = __builtin_fmaf(y, s, 1.0f / 24.0f);
    s = __builtin_fmaf(y, s, 1.0f / 6.0f);
    s = __builtin_fmaf(y, s, 0.5f);
    const bool near = fabsf(x) <= 0.5f;
    K3 o;
    o.k = near ? x * x * s : power - 1.0f + x;
    o.m = near ? o.k - x : power - 1.0f;
    return o;
}

__device__ __forceinline__ Term policy_term(const PolicyArgs& a, float logp, float old, float ref, float adv) {
    // The terms are fp32, as the outputs; their sums are of 64 bits. Rounding the gap
    // to fp32 moves r by |d| 2^-24 of it, and the estimates outside their series are
    // off by a few 2^-24 of their largest term.
    Term o;
    // without old log-probs r is 1, of an infinite logp too; NaN stays
    const double gap = a.old_logp != nullptr || logp != logp ? (double)logp - (double)old : 0.0;
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
    o.back = k3_of(d, 1.0f / o.ratio).k;
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
            const K3 e = k3_of(x, expf(-x));
            o.kl = e.k;
            dk = -e.m;
        }
        if (a.kl_weight != 0.0f) {   // without: a statistic alone, and an infinite one spoils nothing
            o.loss = __builtin_fmaf(a.kl_weight, o.kl, o.loss);
            o.slope = __builtin_fmaf(a.kl_weight, dk, o.slope);
        }
    }
    return o;
}

// ------------------------------------------------------------------- policy

enum { kLoss, kCount, kKl, kClipped, kRatio, kBack };   // a tile's six sums
struct Part {
    double sum, count;
};

struct Tile {
    int64_t t0, t1;
    Span at;   // sequences at its first and last token
};
template <int TOKENS>
__device__ __forceinline__ Tile tile_of(const Tokens& t) {
    Tile o;
    o.t0 = (int64_t)blockIdx.x * TOKENS;
    o.t1 = o.t0 + TOKENS < t.n ? o.t0 + TOKENS : t.n;
    return o;
}
__device__ __forceinline__ void look_up(Tile& o, const Tokens& t) {
    o.at = sequences_at(t, o.t0, o.t1 > o.t0 ? o.t1 - 1 : o.t0);
}

// Nothing differs between the sequences: then the tile's span is that of the
// tokens which lie in one, and none is looked up (1 M tokens in 256 sequences:
// backward 6.4 us, with the search 8.2; tiles of the forward 12.4 and 13.0).
__device__ __forceinline__ bool all_alike(const PolicyArgs& a) { return !a.per_sequence && a.reduction != 2; }

__device__ __forceinline__ void look_up(Tile& o, const PolicyArgs& a) {
    if (all_alike(a)) o.at = Span{border(a.t, 0), border(a.t, a.t.sequences)};
    else look_up(o, a.t);
}

// A thread's tokens t0 + thread, + THREADS, ...: loaded at once; then their terms.
template <int THREADS, int EACH>
struct PolicyTokens {
    float logp[EACH], old[EACH], ref[EACH], adv[EACH];
    int32_t target[EACH];

    __device__ __forceinline__ void load(const PolicyArgs& a, const Tile& tile) {
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const int64_t i = tile.t0 + k * THREADS + threadIdx.x;
            logp[k] = old[k] = ref[k] = adv[k] = 0.0f;
            target[k] = -1;
            if (i >= tile.t1) continue;
            logp[k] = a.logp[i];
            if (a.old_logp != nullptr) old[k] = a.old_logp[i];
            if (a.ref_logp != nullptr) ref[k] = a.ref_logp[i];
            if (!a.per_sequence) adv[k] = a.advantage[i];
            target[k] = a.t.targets != nullptr ? a.t.targets[i] : 0;
        }
    }
    // the token's sequence where it counts, else -1; any sequence where all are one
    __device__ __forceinline__ int64_t place(const PolicyArgs& a, const Tile& tile, int k) const {
        const int64_t i = tile.t0 + k * THREADS + threadIdx.x;
        if (i >= tile.t1 || target[k] < 0) return -1;
        if (all_alike(a)) return i >= tile.at.first && i < tile.at.last ? 0 : -1;
        const int64_t q = sequence_between(a.t, tile.at.first, tile.at.last, i);
        return q < a.t.sequences ? q : -1;
    }
    __device__ __forceinline__ Term term(const PolicyArgs& a, int k, int64_t q) const {
        return policy_term(a, logp[k], old[k], ref[k], a.per_sequence ? a.advantage[q >= 0 ? q : 0] : adv[k]);
    }
};

// A tile's terms, summed per thread; per token kept in LDS where sequences are
// summed apart.
template <int THREADS, int EACH, bool SEQ>
__device__ __forceinline__ void policy_tile(const PolicyArgs& a, Tile& tile, double (&s)[6], float* kept, uint8_t* counts) {
    PolicyTokens<THREADS, EACH> tokens;
    tokens.load(a, tile);
    look_up(tile, a);
#pragma unroll
    for (int k = 0; k < 6; ++k) s[k] = 0.0;
    int count = 0, clipped = 0;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        if (tile.t0 + k * THREADS >= tile.t1) break;   // for all threads
        const int64_t q = tokens.place(a, tile, k);
        const Term o = tokens.term(a, k, q);
        if (q >= 0) {   // whatever stands in the other places takes no part
            if (!SEQ) s[kLoss] += (double)o.loss;
            ++count;
            clipped += o.clipped;
            s[kKl] += (double)o.kl;
            s[kRatio] += (double)o.ratio;
            s[kBack] += (double)o.back;
        }
        if (SEQ) {
            kept[k * THREADS + threadIdx.x] = o.loss;
            counts[k * THREADS + threadIdx.x] = q >= 0;
        }
    }
    s[kCount] = count;
    s[kClipped] = clipped;
}

// One sequence's part of a tile, from LDS, by one wave.
template <typename T>
__device__ __forceinline__ Part part_of(const Tokens& t, const Tile& tile, int64_t q, const T* kept,
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

// The same over the tiles that a sequence touches, from their slots, by `lanes`
// (a power of two) neighbours of a wave.
__device__ __forceinline__ Part part_of(const Tokens& t, int64_t q, const Part* slots, int lanes) {
    const int64_t from = border(t, q), to = border(t, q + 1);
    Part p = {0.0, 0.0};
    if (from < to)
        for (int64_t tile = from / kTileTokens + (threadIdx.x & (lanes - 1)); tile <= (to - 1) / kTileTokens; tile += lanes) {
            const Part o = slots[tile + q];
            p.sum += o.sum;
            p.count += o.count;
        }
    for (int m = 1; m < lanes; m <<= 1) {
        p.sum += __shfl_xor(p.sum, m);
        p.count += __shfl_xor(p.count, m);
    }
    return p;
}

__device__ __forceinline__ double share(int64_t given, double counted) {
    const double d = given >= 0 ? (double)given : counted;
    return d > 0.0 ? 1.0 / d : 0.0;
}

// A sequence's weight in the sequence mean; returns its mean times its share.
__device__ __forceinline__ double weigh(const PolicyArgs& a, int64_t q, const Part& p, bool writes) {
    const double w = p.count > 0.0 ? share(a.num_valid, (double)a.t.sequences) / p.count : 0.0;
    if (writes) a.weights[q] = (float)w;
    return w > 0.0 ? w * p.sum : 0.0;
}

// What is left once the totals are known: called by every thread of the last workgroup.
__device__ __forceinline__ void policy_end(const PolicyArgs& a, const double (&s)[6], int threads) {
    const bool seq = a.reduction == 2;
    const double w = a.reduction == 0 ? share(a.num_valid, s[kCount]) : 1.0;
    if (!seq)   // one weight for all
        for (int64_t q = threadIdx.x; q < a.t.sequences; q += threads) a.weights[q] = (float)w;
    if (threadIdx.x != 0) return;
    a.loss[0] = (float)(seq ? s[kLoss] : w > 0.0 ? w * s[kLoss] : 0.0);
    if (a.stats == nullptr) return;
    const double each = s[kCount] > 0.0 ? 1.0 / s[kCount] : 0.0;
    a.stats[0] = (float)(s[kKl] * each);
    a.stats[1] = (float)(s[kClipped] * each);
    a.stats[2] = (float)(s[kRatio] * each);
    a.stats[3] = (float)(s[kBack] * each);
}

template <int THREADS, bool SEQ>
__global__ __launch_bounds__(THREADS) void policy_whole_kernel(PolicyArgs a) {
    __shared__ double red[6 * THREADS / 64];
    __shared__ float kept[SEQ ? THREADS * kWholeEach : 1];
    __shared__ uint8_t counts[SEQ ? THREADS * kWholeEach : 1];
    Tile tile = tile_of<THREADS * kWholeEach>(a.t);
    double s[6];
    policy_tile<THREADS, kWholeEach, SEQ>(a, tile, s, kept, counts);
    if (SEQ) {   // every sequence by a wave; a lane's share of the loss is its mean
        __syncthreads();
        double means = 0.0;
        for (int64_t q = threadIdx.x >> 6; q < a.t.sequences; q += THREADS / 64)
            means += weigh(a, q, part_of(a.t, tile, q, kept, counts), (threadIdx.x & 63) == 0);
        s[kLoss] = (threadIdx.x & 63) == 0 ? means : 0.0;
    }
    group_sums<6, THREADS>(s, red);
    policy_end(a, s, THREADS);
}

template <bool SEQ>
__global__ __launch_bounds__(kTileThreads) void policy_tiles_kernel(PolicyArgs a, double* tiles, Part* slots) {
    __shared__ double red[6 * kTileThreads / 64];
    __shared__ float kept[SEQ ? kTileTokens : 1];
    __shared__ uint8_t counts[SEQ ? kTileTokens : 1];
    Tile tile = tile_of<kTileTokens>(a.t);
    double s[6];
    policy_tile<kTileThreads, kTileEach, SEQ>(a, tile, s, kept, counts);
    group_sums<6, kTileThreads>(s, red);   // its barrier: kept and counts are written
    if (threadIdx.x == 0)
#pragma unroll
        for (int k = 0; k < 6; ++k) tiles[k * (int64_t)gridDim.x + blockIdx.x] = s[k];
    if (!SEQ) return;
    for (int64_t q = (tile.at.first > 0 ? tile.at.first : 0) + (threadIdx.x >> 6); q <= tile.at.last && q < a.t.sequences;
         q += kTileThreads / 64) {
        const Part p = part_of(a.t, tile, q, kept, counts);
        if ((threadIdx.x & 63) == 0) slots[blockIdx.x + q] = p;
    }
}

__global__ __launch_bounds__(kTileThreads) void policy_sequences_kernel(PolicyArgs a, const Part* slots, double* means) {
    const int64_t q = (int64_t)blockIdx.x * (kTileThreads / 64) + (threadIdx.x >> 6);
    if (q >= a.t.sequences) return;
    const bool writes = (threadIdx.x & 63) == 0;
    const double m = weigh(a, q, part_of(a.t, q, slots, 64), writes);
    if (writes) means[q] = m;
}

// lanes: of the sequences' means, where their parts are added here (a thread each, or more)
__global__ __launch_bounds__(kWholeThreads) void policy_join_kernel(PolicyArgs a, const double* tiles, int64_t count,
                                                                    const double* means, const Part* slots, int lanes) {
    __shared__ double red[6 * kWholeThreads / 64];
    double s[6] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
    for (int64_t i = threadIdx.x; i < count; i += kWholeThreads)
#pragma unroll
        for (int k = 0; k < 6; ++k) s[k] += tiles[k * count + i];
    if (lanes > 0) {
        const int64_t q = threadIdx.x / (unsigned)lanes;
        const bool in = q < a.t.sequences, writes = in && (threadIdx.x & (lanes - 1)) == 0;
        const double m = weigh(a, in ? q : 0, part_of(a.t, in ? q : 0, slots, lanes), writes);
        s[kLoss] = writes ? m : 0.0;
    } else if (a.reduction == 2) {
        s[kLoss] = 0.0;
#pragma unroll 4
        for (int64_t q = threadIdx.x; q < a.t.sequences; q += kWholeThreads) s[kLoss] += means[q];
    }
    group_sums<6, kWholeThreads>(s, red);
    policy_end(a, s, kWholeThreads);
}

__global__ __launch_bounds__(kTileThreads) void policy_bwd_kernel(PolicyArgs a, const float* grad, float* dlogp) {
    Tile tile = tile_of<kTileTokens>(a.t);
    PolicyTokens<kTileThreads, kTileEach> tokens;
    tokens.load(a, tile);
    const float g = grad[0];
    look_up(tile, a);
#pragma unroll
    for (int k = 0; k < kTileEach; ++k) {
        const int64_t i = tile.t0 + k * kTileThreads + threadIdx.x;
        if (i >= tile.t1) continue;
        const int64_t q = tokens.place(a, tile, k);
        const Term o = tokens.term(a, k, q);
        const float w = q >= 0 ? a.weights[q] : 0.0f;   // 0 (a given count of 0) of an infinite slope too
        dlogp[i] = w != 0.0f ? g * (w * o.slope) : 0.0f;
    }
}

// --------------------------------------------------------------- preference
//
// The same tiles and slots; what a thread keeps is a difference, in 64 bits as the
// sums: in fp32 what is left of them between two answers could be its roundings. 512
// pairs over 1 M tokens: tiles 9 us (12 MB; 7.6 with fp32 differences), pairs 6.0, backward 7
// (8 MB); 4 pairs over 2500 tokens in one launch 5.7, backward 4.5. Latency decides all of them.

template <int THREADS, int EACH>
__device__ __forceinline__ void preference_tile(const PreferenceArgs& a, const Tile& tile, double* kept, uint8_t* counts) {
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const int64_t i = tile.t0 + k * THREADS + threadIdx.x;
        double gain = 0.0;
        bool valid = false;
        if (i < tile.t1) {
            gain = (double)a.logp[i] - (a.ref_logp != nullptr ? (double)a.ref_logp[i] : 0.0);
            valid = a.t.targets == nullptr || a.t.targets[i] >= 0;
        }
        kept[k * THREADS + threadIdx.x] = gain;
        counts[k * THREADS + threadIdx.x] = valid;
    }
}

// One pair from its sequences' sums: writes the rewards and coefficients, returns its share of the loss.
__device__ __forceinline__ double pair_loss(const PreferenceArgs& a, int64_t pair, Part c, Part r, bool writes) {
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
    if (writes) {
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

template <int THREADS>
__global__ __launch_bounds__(THREADS) void preference_whole_kernel(PreferenceArgs a) {
    __shared__ double red[THREADS / 64];
    __shared__ double kept[THREADS * kWholeEach];
    __shared__ uint8_t counts[THREADS * kWholeEach];
    const Tile tile = tile_of<THREADS * kWholeEach>(a.t);
    preference_tile<THREADS, kWholeEach>(a, tile, kept, counts);
    __syncthreads();
    const int64_t pairs = a.t.sequences / 2;
    double loss[1] = {0.0};
    for (int64_t j = threadIdx.x >> 6; j < pairs; j += THREADS / 64)
        loss[0] += pair_loss(a, j, part_of(a.t, tile, j, kept, counts), part_of(a.t, tile, pairs + j, kept, counts),
                             (threadIdx.x & 63) == 0);
    if ((threadIdx.x & 63) != 0) loss[0] = 0.0;
    group_sums<1, THREADS>(loss, red);
    if (threadIdx.x == 0) a.loss[0] = (float)loss[0];
}

__global__ __launch_bounds__(kTileThreads) void preference_tiles_kernel(PreferenceArgs a, Part* slots) {
    __shared__ double kept[kTileTokens];
    __shared__ uint8_t counts[kTileTokens];
    Tile tile = tile_of<kTileTokens>(a.t);
    preference_tile<kTileThreads, kTileEach>(a, tile, kept, counts);
    look_up(tile, a.t);
    __syncthreads();
    for (int64_t q = (tile.at.first > 0 ? tile.at.first : 0) + (threadIdx.x >> 6); q <= tile.at.last && q < a.t.sequences;
         q += kTileThreads / 64) {
        const Part p = part_of(a.t, tile, q, kept, counts);
        if ((threadIdx.x & 63) == 0) slots[blockIdx.x + q] = p;
    }
}

__global__ __launch_bounds__(kTileThreads) void preference_pairs_kernel(PreferenceArgs a, const Part* slots, double* each) {
    const int64_t j = (int64_t)blockIdx.x * (kTileThreads / 64) + (threadIdx.x >> 6), pairs = a.t.sequences / 2;
    if (j >= pairs) return;
    const bool writes = (threadIdx.x & 63) == 0;
    const double l = pair_loss(a, j, part_of(a.t, j, slots, 64), part_of(a.t, pairs + j, slots, 64), writes);
    if (writes) each[j] = l;
}

// Both, where a workgroup has `lanes` threads for each pair.
__global__ __launch_bounds__(kWholeThreads) void preference_end_kernel(PreferenceArgs a, const Part* slots, int lanes) {
    __shared__ double red[kWholeThreads / 64];
    const int64_t j = threadIdx.x / (unsigned)lanes, pairs = a.t.sequences / 2;
    const bool in = j < pairs, writes = in && (threadIdx.x & (lanes - 1)) == 0;
    const int64_t pair = in ? j : 0;
    double loss[1];
    loss[0] = pair_loss(a, pair, part_of(a.t, pair, slots, lanes), part_of(a.t, pairs + pair, slots, lanes), writes);
    if (!writes) loss[0] = 0.0;
    group_sums<1, kWholeThreads>(loss, red);
    if (threadIdx.x == 0) a.loss[0] = (float)loss[0];
}

__global__ __launch_bounds__(kWholeThreads) void preference_join_kernel(const double* each, int64_t count, float* loss) {
    __shared__ double red[kWholeThreads / 64];
    double s[1] = {0.0};
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < count; i += kWholeThreads) s[0] += each[i];
    group_sums<1, kWholeThreads>(s, red);
    if (threadIdx.x == 0) loss[0] = (float)s[0];
}

__global__ __launch_bounds__(kTileThreads) void preference_bwd_kernel(Tokens t, const float* grad, const float* coef,
                                                                      float* dlogp) {
    Tile tile = tile_of<kTileTokens>(t);
    int32_t target[kTileEach];
#pragma unroll
    for (int k = 0; k < kTileEach; ++k) {
        const int64_t i = tile.t0 + k * kTileThreads + threadIdx.x;
        target[k] = t.targets != nullptr && i < tile.t1 ? t.targets[i] : 0;
    }
    const float g = grad[0];
    look_up(tile, t);
#pragma unroll
    for (int k = 0; k < kTileEach; ++k) {
        const int64_t i = tile.t0 + k * kTileThreads + threadIdx.x;
        if (i >= tile.t1) continue;
        const int64_t q = sequence_between(t, tile.at.first, tile.at.last, i);
        dlogp[i] = q >= 0 && q < t.sequences && target[k] >= 0 ? g * coef[q] : 0.0f;
    }
}

}  // namespace

// Threads that one workgroup has for each of `count` sequences or pairs: a power
// of two up to 64, or 0 for more than it has threads or for parts that would
// keep them long (many more tiles than threads).
static int lanes_for(int64_t count, int64_t tiles) {
    if (count > kWholeThreads || tiles > 8 * kWholeThreads) return 0;
    int lanes = 64;
    while (count * lanes > kWholeThreads) lanes >>= 1;
    return lanes;
}

static int64_t tiles_of(int64_t n) { return n > 0 ? cdiv(n, kTileTokens) : 1; }
static bool one_launch(int64_t n, int64_t sequences) { return n <= kWholeTokens && sequences <= kWholeSequences; }

size_t policy_workspace(int64_t n, int64_t sequences, int reduction) {
    if (one_launch(n, sequences)) return 256;
    const int64_t tiles = tiles_of(n);
    int64_t bytes = round_up(tiles * 6 * 8, 256);
    if (reduction == 2)
        bytes += round_up((tiles + sequences) * (int64_t)sizeof(Part), 256) + round_up(sequences * 8, 256);
    return (size_t)bytes;
}

void launch_policy(const PolicyArgs& a, void* workspace, hipStream_t s) {
    const bool seq = a.reduction == 2;
    if (one_launch(a.t.n, a.t.sequences)) {
        if (a.t.n <= kFewTokens) {
            if (seq) policy_whole_kernel<kFewThreads, true><<<1, kFewThreads, 0, s>>>(a);
            else policy_whole_kernel<kFewThreads, false><<<1, kFewThreads, 0, s>>>(a);
        } else {
            if (seq) policy_whole_kernel<kWholeThreads, true><<<1, kWholeThreads, 0, s>>>(a);
            else policy_whole_kernel<kWholeThreads, false><<<1, kWholeThreads, 0, s>>>(a);
        }
        return;
    }
    const int64_t tiles = tiles_of(a.t.n);
    char* w = (char*)workspace;
    double* sums = (double*)w;
    Part* slots = (Part*)(w + round_up(tiles * 6 * 8, 256));
    double* means = (double*)((char*)slots + round_up((tiles + a.t.sequences) * (int64_t)sizeof(Part), 256));
    const int lanes = seq ? lanes_for(a.t.sequences, tiles) : 0;
    if (seq) policy_tiles_kernel<true><<<(unsigned)tiles, kTileThreads, 0, s>>>(a, sums, slots);
    else policy_tiles_kernel<false><<<(unsigned)tiles, kTileThreads, 0, s>>>(a, sums, nullptr);
    if (seq && lanes == 0)
        policy_sequences_kernel<<<(unsigned)cdiv(a.t.sequences, kTileThreads / 64), kTileThreads, 0, s>>>(a, slots, means);
    policy_join_kernel<<<1, kWholeThreads, 0, s>>>(a, sums, tiles, means, slots, lanes);
}

void launch_policy_bwd(const PolicyArgs& a, const float* grad, float* dlogp, hipStream_t s) {
    policy_bwd_kernel<<<(unsigned)cdiv(a.t.n, kTileTokens), kTileThreads, 0, s>>>(a, grad, dlogp);
}

size_t preference_workspace(int64_t n, int64_t pairs) {
    if (one_launch(n, 2 * pairs)) return 256;
    return (size_t)(round_up((tiles_of(n) + 2 * pairs) * (int64_t)sizeof(Part), 256) + round_up(pairs * 8, 256));
}

void launch_preference(const PreferenceArgs& a, void* workspace, hipStream_t s) {
    if (one_launch(a.t.n, a.t.sequences)) {
        if (a.t.n <= kFewTokens) preference_whole_kernel<kFewThreads><<<1, kFewThreads, 0, s>>>(a);
        else preference_whole_kernel<kWholeThreads><<<1, kWholeThreads, 0, s>>>(a);
        return;
    }
    const int64_t tiles = tiles_of(a.t.n), pairs = a.t.sequences / 2;
    Part* slots = (Part*)workspace;
    double* each = (double*)((char*)workspace + round_up((tiles + a.t.sequences) * (int64_t)sizeof(Part), 256));
    preference_tiles_kernel<<<(unsigned)tiles, kTileThreads, 0, s>>>(a, slots);
    const int lanes = lanes_for(pairs, tiles);
    if (lanes > 0) {
        preference_end_kernel<<<1, kWholeThreads, 0, s>>>(a, slots, lanes);
        return;
    }
    preference_pairs_kernel<<<(unsigned)cdiv(pairs, kTileThreads / 64), kTileThreads, 0, s>>>(a, slots, each);
    preference_join_kernel<<<1, kWholeThreads, 0, s>>>(each, pairs, a.loss);
}

void launch_preference_bwd(const Tokens& t, const float* grad, const float* coef, float* dlogp, hipStream_t s) {
    preference_bwd_kernel<<<(unsigned)cdiv(t.n, kTileTokens), kTileThreads, 0, s>>>(t, grad, coef, dlogp);
}

}  // namespace lmhead
