// adamw.hip — one AdamW step over many tensors, states in fp32 or in 8 bits.
//
// Mathematics (lmhead_train.h): m' = b1 m + (1 - b1) g, v' = b2 v + (1 - b2) g^2,
// p' = p (1 - lr wd) - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps), all
// in fp32. 8-bit states are e4m3 over blocks of 128: of m, and of sqrt(v), whose
// range is the square root of v's (e4m3 spans 2^17.8 of a block's largest value).
// They round to nearest, or at random (unbiased) where a seed is given: nearest
// rounding swallows changes below half a code's step, which with beta2 = 0.99
// left sqrt(v) 1.15 times too large in the median after 300 steps.
//
// Bound by memory: 10 to 28 bytes per element and about 40 operations. Each
// element is read and written once; eight consecutive ones per lane, so that 16
// lanes hold a block of 128 and its maximum is four shuffles. Tensors share a
// launch; a workgroup finds its tensor by its chunk's number, in a table of up to
// 48 that travels as a kernel argument, or in the caller's table on the device.
// bf16 parameters: 525 M with fp32 gradients and states 2303 us (5.5 TB/s), 622 M
// with bf16 gradients and 8-bit states 1097 us (5.7 TB/s; a large copy reaches
// 4.7), at random rounding 1310 (a hash per element); 129 tensors of 4096 in one
// kernel of 4.8 us, by kernel arguments in three of 5.3, 5.3 and 4.7.
#include "host_util.h"
#include "train_kernels.h"
#include "vec8.h"

namespace lmhead {

namespace {

// lane's eight values at element e; zeros past the end. STREAM: past the caches
template <bool F32, bool STREAM>
__device__ __forceinline__ V8 fetch(const void* p, int64_t e, int64_t numel, bool wide) {
    if (wide && e + 8 <= numel) {
        Raw8<F32> r;
#pragma unroll
        for (int k = 0; k < (F32 ? 2 : 1); ++k) {
            const Words4 w = load_words<STREAM>(p, (F32 ? 2 : 1) * (e >> 3) + k);
            r.w[k] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        return to8<F32>(r);
    }
    V8 f = zeros8();
#pragma unroll
    for (int c = 0; c < 8; ++c)
        if (e + c < numel)
            f.v[c] = F32 ? reinterpret_cast<const float*>(p)[e + c]
                         : __builtin_bit_cast(float, (uint32_t)reinterpret_cast<const bf16_bits*>(p)[e + c] << 16);
    return f;
}
template <bool F32, bool STREAM>
__device__ __forceinline__ void put(void* p, int64_t e, int64_t numel, bool wide, const V8& f) {
    if (wide && e + 8 <= numel) {
        store8<F32, STREAM>(p, e >> 3, f);
        return;
    }
#pragma unroll
    for (int c = 0; c < 8; ++c)
        if (e + c < numel) {
            if (F32) reinterpret_cast<float*>(p)[e + c] = f.v[c];
            else reinterpret_cast<__bf16*>(p)[e + c] = (__bf16)f.v[c];
        }
}
__device__ __forceinline__ uint2 fetch_codes(const void* p, int64_t e, int64_t numel, bool wide) {
    if (wide && e + 8 <= numel) return reinterpret_cast<const uint2*>(p)[e >> 3];
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int c = 0; c < 8; ++c)
        if (e + c < numel) w[c >> 2] |= (uint32_t)reinterpret_cast<const uint8_t*>(p)[e + c] << (8 * (c & 3));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void put_codes(void* p, int64_t e, int64_t numel, bool wide, const uint2& q) {
    if (wide && e + 8 <= numel) {
        __builtin_nontemporal_store((uint64_t)q.y << 32 | q.x, reinterpret_cast<uint64_t*>(p) + (e >> 3));
        return;
    }
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int c = 0; c < 8; ++c)
        if (e + c < numel) reinterpret_cast<uint8_t*>(p)[e + c] = (uint8_t)(w[c >> 2] >> (8 * (c & 3)));
}

// a x + b y with every product rounded
__device__ __forceinline__ float each_rounded(float a, float x, float b, float y) {
#pragma clang fp contract(off)
    const float p = a * x, q = b * y;
    return p + q;
}

// The root instructions take a value below 2^-126 for 0, which with a small eps
// makes a vanishing gradient's step large, and below 2^-100 the remainder of a
// rounded root loses bits: so small values a power of two larger, and back.
template <bool ROUNDED>
__device__ __forceinline__ float root_of(float x) {
    const bool small = x < 0x1p-64f;
    const float z = small ? x * 0x1p64f : x;
    float r;
    if (ROUNDED) {
        // to nearest (but for ties of the last step, within 2^-20 of one): one Newton
        // step with its remainder from the instruction's reciprocal root
        const float y = __builtin_amdgcn_rsqf(z), s = z * y;
        r = __builtin_fmaf(__builtin_fmaf(-s, s, z), 0.5f * y, s);
        r = z > 0.0f && z <= 3.402823466e38f ? r : z;   // zero, infinity and NaN are their own
    } else {
        r = __builtin_amdgcn_sqrtf(z);
    }
    return small ? r * 0x1p-32f : r;
}

// Scale of a block of 8-bit states: its largest magnitude by 448.
__device__ __forceinline__ float state_scale(float amax) {
    return amax > 0.0f ? fmaxf(amax * (1.0f / kE4m3Max), 0x1p-126f) : 1.0f;
}

// over the 16 lanes that hold a block of 128 (NaN left out)
__device__ __forceinline__ float max16(float v) {
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
    return v;
}

// Two rounds of multiplying and folding by odd constants (the golden ratio's and
// e's fractions): every bit of x moves about half of the result's.
__device__ __forceinline__ uint32_t scramble(uint32_t x) {
    x ^= x >> 16;
    x *= 0x9e3779b9u;
    x ^= x >> 15;
    x *= 0xb7e15163u;
    return x ^ x >> 16;
}

// |y| plus a random part of its code's step (20 bits of the fp32 value), cut to
// the code below. Below 2^-6 the codes' step is that of 2^-6 .. 2^-5, so the
// value is moved there and back. NaN stays: bits added to a fraction of ones would
// carry over into its sign and leave a zero.
__device__ __forceinline__ float cut_at_random(float y, uint32_t random20) {
    const float mag = fabsf(y), base = mag < 0x1p-6f ? 0x1p-6f : 0.0f;
    const uint32_t bits = (__builtin_bit_cast(uint32_t, mag + base) + random20) & 0xfff00000u;
    return y == y ? __builtin_copysignf(__builtin_bit_cast(float, bits) - base, y) : y;
}

// e4m3 of eight quotients by the block's scale, the quotients as a division
// rounds them. ROOT: a value above zero gets at
// least the least code. RANDOM: noise of the eight, in bits 4 .. 19.
template <bool ROOT, bool RANDOM>
__device__ __forceinline__ uint2 codes(const V8& f, float scale, const uint32_t* noise) {
    // the quotient of x inv and one step with its remainder: as the division
    // rounds, but where it lies within 2^-22 of a step from the middle of two values
    const float inv = 1.0f / scale;
    V8 y;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const float q = f.v[c] * inv;
        y.v[c] = __builtin_fmaf(__builtin_fmaf(-q, scale, f.v[c]), inv, q);
        if (ROOT && f.v[c] > 0.0f) y.v[c] = y.v[c] < 0x1p-9f ? 0x1p-9f : y.v[c];
        if (RANDOM) y.v[c] = cut_at_random(y.v[c], ROOT ? noise[c] >> 16 << 4 : (noise[c] & 0xffffu) << 4);
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(y.v[4 * i], y.v[4 * i + 1], 0, false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(y.v[4 * i + 2], y.v[4 * i + 3], v, true);
        w[i] = (uint32_t)v;
    }
    return make_uint2(w[0], w[1]);
}

struct Step {
    float beta1, rest1, beta2, rest2, eps, keep, step_size, root_scale, grad_scale;
    uint32_t mix;   // of the random rounding
};

template <bool P32, bool G32, bool S8, bool RANDOM>
__device__ __forceinline__ void update(const AdamWTensor& t, const Step& k, int64_t chunk) {
    // 8-bit states leave few bytes per element: two trips in flight, past the
    // caches (622 M bf16 parameters, before the rounded root: 1050 us; one trip
    // 1139, two through the caches 1093). fp32 states: one trip through them (525 M: 2296 us; two 2323,
    // past the caches 2390).
    constexpr int kTrips = (S8 ? kAdamWChunk8 : kAdamWChunk) / 2048;
    const bool wide = (t.kind & kAdamWWide) != 0;
    const int64_t e0 = chunk * (2048 * kTrips) + threadIdx.x * 8;
    V8 p[kTrips], g[kTrips], m[kTrips], v[kTrips];
    uint2 mq[S8 ? kTrips : 1], vq[S8 ? kTrips : 1];
    float ms[S8 ? kTrips : 1], vs[S8 ? kTrips : 1];
    // every load before the first store
#pragma unroll
    for (int j = 0; j < kTrips; ++j) {
        const int64_t e = e0 + j * 2048;
        p[j] = fetch<P32, S8>(t.param, e, t.numel, wide);
        g[j] = fetch<G32, S8>(t.grad, e, t.numel, wide);
        if (S8) {
            mq[S8 ? j : 0] = fetch_codes(t.m, e, t.numel, wide);
            vq[S8 ? j : 0] = fetch_codes(t.v, e, t.numel, wide);
            ms[S8 ? j : 0] = e < t.numel ? t.m_scale[e >> 7] : 0.0f;
            vs[S8 ? j : 0] = e < t.numel ? t.v_scale[e >> 7] : 0.0f;
        } else {
            m[j] = fetch<true, false>(t.m, e, t.numel, wide);
            v[j] = fetch<true, false>(t.v, e, t.numel, wide);
        }
    }
#pragma unroll
    for (int j = 0; j < kTrips; ++j) {
        const int64_t e = e0 + j * 2048;
        if (S8) {
            m[j] = e4m3_to8(mq[S8 ? j : 0]);
            v[j] = e4m3_to8(vq[S8 ? j : 0]);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                m[j].v[c] *= ms[S8 ? j : 0];
                v[j].v[c] *= vs[S8 ? j : 0];
                v[j].v[c] *= v[j].v[c];
            }
        }
        V8 root;
        float m_max = 0.0f, v_max = 0.0f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float gc = g[j].v[c] * k.grad_scale;
            // What becomes 8 bits is rounded operation by operation, as elementwise
            // programs do: a last bit that differs between two ways of computing
            // m' is a code's step where it lies at a border, and the next step's
            // scale where that code is its block's largest.
            const float mc = S8 ? each_rounded(k.beta1, m[j].v[c], k.rest1, gc)
                                : __builtin_fmaf(k.rest1, gc, k.beta1 * m[j].v[c]);
            const float vc = S8 ? each_rounded(k.beta2, v[j].v[c], k.rest2, gc * gc)
                                : __builtin_fmaf(k.rest2 * gc, gc, k.beta2 * v[j].v[c]);
            // the instructions' own root and reciprocal, each within 2^-23: the
            // library's correctly rounded ones would double the arithmetic. A root
            // that becomes 8 bits is rounded, 41 of the 1097 us of 622 M parameters; the
            // library's would take 158.
            const float rc = root_of<S8>(vc);
            const float step = mc * __builtin_amdgcn_rcpf(__builtin_fmaf(rc, k.root_scale, k.eps));
            p[j].v[c] = __builtin_fmaf(-k.step_size, step, p[j].v[c] * k.keep);
            m[j].v[c] = mc;
            v[j].v[c] = vc;
            root.v[c] = rc;
            if (S8) {
                m_max = fmaxf(m_max, fabsf(mc));
                v_max = fmaxf(v_max, rc);
            }
        }
        put<P32, S8>(t.param, e, t.numel, wide, p[j]);
        if (t.copy != nullptr) put<false, S8>(t.copy, e, t.numel, wide, p[j]);
        if (S8) {
            uint32_t noise[RANDOM ? 8 : 1];
            if (RANDOM)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    noise[RANDOM ? c : 0] = scramble((uint32_t)(e + c) ^ k.mix ^ (uint32_t)(e >> 32) * 0x9e3779b9u);
            const float sm = state_scale(max16(m_max)), sv = state_scale(max16(v_max));
            put_codes(t.m, e, t.numel, wide, codes<false, RANDOM>(m[j], sm, noise));
            put_codes(t.v, e, t.numel, wide, codes<true, RANDOM>(root, sv, noise));
            if ((threadIdx.x & 15) == 0 && e < t.numel) {
                t.m_scale[e >> 7] = sm;
                t.v_scale[e >> 7] = sv;
            }
        } else {
            put<true, false>(t.m, e, t.numel, wide, m[j]);
            put<true, false>(t.v, e, t.numel, wide, v[j]);
        }
    }
}

// The step's numbers, from the device where they stand there.
__device__ __forceinline__ Step step_of(const AdamWScalars& k, float* now) {
    Step s = {k.beta1, k.rest1, k.beta2, k.rest2, k.eps, k.keep, k.step_size, k.root_scale, 1.0f, 0u};
    if (k.grad_scale != nullptr) s.grad_scale = k.grad_scale[0];
    if (k.step != nullptr || k.device_lr != nullptr) {
        if (threadIdx.x == 0) {
            int64_t t = k.step != nullptr ? (int64_t)k.step[0] : k.host_step;
            if (t < 1) t = 1;
            const double lr = k.device_lr != nullptr ? (double)k.device_lr[0] : k.host_lr;
            now[0] = (float)(1.0 - lr * k.weight_decay);
            now[1] = (float)(lr / -expm1((double)t * k.log_beta1));
            now[2] = (float)(1.0 / sqrt(-expm1((double)t * k.log_beta2)));
        }
        __syncthreads();
        s.keep = now[0];
        s.step_size = now[1];
        s.root_scale = now[2];
    }
    return s;
}

__device__ __forceinline__ void update_any(const AdamWScalars& k, const AdamWTensor& t, Step& s, int64_t chunk) {
    if (k.stochastic) {
        const int64_t step = k.step != nullptr ? (k.step[0] < 1 ? 1 : k.step[0]) : k.host_step;
        s.mix = scramble(k.seed + scramble((uint32_t)step + scramble(t.kind >> kAdamWPlace)));
        switch (t.kind & 7) {
            case 4: return update<false, false, true, true>(t, s, chunk);
            case 5: return update<true, false, true, true>(t, s, chunk);
            case 6: return update<false, true, true, true>(t, s, chunk);
            case 7: return update<true, true, true, true>(t, s, chunk);
            default: break;   // fp32 states
        }
    }
    switch (t.kind & 7) {
        case 0: return update<false, false, false, false>(t, s, chunk);
        case 1: return update<true, false, false, false>(t, s, chunk);
        case 2: return update<false, true, false, false>(t, s, chunk);
        case 3: return update<true, true, false, false>(t, s, chunk);
        case 4: return update<false, false, true, false>(t, s, chunk);
        case 5: return update<true, false, true, false>(t, s, chunk);
        case 6: return update<false, true, true, false>(t, s, chunk);
        default: return update<true, true, true, false>(t, s, chunk);
    }
}

__global__ __launch_bounds__(256) void adamw_kernel(AdamWArgs a) {
    __shared__ float now[3];
    Step s = step_of(a.k, now);
    int lo = 0, hi = a.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.tensor[mid].first <= blockIdx.x) lo = mid;
        else hi = mid - 1;
    }
    const AdamWTensor t = a.tensor[lo];
    update_any(a.k, t, s, blockIdx.x - t.first);
}

// The tensor is the last one whose first chunk is at or before the workgroup's:
// 64 of them are looked at at once.
__global__ __launch_bounds__(256) void adamw_table_kernel(AdamWScalars k, AdamWTable table) {
    __shared__ float now[3];
    int64_t lo = 0, hi = table.count;   // the number of first chunks <= blockIdx.x
    while (lo < hi) {
        const int64_t step = (hi - lo + 63) >> 6, at = lo + (threadIdx.x & 63) * step;
        const int c = __popcll(__ballot(at < hi && table.first[at] <= blockIdx.x));
        if (c == 0) break;
        const int64_t end = lo + c * step;
        lo = lo + (c - 1) * step + 1;
        hi = end < hi ? end : hi;
    }
    Step s = step_of(k, now);
    const AdamWTensor t = table.tensor[lo - 1];
    update_any(k, t, s, blockIdx.x - t.first);
}

}  // namespace

void launch_adamw(const AdamWArgs& a, hipStream_t s) { adamw_kernel<<<a.chunks, 256, 0, s>>>(a); }
void launch_adamw_table(const AdamWScalars& k, const AdamWTable& t, uint32_t chunks, hipStream_t s) {
    adamw_table_kernel<<<chunks, 256, 0, s>>>(k, t);
}

}  // namespace lmhead
