// vec8.h — eight consecutive values of a row in registers: bf16 (16 bytes),
// fp32 (two of 16) or e4m3 (8 bytes) in memory, fp32 in between.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_core.h"

namespace lmhead {

struct V8 {
    float v[8];
};

__device__ __forceinline__ V8 zeros8() { return V8{{0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}}; }

__device__ __forceinline__ V8 bf16_to8(const uint4& p) {
    V8 f;
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f.v[2 * i] = __builtin_bit_cast(float, w[i] << 16);
        f.v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
    }
    return f;
}
__device__ __forceinline__ uint4 to_bf16x8(const V8& f) {
    return make_uint4(pack_bf16x2(f.v[0], f.v[1]), pack_bf16x2(f.v[2], f.v[3]), pack_bf16x2(f.v[4], f.v[5]),
                      pack_bf16x2(f.v[6], f.v[7]));
}
__device__ __forceinline__ V8 e4m3_to8(const uint2& p) {
    V8 f;
    const uint32_t w[2] = {p.x, p.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
        f.v[4 * i] = lo[0];
        f.v[4 * i + 1] = lo[1];
        f.v[4 * i + 2] = hi[0];
        f.v[4 * i + 3] = hi[1];
    }
    return f;
}

// vector i of a row: elements 8 i .. 8 i + 7
template <bool F32>
__device__ __forceinline__ V8 load8(const void* p, int64_t i) {
    if (F32) {
        const float4 a = reinterpret_cast<const float4*>(p)[2 * i], b = reinterpret_cast<const float4*>(p)[2 * i + 1];
        return V8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    }
    return bf16_to8(reinterpret_cast<const uint4*>(p)[i]);
}
// as it stands in memory, to be turned into fp32 when it is used
template <bool F32>
struct Raw8 {
    uint4 w[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw8<F32> load_raw8(const void* p, int64_t i) {
    Raw8<F32> r;
#pragma unroll
    for (int k = 0; k < (F32 ? 2 : 1); ++k) r.w[k] = reinterpret_cast<const uint4*>(p)[(F32 ? 2 : 1) * i + k];
    return r;
}
template <bool F32>
__device__ __forceinline__ V8 to8(const Raw8<F32>& r) {
    if (!F32) return bf16_to8(r.w[0]);
    const uint4 a = r.w[0], b = r.w[F32 ? 1 : 0];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    V8 f;
#pragma unroll
    for (int c = 0; c < 8; ++c) f.v[c] = __builtin_bit_cast(float, w[c]);
    return f;
}

typedef uint32_t Words4 __attribute__((ext_vector_type(4)));

// STREAM: past the caches
template <bool STREAM>
__device__ __forceinline__ Words4 load_words(const void* p, int64_t i) {
    const Words4* at = reinterpret_cast<const Words4*>(p) + i;
    return STREAM ? __builtin_nontemporal_load(at) : *at;
}
template <bool STREAM>
__device__ __forceinline__ void store_words(void* p, int64_t i, const Words4& w) {
    Words4* at = reinterpret_cast<Words4*>(p) + i;
    if (STREAM) __builtin_nontemporal_store(w, at);
    else *at = w;
}
template <bool F32, bool STREAM = false>
__device__ __forceinline__ void store8(void* p, int64_t i, const V8& f) {
    if (F32) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            Words4 w;
#pragma unroll
            for (int c = 0; c < 4; ++c) w[c] = __builtin_bit_cast(uint32_t, f.v[4 * k + c]);
            store_words<STREAM>(p, 2 * i + k, w);
        }
    } else {
        const uint4 w = to_bf16x8(f);
        store_words<STREAM>(p, i, Words4{w.x, w.y, w.z, w.w});
    }
}

}  // namespace lmhead
