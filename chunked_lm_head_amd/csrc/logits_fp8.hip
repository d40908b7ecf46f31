// logits_fp8.hip — logits from e4m3 rows and an e4m3 vocabulary matrix with a
// scale per block of 128 columns (rows) or 128 x 128 (W):
//   out[i, v] = sum_b sa[i, b] sw[v / 128, b] sum_{j in b} a[i, j] w[v, j].
// The e4m3 values are widened to bf16 (exact: 4 significant bits) and the inner
// sum of a block is four v_mfma_f32_16x16x32_bf16, whose products and sums
// keep fp32 precision; it is added to the fp32 sum after the two scales, in
// ascending b. The 8-bit matrix instructions do not keep that precision: they
// align each 8 consecutive products to the largest and cut them off 13 bits
// below its power of two, which left sums 1.5e-5 off (relative, 2-norm).
#include "decode_kernels.h"
#include "host_util.h"

namespace lmhead {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// four e4m3 values to bf16 (gfx950's packed conversion, scale 1)
__device__ __forceinline__ void widen4(uint32_t v, bf16x8& f, int at) {
    const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false);
    const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true);
    f[at] = lo[0], f[at + 1] = lo[1], f[at + 2] = hi[0], f[at + 3] = hi[1];
}

// A 16 x 128 operand block as four 16 x 32 bf16 fragments: lane l holds row
// l % 16, bytes 16 (l / 16) .. + 16 of each 64-byte half. Both operands use the
// same order of k, so the sum over k does not depend on it, and a lane's two
// 16-byte loads sit in lines that the four lanes of its row read whole.
struct Frag {
    uint4 lo, hi;
    __device__ __forceinline__ void load(const uint8_t* row, int k0, int g) {
        lo = *reinterpret_cast<const uint4*>(row + k0 + 16 * g);
        hi = *reinterpret_cast<const uint4*>(row + k0 + 64 + 16 * g);
    }
    __device__ __forceinline__ bf16x8 part(int s) const {
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        bf16x8 f;
        widen4(w[2 * s], f, 0);
        widen4(w[2 * s + 1], f, 4);
        return f;
    }
};

__device__ __forceinline__ floatx4 block_sum(const Frag& a, const Frag& b) {
    floatx4 z = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < 4; ++s) z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.part(s), b.part(s), z, 0, 0, 0);
    return z;
}

// One wave per 16 vocabulary rows x 16 input rows.
__global__ __launch_bounds__(256) void logits_tile16_kernel(LogitsArgs a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int64_t tiles_v = (a.vocab + 63) / 64;
    const int64_t ti = blockIdx.x / tiles_v, tv = blockIdx.x - ti * tiles_v;
    const int64_t v0 = tv * 64 + wave * 16, i0 = ti * 16;
    if (v0 >= a.vocab) return;
    const int nb = a.hidden / kQBlock;
    const int64_t vr = v0 + c < a.vocab ? v0 + c : a.vocab - 1;
    const int64_t ir = i0 + c < a.n ? i0 + c : a.n - 1;
    const uint8_t* w = a.w + vr * a.hidden;
    const uint8_t* x = a.a + ir * a.hidden;
    const float* sa = a.a_scale + ir * nb;
    const float* sw = a.w_scale + (v0 / kQBlock) * nb;   // 16 rows from a multiple of 16: one block
    floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int b = 0; b < nb; ++b) {
        Frag fw, fx;
        fw.load(w, b * kQBlock, g);
        fx.load(x, b * kQBlock, g);
        const floatx4 z = block_sum(fw, fx);
        const float s = sa[b] * sw[b];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(z[e], s, acc[e]);
    }
    // lane holds vocabulary rows v0 + 4 g .. + 4 of input row i0 + c
    if (i0 + c >= a.n) return;
    const int64_t at = (i0 + c) * a.ld + v0 + 4 * g;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (v0 + 4 * g + e >= a.vocab) break;
        if (a.out_f32)
            reinterpret_cast<float*>(a.out)[at + e] = acc[e];
        else
            reinterpret_cast<__bf16*>(a.out)[at + e] = (__bf16)acc[e];
    }
}

}  // namespace

void launch_logits(const LogitsArgs& a, void* workspace, hipStream_t s) {
    (void)workspace;
    logits_tile16_kernel<<<(unsigned)(cdiv(a.n, 16) * cdiv(a.vocab, 64)), 256, 0, s>>>(a);
}

}  // namespace lmhead
