// decode_kernels.h — argument blocks and declarations shared by the kernels
// around the projection (rms_norm.hip, logits_fp8.hip, sample.hip) and their
// host side (decode_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lmhead_kernels.h"

namespace lmhead {

constexpr int kDevErrLogit = 8;
constexpr int kDevErrSampling = 16;
constexpr float kE4m3Max = 448.0f;
constexpr int kQBlock = 128;   // columns per scale

// Scale of a block whose largest magnitude is amax (lmhead_decode.h).
__device__ __forceinline__ float block_scale(float amax) {
    return amax > 0.0f ? fmaxf(amax / kE4m3Max, 1.17549435e-38f) : 1.0f;
}

// ------------------------------------------------------------ rms_norm.hip
struct NormArgs {
    const bf16_bits *x, *residual;
    const void* weight;
    int weight_f32;
    bf16_bits *residual_out, *y;
    uint8_t* q;
    float *scale, *rstd;
    int64_t n;
    int hidden;
    float eps, offset;
};
struct NormBwdArgs {
    const bf16_bits *dy, *r, *dresidual;
    const void* weight;
    int weight_f32;
    const float* rstd;
    bf16_bits* dx;
    float* partial;   // [groups, hidden], null: no dweight
    int64_t n;
    int groups;       // workgroups: group g takes rows g, g + groups, ...
    int hidden;
    float offset;
};
constexpr int kNormMaxGroups = 512;
void launch_rms_norm(const NormArgs& a, hipStream_t s);
void launch_rms_norm_bwd(const NormBwdArgs& a, void* dweight, hipStream_t s);
void launch_quantize(const bf16_bits* x, int64_t rows, int cols, int block_rows, uint8_t* q, float* scale,
                     hipStream_t s);

// ---------------------------------------------------------- logits_fp8.hip
struct LogitsArgs {
    const uint8_t *a, *w;
    const float *a_scale, *w_scale;
    void* out;
    int out_f32;
    int64_t n, vocab, ld;
    int hidden;
    int quads;   // four consecutive logits of a row from a column that four divides are aligned to their size
    int lines;   // so are 16 bytes of them
};
size_t logits_workspace(int64_t n, int hidden, int out_f32);
void launch_logits(const LogitsArgs& a, void* workspace, hipStream_t s);

// -------------------------------------------------------------- sample.hip
constexpr int kWeightBits = 44;   // finest step of the integer weights: 2^-44
struct SampleArgs {
    const void* logits;
    int logits_f32;
    int64_t n, vocab, ld;
    Temperature T;
    int top_k;
    float top_p, min_p;
    const int32_t* row_top_k;
    const float *row_top_p, *row_min_p;
    const float* u;
    int32_t* token;
    float* logprob;
    int32_t* hdr;
    int shift;   // weights are integers of 2^-shift
};
size_t sample_workspace(int64_t n, int64_t vocab);
void launch_sample(const SampleArgs& a, void* workspace, hipStream_t s);

}  // namespace lmhead
