// decode_api.hip — host side of the C ABI declared in include/lmhead_decode.h:
// argument validation and launches. Host-checkable errors return before
// anything is enqueued; nothing here allocates or synchronises.
#include <hip/hip_runtime.h>

#include "decode_kernels.h"
#include "host_util.h"
#include "lmhead_decode.h"

namespace {

using namespace lmhead;

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxVocab = int64_t(1) << 30;
constexpr int64_t kMaxHidden = 65536;
constexpr int64_t kMaxGroups = 16777215;   // 256-thread workgroups of one launch: 2^32 - 1 work-items
constexpr float kMaxFloat = 3.402823466e38f;

bool finite(float v) { return v >= -kMaxFloat && v <= kMaxFloat; }
bool dtype_ok(int32_t d) { return d == LMHEAD_DTYPE_BF16 || d == LMHEAD_DTYPE_F32; }

int validate(const lmhead_norm* p) {
    if (p == nullptr || p->reserved != 0 || !dtype_ok(p->weight_dtype)) return LMHEAD_ERR_ARG;
    if (!(p->eps >= 0.0f && p->eps <= kMaxFloat) || !finite(p->weight_offset)) return LMHEAD_ERR_ARG;
    if (p->n < 0 || p->n > kMaxRows) return LMHEAD_ERR_SHAPE;
    if (p->hidden < 64 || p->hidden > kMaxHidden || p->hidden % 64 != 0) return LMHEAD_ERR_SHAPE;
    return LMHEAD_OK;
}

int validate(const lmhead_fp8_problem* p) {
    if (p == nullptr || p->reserved != 0 || !dtype_ok(p->out_dtype)) return LMHEAD_ERR_ARG;
    if (p->n < 0 || p->n > (int64_t(1) << 24)) return LMHEAD_ERR_SHAPE;
    if (p->vocab < 1 || p->vocab > kMaxVocab || p->ld < p->vocab || p->ld > (int64_t(1) << 32)) return LMHEAD_ERR_SHAPE;
    if (p->hidden < kQBlock || p->hidden > kMaxHidden || p->hidden % kQBlock != 0) return LMHEAD_ERR_SHAPE;
    if (cdiv(p->n, 16) * cdiv(p->vocab, 64) > kMaxGroups) return LMHEAD_ERR_SHAPE;
    return LMHEAD_OK;
}

int validate(const lmhead_sample_problem* p) {
    if (p == nullptr || p->reserved != 0 || !dtype_ok(p->logits_dtype)) return LMHEAD_ERR_ARG;
    if (!(p->temperature >= 0.0f && p->temperature <= kMaxFloat)) return LMHEAD_ERR_ARG;
    if (!(p->top_p >= 0.0f && p->top_p <= 1.0f) || !(p->min_p >= 0.0f && p->min_p <= 1.0f) || p->top_k < 0)
        return LMHEAD_ERR_ARG;
    if (p->n < 0 || p->n > kMaxRows) return LMHEAD_ERR_SHAPE;
    if (p->vocab < 1 || p->vocab > kMaxVocab || p->ld < p->vocab || p->ld > (int64_t(1) << 32)) return LMHEAD_ERR_SHAPE;
    return LMHEAD_OK;
}

int64_t norm_groups(const lmhead_norm& p) { return p.n < kNormMaxGroups ? p.n : kNormMaxGroups; }

}  // namespace

extern "C" {

int lmhead_rms_norm_fwd(const lmhead_norm* p, const void* x, const void* residual, const void* weight,
                        void* residual_out, void* y, void* q, float* scale, float* rstd, void* stream) {
    int st = validate(p);
    if (st != LMHEAD_OK) return st;
    if ((q == nullptr) != (scale == nullptr)) return LMHEAD_ERR_ARG;
    if (residual_out != nullptr && residual == nullptr) return LMHEAD_ERR_ARG;
    if (residual_out != nullptr && residual_out == y) return LMHEAD_ERR_ARG;
    if (p->n > 0) {
        if (x == nullptr || weight == nullptr) return LMHEAD_ERR_ARG;
        if (y == nullptr && q == nullptr && rstd == nullptr && residual_out == nullptr) return LMHEAD_ERR_ARG;
    }
    if (q != nullptr && p->hidden % kQBlock != 0) return LMHEAD_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(residual_out, 16) ||
        !aligned(y, 16) || !aligned(q, 16) || !aligned(scale, 4) || !aligned(rstd, 4))
        return LMHEAD_ERR_ALIGN;
    st = check_device();
    if (st != LMHEAD_OK) return st;
    if (p->n == 0) return LMHEAD_OK;
    NormArgs a;
    a.x = (const bf16_bits*)x;
    a.residual = (const bf16_bits*)residual;
    a.weight = weight;
    a.weight_f32 = p->weight_dtype == LMHEAD_DTYPE_F32;
    a.residual_out = (bf16_bits*)residual_out;
    a.y = (bf16_bits*)y;
    a.q = (uint8_t*)q;
    a.scale = scale;
    a.rstd = rstd;
    a.n = p->n;
    a.hidden = (int)p->hidden;
    a.eps = p->eps;
    a.offset = p->weight_offset;
    launch_rms_norm(a, (hipStream_t)stream);
    return launched();
}

size_t lmhead_rms_norm_bwd_workspace_size(const lmhead_norm* p) {
    if (validate(p) != LMHEAD_OK) return 0;
    return (size_t)round_up(4 * (norm_groups(*p) > 0 ? norm_groups(*p) : 1) * p->hidden, 256);
}

int lmhead_rms_norm_bwd(const lmhead_norm* p, const void* dy, const void* r, const void* weight,
                        const float* rstd, const void* dresidual, void* dx, void* dweight,
                        void* workspace, size_t workspace_bytes, void* stream) {
    int st = validate(p);
    if (st != LMHEAD_OK) return st;
    if (p->n > 0 && (dy == nullptr || r == nullptr || weight == nullptr || rstd == nullptr)) return LMHEAD_ERR_ARG;
    if (dweight != nullptr && p->n > 0 && workspace == nullptr) return LMHEAD_ERR_ARG;
    if (!aligned(dy, 16) || !aligned(r, 16) || !aligned(weight, 16) || !aligned(rstd, 4) ||
        !aligned(dresidual, 16) || !aligned(dx, 16) || !aligned(dweight, 4) || !aligned(workspace, 256))
        return LMHEAD_ERR_ALIGN;
    if (dweight != nullptr && p->n > 0 && workspace_bytes < lmhead_rms_norm_bwd_workspace_size(p))
        return LMHEAD_ERR_WORKSPACE;
    st = check_device();
    if (st != LMHEAD_OK) return st;
    if (dx == nullptr && dweight == nullptr) return LMHEAD_OK;
    hipStream_t s = (hipStream_t)stream;
    const int weight_f32 = p->weight_dtype == LMHEAD_DTYPE_F32;
    if (p->n == 0) {
        const int64_t words = p->hidden * (weight_f32 ? 4 : 2) / 4;
        if (dweight != nullptr)
            fill_u32_kernel<<<grid_1d(words, kThreads, 4096), kThreads, 0, s>>>((uint32_t*)dweight, words, 0u);
        return launched();
    }
    NormBwdArgs a;
    a.dy = (const bf16_bits*)dy;
    a.r = (const bf16_bits*)r;
    a.dresidual = (const bf16_bits*)dresidual;
    a.weight = weight;
    a.weight_f32 = weight_f32;
    a.rstd = rstd;
    a.dx = (bf16_bits*)dx;
    a.partial = dweight != nullptr ? (float*)workspace : nullptr;
    a.n = p->n;
    a.groups = 0;
    a.hidden = (int)p->hidden;
    a.offset = p->weight_offset;
    launch_rms_norm_bwd(a, dweight, s);
    return launched();
}

int lmhead_quantize_fp8(int64_t rows, int64_t cols, int32_t block_rows, const void* x, void* q,
                        float* scale, void* stream) {
    if (block_rows != 1 && block_rows != kQBlock) return LMHEAD_ERR_ARG;
    if (rows < 0 || rows > kMaxRows || cols < kQBlock || cols > kMaxHidden || cols % kQBlock != 0)
        return LMHEAD_ERR_SHAPE;
    if (block_rows == kQBlock && cdiv(rows, kQBlock) * (cols / kQBlock) > kMaxGroups) return LMHEAD_ERR_SHAPE;
    if (rows > 0 && (x == nullptr || q == nullptr || scale == nullptr)) return LMHEAD_ERR_ARG;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4)) return LMHEAD_ERR_ALIGN;
    const int st = check_device();
    if (st != LMHEAD_OK) return st;
    if (rows == 0) return LMHEAD_OK;
    launch_quantize((const bf16_bits*)x, rows, (int)cols, block_rows, (uint8_t*)q, scale, (hipStream_t)stream);
    return launched();
}

size_t lmhead_logits_fp8_workspace_size(const lmhead_fp8_problem* p) {
    return validate(p) == LMHEAD_OK ? logits_workspace(p->n, (int)p->hidden, p->out_dtype == LMHEAD_DTYPE_F32) : 0;
}

int lmhead_logits_fp8(const lmhead_fp8_problem* p, const void* a, const float* a_scale, const void* w,
                      const float* w_scale, void* out, void* workspace, size_t workspace_bytes,
                      void* stream) {
    int st = validate(p);
    if (st != LMHEAD_OK) return st;
    if (workspace == nullptr) return LMHEAD_ERR_ARG;
    if (p->n > 0 && (a == nullptr || a_scale == nullptr || w == nullptr || w_scale == nullptr || out == nullptr))
        return LMHEAD_ERR_ARG;
    const int out_bytes = p->out_dtype == LMHEAD_DTYPE_F32 ? 4 : 2;
    if (!aligned(a, 16) || !aligned(a_scale, 4) || !aligned(w, 16) || !aligned(w_scale, 4) ||
        !aligned(out, out_bytes) || !aligned(workspace, 256))
        return LMHEAD_ERR_ALIGN;
    if (workspace_bytes < lmhead_logits_fp8_workspace_size(p)) return LMHEAD_ERR_WORKSPACE;
    st = check_device();
    if (st != LMHEAD_OK) return st;
    if (p->n == 0) return LMHEAD_OK;
    LogitsArgs g;
    g.a = (const uint8_t*)a;
    g.w = (const uint8_t*)w;
    g.a_scale = a_scale;
    g.w_scale = w_scale;
    g.out = out;
    g.out_f32 = p->out_dtype == LMHEAD_DTYPE_F32;
    g.n = p->n;
    g.vocab = p->vocab;
    g.ld = p->ld;
    g.hidden = (int)p->hidden;
    g.quads = p->ld % 4 == 0 && aligned(out, 4 * out_bytes);
    g.lines = p->ld % (16 / out_bytes) == 0 && aligned(out, 16);
    launch_logits(g, workspace, (hipStream_t)stream);
    return launched();
}

size_t lmhead_sample_workspace_size(const lmhead_sample_problem* p) {
    return validate(p) == LMHEAD_OK ? sample_workspace(p->n, p->vocab) : 0;
}

int lmhead_sample(const lmhead_sample_problem* p, const void* logits, const float* u, int32_t* token,
                  float* logprob, void* workspace, size_t workspace_bytes, void* stream) {
    int st = validate(p);
    if (st != LMHEAD_OK) return st;
    if (workspace == nullptr) return LMHEAD_ERR_ARG;
    if (p->n > 0 && (logits == nullptr || u == nullptr || token == nullptr)) return LMHEAD_ERR_ARG;
    if (!aligned(logits, p->logits_dtype == LMHEAD_DTYPE_F32 ? 4 : 2) || !aligned(workspace, 256) || !aligned(u, 4) ||
        !aligned(token, 4) || !aligned(logprob, 4) || !aligned(p->row_temperature, 4) || !aligned(p->row_top_k, 4) ||
        !aligned(p->row_top_p, 4) || !aligned(p->row_min_p, 4))
        return LMHEAD_ERR_ALIGN;
    if (workspace_bytes < lmhead_sample_workspace_size(p)) return LMHEAD_ERR_WORKSPACE;
    st = check_device();
    if (st != LMHEAD_OK) return st;
    hipStream_t s = (hipStream_t)stream;
    if (p->n == 0) {
        init_header_kernel<<<1, 64, 0, s>>>((int32_t*)workspace);
        return launched();
    }
    SampleArgs a;   // the first launch clears the header
    a.logits = logits;
    a.logits_f32 = p->logits_dtype == LMHEAD_DTYPE_F32;
    a.n = p->n;
    a.vocab = p->vocab;
    a.ld = p->ld;
    a.T.t = p->temperature == 0.0f ? 1.0f : p->temperature;
    a.T.row = p->row_temperature;
    a.top_k = p->top_k;
    a.top_p = p->top_p;
    a.min_p = p->min_p;
    a.row_top_k = p->row_top_k;
    a.row_top_p = p->row_top_p;
    a.row_min_p = p->row_min_p;
    a.u = u;
    a.token = token;
    a.logprob = logprob;
    a.hdr = (int32_t*)workspace;
    // vocab weights of at most 2^shift each sum below 2^63
    int bits = 0;
    while ((int64_t(1) << bits) < p->vocab) ++bits;
    a.shift = 62 - bits < kWeightBits ? 62 - bits : kWeightBits;
    launch_sample(a, workspace, s);
    return launched();
}

}  // extern "C"
