// train_api.hip — host side of the C ABI declared in include/lmhead_train.h:
// argument validation and launches. Host-checkable errors return before
// anything is enqueued; nothing here allocates or synchronises.
#include <math.h>

#include <hip/hip_runtime.h>

#include "host_util.h"
#include "lmhead_train.h"
#include "train_kernels.h"

namespace {

using namespace lmhead;

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxVocab = int64_t(1) << 30;
constexpr int64_t kMaxHidden = 65536;
constexpr int64_t kMaxGroups = 16777215;   // 256-thread workgroups of one launch: 2^32 - 1 work-items
constexpr int64_t kMaxGathered = int64_t(1) << 26;    // tokens of an embedding gradient
constexpr int64_t kMaxGradVocab = int64_t(1) << 28;   // 1024 threads for each 512 ids
constexpr int64_t kMaxSequences = int64_t(1) << 24;
constexpr int64_t kMaxTensors = int64_t(1) << 20;
constexpr int64_t kMaxNumel = (int64_t(1) << 35) - (int64_t(1) << 24);
constexpr float kMaxFloat = 3.402823466e38f;

// as the fp32 number that the kernels get
bool finite32(double v) { return (float)v >= -kMaxFloat && (float)v <= kMaxFloat; }
bool dtype_ok(int32_t d) { return d == LMHEAD_DTYPE_BF16 || d == LMHEAD_DTYPE_F32; }

int validate(const lmhead_embedding* p, bool backward) {
    if (p == nullptr || !dtype_ok(p->out_dtype) || (p->accumulate != 0 && p->accumulate != 1)) return LMHEAD_ERR_ARG;
    if (!dtype_ok(p->weight_dtype) && (backward || p->weight_dtype != LMHEAD_DTYPE_E4M3)) return LMHEAD_ERR_ARG;
    if (!finite32(p->scale)) return LMHEAD_ERR_ARG;
    if (p->n < 0 || p->n > kMaxRows || p->vocab < 1 || p->vocab > kMaxVocab) return LMHEAD_ERR_SHAPE;
    if (p->hidden < 64 || p->hidden > kMaxHidden || p->hidden % 64 != 0) return LMHEAD_ERR_SHAPE;
    if (p->weight_dtype == LMHEAD_DTYPE_E4M3 && p->hidden % kQBlock != 0) return LMHEAD_ERR_SHAPE;
    if (backward && (p->n > kMaxGathered || p->vocab > kMaxGradVocab || cdiv(p->n, 16) * cdiv(p->hidden, 1024) > kMaxGroups))
        return LMHEAD_ERR_SHAPE;
    return LMHEAD_OK;
}

int validate(const lmhead_policy_problem* p) {
    if (p == nullptr || p->reserved != 0 || p->num_valid < -1) return LMHEAD_ERR_ARG;
    if (!(p->clip_low >= 0.0 && p->clip_low <= 1.0) || !(p->clip_high >= 0.0) || !finite32(p->clip_high))
        return LMHEAD_ERR_ARG;
    if (p->dual_clip != 0.0 && (!(p->dual_clip > 1.0) || !finite32(p->dual_clip))) return LMHEAD_ERR_ARG;
    if (!finite32(p->kl_weight) || p->kl_kind < LMHEAD_KL_K1 || p->kl_kind > LMHEAD_KL_K3) return LMHEAD_ERR_ARG;
    if (p->reduction < LMHEAD_REDUCE_MEAN || p->reduction > LMHEAD_REDUCE_SEQUENCE_MEAN) return LMHEAD_ERR_ARG;
    if (p->advantage_per_sequence != 0 && (p->advantage_per_sequence != 1 || p->sequences == 0)) return LMHEAD_ERR_ARG;
    if (p->n < 0 || p->n > kMaxRows || p->sequences < 0 || p->sequences > kMaxSequences) return LMHEAD_ERR_SHAPE;
    return LMHEAD_OK;
}

int validate(const lmhead_preference_problem* p) {
    if (p == nullptr || p->num_pairs < -1 || (p->average != 0 && p->average != 1)) return LMHEAD_ERR_ARG;
    if (p->kind < LMHEAD_PREFERENCE_SIGMOID || p->kind > LMHEAD_PREFERENCE_SQUARED) return LMHEAD_ERR_ARG;
    if (!((float)p->beta > 0.0f) || !finite32(p->beta) || !finite32(p->margin)) return LMHEAD_ERR_ARG;
    if (!(p->label_smoothing >= 0.0 && p->label_smoothing <= 0.5)) return LMHEAD_ERR_ARG;
    if (p->label_smoothing != 0.0 && p->kind != LMHEAD_PREFERENCE_SIGMOID) return LMHEAD_ERR_ARG;
    if (p->n < 0 || p->n > kMaxRows || p->pairs < 1 || p->pairs > kMaxSequences / 2) return LMHEAD_ERR_SHAPE;
    return LMHEAD_OK;
}

int validate(const lmhead_adamw* p) {
    if (p == nullptr || !finite32(p->lr) || !(p->weight_decay >= 0.0) || !finite32(p->weight_decay))
        return LMHEAD_ERR_ARG;
    // as fp32 too: 1 would leave no step at all
    if (!(p->beta1 >= 0.0 && (float)p->beta1 < 1.0f) || !(p->beta2 >= 0.0 && (float)p->beta2 < 1.0f))
        return LMHEAD_ERR_ARG;
    if (!((float)p->eps >= 0x1p-126f) || !finite32(p->eps) || p->step < 1) return LMHEAD_ERR_ARG;
    if (p->stochastic != 0 && p->stochastic != 1) return LMHEAD_ERR_ARG;
    return LMHEAD_OK;
}

int check(const lmhead_adamw_tensor& t) {
    if (!dtype_ok(t.param_dtype) || !dtype_ok(t.grad_dtype) || t.reserved != 0) return LMHEAD_ERR_ARG;
    const bool e8 = t.state_dtype == LMHEAD_DTYPE_E4M3;
    if (!e8 && t.state_dtype != LMHEAD_DTYPE_F32) return LMHEAD_ERR_ARG;
    if (t.numel < 0 || t.numel > kMaxNumel) return LMHEAD_ERR_SHAPE;
    if (t.numel == 0) return LMHEAD_OK;
    if (t.param == nullptr || t.grad == nullptr || t.exp_avg == nullptr || t.exp_avg_sq == nullptr) return LMHEAD_ERR_ARG;
    if ((t.exp_avg_scale != nullptr) != e8 || (t.exp_avg_sq_scale != nullptr) != e8) return LMHEAD_ERR_ARG;
    if (!aligned(t.param, t.param_dtype == LMHEAD_DTYPE_F32 ? 4 : 2) ||
        !aligned(t.grad, t.grad_dtype == LMHEAD_DTYPE_F32 ? 4 : 2) || !aligned(t.exp_avg, e8 ? 1 : 4) ||
        !aligned(t.exp_avg_sq, e8 ? 1 : 4) || !aligned(t.exp_avg_scale, 4) || !aligned(t.exp_avg_sq_scale, 4) ||
        !aligned(t.copy, 2))
        return LMHEAD_ERR_ALIGN;
    return LMHEAD_OK;
}

int64_t chunks_of(const lmhead_adamw_tensor& t) {   // at most 2^24 - 2^13, of fp32 states
    return cdiv(t.numel, t.state_dtype == LMHEAD_DTYPE_E4M3 ? kAdamWChunk8 : kAdamWChunk);
}

size_t table_tensors(int64_t count) { return (size_t)round_up(4 * count, 64); }   // where a table's tensors begin

AdamWTensor packed(const lmhead_adamw_tensor& t, int64_t place, uint32_t first) {
    AdamWTensor o;
    const bool e8 = t.state_dtype == LMHEAD_DTYPE_E4M3;
    o.param = t.param;
    o.grad = t.grad;
    o.m = t.exp_avg;
    o.v = t.exp_avg_sq;
    o.m_scale = t.exp_avg_scale;
    o.v_scale = t.exp_avg_sq_scale;
    o.copy = (bf16_bits*)t.copy;
    o.numel = t.numel;
    o.first = first;
    o.kind = (t.param_dtype == LMHEAD_DTYPE_F32 ? kAdamWParamF32 : 0) |
             (t.grad_dtype == LMHEAD_DTYPE_F32 ? kAdamWGradF32 : 0) | (e8 ? kAdamWState8 : 0) |
             (uint32_t)place << kAdamWPlace;
    if (aligned(t.param, 16) && aligned(t.grad, 16) && aligned(t.exp_avg, e8 ? 8 : 16) &&
        aligned(t.exp_avg_sq, e8 ? 8 : 16) && aligned(t.copy, 16))
        o.kind |= kAdamWWide;
    return o;
}

Tokens tokens(int64_t n, int64_t sequences, const int32_t* targets, const int32_t* cu) {
    Tokens t;
    t.targets = targets;
    t.cu = cu;
    t.n = n;
    t.sequences = sequences > 0 ? sequences : 1;
    return t;
}

PolicyArgs policy_args(const lmhead_policy_problem* p, const float* logp, const float* old_logp, const float* ref_logp,
                       const float* advantage, const int32_t* targets, const int32_t* cu) {
    PolicyArgs a;
    a.t = tokens(p->n, p->sequences, targets, cu);
    a.logp = logp;
    a.old_logp = old_logp;
    a.ref_logp = ref_logp;
    a.advantage = advantage;
    a.per_sequence = p->advantage_per_sequence;
    a.reduction = p->reduction;
    a.kl_kind = p->kl_kind;
    a.num_valid = p->num_valid;
    a.log_high = log1p(p->clip_high);
    a.log_low = log1p(-p->clip_low);
    a.log_dual = p->dual_clip > 0.0 ? log(p->dual_clip) : HUGE_VAL;
    a.high = (float)(1.0 + p->clip_high);
    a.low = (float)(1.0 - p->clip_low);
    a.dual = (float)p->dual_clip;
    a.kl_weight = (float)p->kl_weight;
    a.loss = a.stats = a.weights = nullptr;
    return a;
}

// what both directions of the policy loss ask of the arrays
int policy_arrays(const lmhead_policy_problem* p, const float* logp, const float* old_logp, const float* ref_logp,
                  const float* advantage, const int32_t* targets, const int32_t* cu) {
    if (p->n > 0 && (logp == nullptr || advantage == nullptr)) return LMHEAD_ERR_ARG;
    if ((p->sequences > 0) != (cu != nullptr)) return LMHEAD_ERR_ARG;
    if (p->kl_weight != 0.0 && ref_logp == nullptr && p->n > 0) return LMHEAD_ERR_ARG;
    if (!aligned(logp, 4) || !aligned(old_logp, 4) || !aligned(ref_logp, 4) || !aligned(advantage, 4) ||
        !aligned(targets, 4) || !aligned(cu, 4))
        return LMHEAD_ERR_ALIGN;
    return LMHEAD_OK;
}

}  // namespace

extern "C" {

int lmhead_embedding_fwd(const lmhead_embedding* p, const int32_t* ids, const void* weight,
                         const float* weight_scale, void* out, void* workspace, size_t workspace_bytes,
                         void* stream) {
    int st = validate(p, false);
    if (st != LMHEAD_OK) return st;
    const bool e8 = p->weight_dtype == LMHEAD_DTYPE_E4M3;
    if (p->n > 0 && (ids == nullptr || weight == nullptr || out == nullptr || (weight_scale != nullptr) != e8))
        return LMHEAD_ERR_ARG;
    if (!aligned(ids, 4) || !aligned(weight, 16) || !aligned(weight_scale, 4) || !aligned(out, 16) ||
        !aligned(workspace, 256))
        return LMHEAD_ERR_ALIGN;
    if (workspace != nullptr && workspace_bytes < 256) return LMHEAD_ERR_WORKSPACE;
    st = check_device();
    if (st != LMHEAD_OK) return st;
    if (p->n == 0) {
        if (workspace == nullptr) return LMHEAD_OK;
        init_header_kernel<<<1, 64, 0, (hipStream_t)stream>>>((int32_t*)workspace);
        return launched();
    }
    EmbedArgs a;
    a.ids = ids;
    a.weight = weight;
    a.weight_scale = weight_scale;
    a.out = out;
    a.n = p->n;
    a.vocab = p->vocab;
    a.hidden = (int)p->hidden;
    a.scale = p->scale;
    a.hdr = (int32_t*)workspace;
    a.weight_type = e8 ? kEmbedE4m3 : p->weight_dtype == LMHEAD_DTYPE_F32 ? kEmbedF32 : kEmbedBf16;
    a.out_f32 = p->out_dtype == LMHEAD_DTYPE_F32;
    launch_embedding(a, (hipStream_t)stream);
    return launched();
}

size_t lmhead_embedding_bwd_workspace_size(const lmhead_embedding* p) {
    return validate(p, true) == LMHEAD_OK ? embedding_bwd_workspace(p->n, p->vocab, (int)p->hidden) : 0;
}

int lmhead_embedding_bwd(const lmhead_embedding* p, const int32_t* ids, const void* dout, void* dweight,
                         void* workspace, size_t workspace_bytes, void* stream) {
    int st = validate(p, true);
    if (st != LMHEAD_OK) return st;
    if (workspace == nullptr || dweight == nullptr) return LMHEAD_ERR_ARG;
    if (p->n > 0 && (ids == nullptr || dout == nullptr)) return LMHEAD_ERR_ARG;
    if (!aligned(ids, 4) || !aligned(dout, 16) || !aligned(dweight, 16) || !aligned(workspace, 256))
        return LMHEAD_ERR_ALIGN;
    if (workspace_bytes < lmhead_embedding_bwd_workspace_size(p)) return LMHEAD_ERR_WORKSPACE;
    st = check_device();
    if (st != LMHEAD_OK) return st;
    EmbedBwdArgs a;
    a.ids = ids;
    a.dout = dout;
    a.dweight = dweight;
    a.n = p->n;
    a.vocab = p->vocab;
    a.hidden = (int)p->hidden;
    a.scale = p->scale;
    a.dout_f32 = p->out_dtype == LMHEAD_DTYPE_F32;
    a.dweight_f32 = p->weight_dtype == LMHEAD_DTYPE_F32;
    a.accumulate = p->accumulate;
    launch_embedding_bwd(a, workspace, (hipStream_t)stream);
    return launched();
}

size_t lmhead_policy_loss_workspace_size(const lmhead_policy_problem* p) {
    return validate(p) == LMHEAD_OK ? policy_workspace(p->n, p->sequences > 0 ? p->sequences : 1, p->reduction) : 0;
}

int lmhead_policy_loss_fwd(const lmhead_policy_problem* p, const float* logp, const float* old_logp,
                           const float* ref_logp, const float* advantage, const int32_t* targets,
                           const int32_t* cu_seqlens, float* loss, float* stats, float* weights,
                           void* workspace, size_t workspace_bytes, void* stream) {
    int st = validate(p);
    if (st != LMHEAD_OK) return st;
    if (loss == nullptr || weights == nullptr || workspace == nullptr) return LMHEAD_ERR_ARG;
    st = policy_arrays(p, logp, old_logp, ref_logp, advantage, targets, cu_seqlens);
    if (st != LMHEAD_OK) return st;
    if (!aligned(loss, 4) || !aligned(stats, 4) || !aligned(weights, 4) || !aligned(workspace, 256))
        return LMHEAD_ERR_ALIGN;
    if (workspace_bytes < lmhead_policy_loss_workspace_size(p)) return LMHEAD_ERR_WORKSPACE;
    st = check_device();
    if (st != LMHEAD_OK) return st;
    PolicyArgs a = policy_args(p, logp, old_logp, ref_logp, advantage, targets, cu_seqlens);
    a.loss = loss;
    a.stats = stats;
    a.weights = weights;
    launch_policy(a, workspace, (hipStream_t)stream);
    return launched();
}

int lmhead_policy_loss_bwd(const lmhead_policy_problem* p, const float* grad, const float* weights,
                           const float* logp, const float* old_logp, const float* ref_logp,
                           const float* advantage, const int32_t* targets, const int32_t* cu_seqlens,
                           float* dlogp, void* stream) {
    int st = validate(p);
    if (st != LMHEAD_OK) return st;
    if (p->n > 0 && (grad == nullptr || weights == nullptr || dlogp == nullptr)) return LMHEAD_ERR_ARG;
    st = policy_arrays(p, logp, old_logp, ref_logp, advantage, targets, cu_seqlens);
    if (st != LMHEAD_OK) return st;
    if (!aligned(grad, 4) || !aligned(weights, 4) || !aligned(dlogp, 4)) return LMHEAD_ERR_ALIGN;
    st = check_device();
    if (st != LMHEAD_OK) return st;
    if (p->n == 0) return LMHEAD_OK;
    PolicyArgs a = policy_args(p, logp, old_logp, ref_logp, advantage, targets, cu_seqlens);
    a.weights = const_cast<float*>(weights);
    launch_policy_bwd(a, grad, dlogp, (hipStream_t)stream);
    return launched();
}

size_t lmhead_preference_loss_workspace_size(const lmhead_preference_problem* p) {
    return validate(p) == LMHEAD_OK ? preference_workspace(p->n, p->pairs) : 0;
}

int lmhead_preference_loss_fwd(const lmhead_preference_problem* p, const float* logp, const float* ref_logp,
                               const int32_t* targets, const int32_t* cu_seqlens, float* loss,
                               float* rewards, float* coef, void* workspace, size_t workspace_bytes,
                               void* stream) {
    int st = validate(p);
    if (st != LMHEAD_OK) return st;
    if (loss == nullptr || coef == nullptr || workspace == nullptr || cu_seqlens == nullptr) return LMHEAD_ERR_ARG;
    if (p->n > 0 && logp == nullptr) return LMHEAD_ERR_ARG;
    if (!aligned(logp, 4) || !aligned(ref_logp, 4) || !aligned(targets, 4) || !aligned(cu_seqlens, 4) ||
        !aligned(loss, 4) || !aligned(rewards, 4) || !aligned(coef, 4) || !aligned(workspace, 256))
        return LMHEAD_ERR_ALIGN;
    if (workspace_bytes < lmhead_preference_loss_workspace_size(p)) return LMHEAD_ERR_WORKSPACE;
    st = check_device();
    if (st != LMHEAD_OK) return st;
    PreferenceArgs a;
    a.t = tokens(p->n, 2 * p->pairs, targets, cu_seqlens);
    a.logp = logp;
    a.ref_logp = ref_logp;
    a.kind = p->kind;
    a.average = p->average;
    a.num_pairs = p->num_pairs;
    a.beta = p->beta;
    a.margin = p->margin;
    a.smoothing = p->label_smoothing;
    a.loss = loss;
    a.rewards = rewards;
    a.coef = coef;
    launch_preference(a, workspace, (hipStream_t)stream);
    return launched();
}

int lmhead_preference_loss_bwd(const lmhead_preference_problem* p, const float* grad, const float* coef,
                               const int32_t* targets, const int32_t* cu_seqlens, float* dlogp, void* stream) {
    int st = validate(p);
    if (st != LMHEAD_OK) return st;
    if (p->n > 0 && (grad == nullptr || coef == nullptr || cu_seqlens == nullptr || dlogp == nullptr))
        return LMHEAD_ERR_ARG;
    if (!aligned(grad, 4) || !aligned(coef, 4) || !aligned(targets, 4) || !aligned(cu_seqlens, 4) || !aligned(dlogp, 4))
        return LMHEAD_ERR_ALIGN;
    st = check_device();
    if (st != LMHEAD_OK) return st;
    if (p->n == 0) return LMHEAD_OK;
    launch_preference_bwd(tokens(p->n, 2 * p->pairs, targets, cu_seqlens), grad, coef, dlogp, (hipStream_t)stream);
    return launched();
}

size_t lmhead_adamw_table_size(int64_t count) {
    return count < 0 || count > kMaxTensors ? 0 : table_tensors(count) + (size_t)count * sizeof(AdamWTensor);
}

int lmhead_adamw_table(const lmhead_adamw_tensor* tensors, int64_t count, void* table, size_t table_bytes) {
    if (count < 0 || count > kMaxTensors) return LMHEAD_ERR_SHAPE;
    if (count > 0 && (tensors == nullptr || table == nullptr)) return LMHEAD_ERR_ARG;
    if (!aligned(table, 8)) return LMHEAD_ERR_ALIGN;
    if (table_bytes < lmhead_adamw_table_size(count)) return LMHEAD_ERR_WORKSPACE;
    for (int64_t i = 0; i < count; ++i) {
        const int st = check(tensors[i]);
        if (st != LMHEAD_OK) return st;
    }
    uint32_t* first = (uint32_t*)table;
    AdamWTensor* out = (AdamWTensor*)((char*)table + table_tensors(count));
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (chunks > kMaxGroups) return LMHEAD_ERR_SHAPE;
        first[i] = (uint32_t)chunks;
        out[i] = packed(tensors[i], i, (uint32_t)chunks);
        chunks += chunks_of(tensors[i]);
    }
    return chunks > kMaxGroups ? LMHEAD_ERR_SHAPE : LMHEAD_OK;
}

int lmhead_adamw_step(const lmhead_adamw* p, const lmhead_adamw_tensor* tensors, int64_t count, const void* table,
                      void* stream) {
    int st = validate(p);
    if (st != LMHEAD_OK) return st;
    if (count < 0 || count > kMaxTensors) return LMHEAD_ERR_SHAPE;
    if (count > 0 && tensors == nullptr) return LMHEAD_ERR_ARG;
    if (!aligned(p->device_step, 4) || !aligned(p->device_lr, 4) || !aligned(p->grad_scale, 4) || !aligned(table, 8))
        return LMHEAD_ERR_ALIGN;
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i) {
        st = check(tensors[i]);
        if (st != LMHEAD_OK) return st;
        chunks += chunks_of(tensors[i]);
    }
    st = check_device();
    if (st != LMHEAD_OK) return st;
    AdamWArgs a;
    AdamWScalars& k = a.k;
    k.beta1 = (float)p->beta1;
    k.rest1 = (float)(1.0 - p->beta1);
    k.beta2 = (float)p->beta2;
    k.rest2 = (float)(1.0 - p->beta2);
    k.eps = (float)p->eps;
    k.weight_decay = p->weight_decay;
    k.log_beta1 = log(p->beta1);   // beta 0: -infinity, and 1 - beta^t = 1
    k.log_beta2 = log(p->beta2);
    k.step = p->device_step;
    k.device_lr = p->device_lr;
    k.host_lr = p->lr;
    k.host_step = p->step;
    k.grad_scale = p->grad_scale;
    k.stochastic = p->stochastic;
    k.seed = p->seed;
    k.keep = (float)(1.0 - p->lr * p->weight_decay);
    k.step_size = (float)(p->lr / -expm1((double)p->step * k.log_beta1));
    k.root_scale = (float)(1.0 / sqrt(-expm1((double)p->step * k.log_beta2)));
    if (table != nullptr && count > kAdamWTensors && chunks > 0 && chunks <= kMaxGroups) {
        AdamWTable t;
        t.first = (const uint32_t*)table;
        t.tensor = (const AdamWTensor*)((const char*)table + table_tensors(count));
        t.count = count;
        launch_adamw_table(k, t, (uint32_t)chunks, (hipStream_t)stream);
        return launched();
    }
    a.count = 0;
    a.chunks = 0;
    const auto flush = [&]() {
        if (a.count > 0) launch_adamw(a, (hipStream_t)stream);
        a.count = 0;
        a.chunks = 0;
    };
    for (int64_t i = 0; i < count; ++i) {
        if (tensors[i].numel == 0) continue;
        const int64_t more = chunks_of(tensors[i]);
        if (a.count == kAdamWTensors || a.chunks + more > kMaxGroups) flush();
        a.tensor[a.count++] = packed(tensors[i], i, a.chunks);
        a.chunks += (uint32_t)more;
    }
    flush();
    return launched();
}

}  // extern "C"
