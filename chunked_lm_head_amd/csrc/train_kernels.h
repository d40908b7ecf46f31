// train_kernels.h — argument blocks and declarations shared by the kernels of a
// training step around the projection (embedding.hip, token_losses.hip,
// adamw.hip) and their host side (train_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decode_kernels.h"

namespace lmhead {

constexpr int kDevErrToken = 32;

// ----------------------------------------------------------- embedding.hip
enum EmbedType { kEmbedBf16 = 0, kEmbedF32 = 1, kEmbedE4m3 = 2 };

struct EmbedArgs {
    const int32_t* ids;
    const void* weight;
    const float* weight_scale;   // e4m3: [ceil(vocab / 128), hidden / 128]
    void* out;
    int64_t n, vocab;
    int hidden;
    float scale;
    int32_t* hdr;   // error word, or null
    int weight_type, out_f32;
};
void launch_embedding(const EmbedArgs& a, hipStream_t s);

struct EmbedBwdArgs {
    const int32_t* ids;
    const void* dout;
    void* dweight;
    int64_t n, vocab;
    int hidden;
    float scale;
    int dout_f32, dweight_f32, accumulate;
};
size_t embedding_bwd_workspace(int64_t n, int64_t vocab, int hidden);
void launch_embedding_bwd(const EmbedBwdArgs& a, void* workspace, hipStream_t s);

// -------------------------------------------------------- token_losses.hip
struct Tokens {
    const int32_t* targets;   // or null
    const int32_t* cu;        // or null: one sequence of all tokens
    int64_t n;
    int64_t sequences;        // at least 1
};
struct PolicyArgs {
    Tokens t;
    const float *logp, *old_logp, *ref_logp, *advantage;
    int per_sequence;   // advantage [sequences]
    int reduction;
    int kl_kind;
    int64_t num_valid;
    double log_high, log_low, log_dual;   // borders of logp - old_logp
    float high, low, dual;                // and of the ratio
    float kl_weight;
    float *loss, *stats, *weights;
};
size_t policy_workspace(int64_t n, int64_t sequences, int reduction);
void launch_policy(const PolicyArgs& a, void* workspace, hipStream_t s);
void launch_policy_bwd(const PolicyArgs& a, const float* grad, float* dlogp, hipStream_t s);

struct PreferenceArgs {
    Tokens t;
    const float *logp, *ref_logp;
    int kind, average;
    int64_t num_pairs;
    double beta, margin, smoothing;
    float *loss, *rewards, *coef;
};
size_t preference_workspace(int64_t n, int64_t pairs);
void launch_preference(const PreferenceArgs& a, void* workspace, hipStream_t s);
void launch_preference_bwd(const Tokens& t, const float* grad, const float* coef, float* dlogp, hipStream_t s);

// --------------------------------------------------------------- adamw.hip
struct AdamWTensor {
    void* param;
    const void* grad;
    void *m, *v;
    float *m_scale, *v_scale;
    bf16_bits* copy;
    int64_t numel;
    uint32_t first;   // its first chunk in the launch
    uint32_t kind;    // bits: kAdamW..., and from kAdamWPlace on its place in the call
};
constexpr uint32_t kAdamWParamF32 = 1, kAdamWGradF32 = 2, kAdamWState8 = 4, kAdamWWide = 8;
constexpr int kAdamWPlace = 4;
constexpr int kAdamWTensors = 48;   // per launch where the table travels as a kernel argument
struct AdamWScalars {
    float beta1, rest1, beta2, rest2, eps;
    float step_size, root_scale, keep;   // of the host's step and lr
    double log_beta1, log_beta2, weight_decay;
    const int32_t* step;
    const float* device_lr;
    double host_lr;
    int64_t host_step;
    const float* grad_scale;
    int stochastic;
    uint32_t seed;
};
struct AdamWArgs {
    AdamWScalars k;
    int count;
    uint32_t chunks;
    AdamWTensor tensor[kAdamWTensors];
};
// On the device: each tensor's first chunk, then the tensors.
struct AdamWTable {
    const uint32_t* first;
    const AdamWTensor* tensor;
    int64_t count;
};
// elements of a workgroup: 2048 with fp32 states, twice as many with 8-bit ones
constexpr int kAdamWChunk = 2048, kAdamWChunk8 = 4096;
void launch_adamw(const AdamWArgs& a, hipStream_t s);
void launch_adamw_table(const AdamWScalars& k, const AdamWTable& t, uint32_t chunks, hipStream_t s);

}  // namespace lmhead
