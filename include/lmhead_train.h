/*
 * lmhead_train.h — the operators around the vocabulary projection in a
 * training step, in the same library as lmhead.h (liblmhead.so, gfx950):
 *
 *   lmhead_embedding_fwd / _bwd        rows of the vocabulary matrix by token,
 *                                      scaled, and their gradient (whole, or
 *                                      added to what the projection's backward
 *                                      has accumulated);
 *   lmhead_policy_loss_fwd / _bwd      clipped policy loss with a KL term on
 *                                      lmhead_logprob's output;
 *   lmhead_preference_loss_fwd / _bwd  losses of pairs of answers on the same;
 *   lmhead_adamw_step                  AdamW over many tensors, states in fp32
 *                                      or in 8 bits.
 *
 * The conventions of lmhead.h hold for every entry: device pointers on the
 * current HIP device, caller-owned buffers and workspace, no allocation, no
 * synchronisation, all work on `stream`, host-checkable errors as a status
 * before anything is enqueued, reductions in a fixed order (two calls with
 * the same arguments give the same bits). n = 0 is a valid, empty call. An
 * output may be the same buffer as an input only where an entry says so. Two
 * calls in flight at once need a workspace each.
 */
#ifndef LMHEAD_TRAIN_H
#define LMHEAD_TRAIN_H

#include "lmhead_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Beside enum lmhead_dtype, where an entry says so. */
enum lmhead_train_dtype {
    LMHEAD_DTYPE_E4M3 = 2
};

/* Further device error codes (bits, beside enum lmhead_device_error). */
enum lmhead_train_device_error {
    LMHEAD_DEVERR_TOKEN = 32 /* a token id >= vocab */
};

/* ------------------------------------------------------------ embedding */

/*
 *   n             tokens, 0 <= n <= 2^30.
 *   vocab         1 <= vocab <= 2^30.
 *   hidden        a multiple of 64, 64 <= hidden <= 65536; with an 8-bit
 *                 weight a multiple of 128.
 *   scale         finite.
 *   weight_dtype  type of weight (enum lmhead_dtype, or LMHEAD_DTYPE_E4M3) and
 *                 of dweight (enum lmhead_dtype).
 *   out_dtype     type of out and dout (enum lmhead_dtype).
 *   accumulate    0 or 1, lmhead_embedding_bwd: 1 adds to dweight.
 *   The backward (launch sizes): n <= 2^26, vocab <= 2^28,
 *   ceil(n / 16) * ceil(hidden / 1024) <= 16,777,215.
 */
typedef struct lmhead_embedding {
    int64_t n;
    int64_t vocab;
    int64_t hidden;
    float scale;
    int32_t weight_dtype;
    int32_t out_dtype;
    int32_t accumulate;
} lmhead_embedding;

/*
 * out[i] = scale weight[ids[i]], one fp32 product (two with an 8-bit weight:
 * value times block scale first) and one rounding. A negative id marks a
 * padded place: its row is zero.
 *   ids           device, int32 [n].
 *   weight        device, weight_dtype [vocab, hidden].
 *   weight_scale  device, fp32 [ceil(vocab / 128), hidden / 128] with an 8-bit
 *                 weight (lmhead_quantize_fp8 with block_rows 128), else NULL.
 *   out           device, out_dtype [n, hidden].
 *   workspace     256 bytes for the error word, or NULL: an id >= vocab gives a
 *                 row of NaN either way.
 * weight and out 16-byte aligned, ids and weight_scale 4, workspace 256.
 */
int lmhead_embedding_fwd(const lmhead_embedding* p, const int32_t* ids, const void* weight,
                         const float* weight_scale, void* out, void* workspace, size_t workspace_bytes,
                         void* stream);

/* Bytes of workspace lmhead_embedding_bwd needs (0 for an invalid problem):
 * the tokens in the order of their ids, and fp32 sums of pieces of 16 tokens
 * (64 above 8192) of one id. */
size_t lmhead_embedding_bwd_workspace_size(const lmhead_embedding* p);

/*
 * dweight[v] = scale * sum of dout[i] over the tokens i with ids[i] = v, in
 * fp32 and in a fixed order, rounded once. Without accumulate the whole
 * [vocab, hidden] is written, zeros where no token has the id; with it the sum
 * is added (in fp32) to dweight[v], and rows without a token are neither read
 * nor written. Negative ids take no part; an id >= vocab takes none either and
 * sets the error word.
 *   dout       device, out_dtype [n, hidden].
 *   dweight    device, weight_dtype (bf16 or fp32) [vocab, hidden].
 * dout and dweight 16-byte aligned, ids 4, workspace 256.
 */
int lmhead_embedding_bwd(const lmhead_embedding* p, const int32_t* ids, const void* dout, void* dweight,
                         void* workspace, size_t workspace_bytes, void* stream);

/* ----------------------------------------- losses on log-probabilities */

/*
 * Both losses take packed tokens: sequence s holds the tokens cu_seqlens[s] ..
 * cu_seqlens[s + 1] - 1 (int32, ascending, within 0 .. n; a sequence may be
 * empty). A token counts when it lies in a sequence and its target is not
 * negative (targets int32 [n] as in lmhead.h, or NULL: all). A token that does
 * not count has gradient 0 whatever stands in its place in the other arrays.
 * cu_seqlens that descend give undefined numbers (no access goes astray).
 */

enum lmhead_kl_kind {
    LMHEAD_KL_K1 = 1, /* x, with x = logp - ref */
    LMHEAD_KL_K2 = 2, /* x^2 / 2 */
    LMHEAD_KL_K3 = 3  /* exp(-x) - 1 + x */
};

enum lmhead_reduction {
    LMHEAD_REDUCE_MEAN = 0,         /* over the tokens that count */
    LMHEAD_REDUCE_SUM = 1,
    LMHEAD_REDUCE_SEQUENCE_MEAN = 2 /* over sequences, of each one's mean (0 where none of its tokens counts) */
};

/*
 *   n                tokens, 0 <= n <= 2^30.
 *   sequences        0 <= sequences <= 2^24; 0: one sequence of all n tokens,
 *                    cu_seqlens NULL.
 *   num_valid        -1: the tokens that count (sequence mean: the sequences);
 *                    >= 0: this number in its place ("given counts", for
 *                    micro-batches of one mean); 0 gives loss and gradient 0.
 *                    A sum does not use it.
 *   clip_low         in [0, 1]; clip_high >= 0; both finite.
 *   dual_clip        0 = off, else > 1 and finite.
 *   kl_weight        finite; needs ref_logp unless 0. With 0 ref_logp goes into
 *                    the statistics alone.
 *   kl_kind          enum lmhead_kl_kind; reduction: enum lmhead_reduction.
 *   advantage_per_sequence  0: advantage [n]; 1: advantage [sequences] (needs
 *                    sequences).
 *   reserved         must be 0.
 */
typedef struct lmhead_policy_problem {
    int64_t n;
    int64_t sequences;
    int64_t num_valid;
    double clip_low;
    double clip_high;
    double dual_clip;
    double kl_weight;
    int32_t kl_kind;
    int32_t reduction;
    int32_t advantage_per_sequence;
    int32_t reserved;
} lmhead_policy_problem;

/* Bytes of workspace lmhead_policy_loss_fwd needs (0 for an invalid problem). */
size_t lmhead_policy_loss_workspace_size(const lmhead_policy_problem* p);

/*
 * Per token, with d = logp - old_logp and r = exp(d):
 *   rho = min(r, 1 + clip_high) for advantage A >= 0, max(r, 1 - clip_low) for
 *   A < 0, and there, with dual_clip, min(rho, dual_clip);
 *   L = -A rho + kl_weight KL(logp - ref_logp).
 * Where rho is a border the token is clipped and the first term has no
 * gradient; the border is decided in 64 bits on d. loss = sum of w L, with w = 1
 * / count, 1, or 1 / (sequences * the sequence's count).
 *   logp      device, fp32 [n] (lmhead_logprob's).
 *   old_logp  device, fp32 [n], or NULL: logp itself (r = 1, of an infinite logp
 *             too; NaN of NaN).
 *   ref_logp  device, fp32 [n], or NULL.
 *   loss      device, fp32 [1].
 *   stats     device, fp32 [4] or NULL: means over the counted tokens of the
 *             KL estimate, of being clipped, of r, and of exp(-d) - 1 + d.
 *   weights   device, fp32 [max(sequences, 1)]: each sequence's w, for the
 *             backward.
 *   workspace 256-byte aligned; the other pointers 4.
 */
int lmhead_policy_loss_fwd(const lmhead_policy_problem* p, const float* logp, const float* old_logp,
                           const float* ref_logp, const float* advantage, const int32_t* targets,
                           const int32_t* cu_seqlens, float* loss, float* stats, float* weights,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * dlogp = grad w (-A r [not clipped] + kl_weight KL'), 0 for a token that does
 * not count; without old_logp, r = 1 and the gradient of the ratio is -A.
 *   grad     device, fp32 [1]; weights: the forward's.
 *   dlogp    device, fp32 [n].
 */
int lmhead_policy_loss_bwd(const lmhead_policy_problem* p, const float* grad, const float* weights,
                           const float* logp, const float* old_logp, const float* ref_logp,
                           const float* advantage, const int32_t* targets, const int32_t* cu_seqlens,
                           float* dlogp, void* stream);

enum lmhead_preference_kind {
    LMHEAD_PREFERENCE_SIGMOID = 0, /* -(1 - e) log sigmoid(h) - e log sigmoid(-h), e = label_smoothing */
    LMHEAD_PREFERENCE_HINGE = 1,   /* max(0, 1 - h) */
    LMHEAD_PREFERENCE_SQUARED = 2  /* ((h - 1/2) / beta)^2 */
};

/*
 *   n          tokens, 0 <= n <= 2^30.
 *   pairs      1 <= pairs <= 2^23: sequence j < pairs is the chosen answer of
 *              pair j, sequence pairs + j the rejected one.
 *   num_pairs  -1: pairs; >= 0: the mean's denominator in its place; 0 gives
 *              loss and gradient 0.
 *   beta       positive and finite; margin: finite.
 *   label_smoothing  in [0, 1/2]; 0 unless sigmoid.
 *   kind       enum lmhead_preference_kind.
 *   average    0: s is the sum over a sequence's counted tokens; 1: the mean.
 */
typedef struct lmhead_preference_problem {
    int64_t n;
    int64_t pairs;
    int64_t num_pairs;
    double beta;
    double margin;
    double label_smoothing;
    int32_t kind;
    int32_t average;
} lmhead_preference_problem;

/* Bytes of workspace lmhead_preference_loss_fwd needs (0 for an invalid problem). */
size_t lmhead_preference_loss_workspace_size(const lmhead_preference_problem* p);

/*
 * s = sum (or mean) over a sequence's counted tokens of logp - ref_logp (0
 * where none counts), in 64 bits; h = beta (s_chosen - s_rejected) - margin;
 * loss = mean over pairs of the kind's function of h.
 *   logp, ref_logp  device, fp32 [n]; ref_logp may be NULL (0).
 *   cu_seqlens      device, int32 [2 pairs + 1].
 *   loss            device, fp32 [1].
 *   rewards         device, fp32 [2 pairs] or NULL: beta s.
 *   coef            device, fp32 [2 pairs]: what a counted token's logp changes
 *                   the loss by, for the backward.
 *   workspace       256-byte aligned; the other pointers 4.
 */
int lmhead_preference_loss_fwd(const lmhead_preference_problem* p, const float* logp, const float* ref_logp,
                               const int32_t* targets, const int32_t* cu_seqlens, float* loss,
                               float* rewards, float* coef, void* workspace, size_t workspace_bytes,
                               void* stream);

/* dlogp[i] = grad coef[the token's sequence], 0 for a token that does not
 * count. Of p only n and pairs matter. grad: device, fp32 [1]. */
int lmhead_preference_loss_bwd(const lmhead_preference_problem* p, const float* grad, const float* coef,
                               const int32_t* targets, const int32_t* cu_seqlens, float* dlogp,
                               void* stream);

/* ---------------------------------------------------------------- AdamW */

/*
 * One tensor of the step (host memory; the pointers are device's). Elements
 * are taken in the order of memory.
 *   param, grad      param_dtype, grad_dtype (enum lmhead_dtype) [numel].
 *   exp_avg, exp_avg_sq  state_dtype [numel]: fp32 m and v; or e4m3, m and
 *                    sqrt(v) over their scales.
 *   exp_avg_scale, exp_avg_sq_scale  fp32 [ceil(numel / 128)] with e4m3, else
 *                    NULL.
 *   copy             bf16 [numel] or NULL: the updated parameter rounded (for
 *                    fp32 parameters that a bf16 model is run from).
 * Each aligned to its element; tensors whose parameter, gradient and fp32
 * states are 16-byte aligned (e4m3: 8) take wide loads. No buffer may overlap
 * another one of the call.
 */
typedef struct lmhead_adamw_tensor {
    void* param;
    const void* grad;
    void* exp_avg;
    void* exp_avg_sq;
    float* exp_avg_scale;
    float* exp_avg_sq_scale;
    void* copy;
    int64_t numel;
    int32_t param_dtype;
    int32_t grad_dtype;
    int32_t state_dtype;
    int32_t reserved;
} lmhead_adamw_tensor;

/*
 *   lr             finite; weight_decay: finite, >= 0.
 *   beta1, beta2   in [0, 1); eps: finite, >= 2^-126.
 *   step           1 for the first step; 1 <= step.
 *   device_step    device, int32 [1] or NULL: the step instead of `step` (a
 *                  captured graph reads it at each replay). Below 1 it counts
 *                  as 1.
 *   device_lr      device, fp32 [1] or NULL: the learning rate instead of `lr`.
 *   grad_scale     device, fp32 [1] or NULL: multiplies every gradient (a
 *                  clipping coefficient, or 1 / loss scale).
 *   stochastic     0: 8-bit states round to nearest even; 1: up or down at
 *                  random, in proportion to the distance, from seed, the step,
 *                  the tensor's place in the call and the element (the same ones
 *                  give the same bits). To nearest, a value that moves by less
 *                  than half of its code's step (2^-4 of it) at a time holds
 *                  still until its block's scale has moved: with beta2 near 1
 *                  sqrt(v) falls late or not at all where gradients get smaller
 *                  (medians of 1.15 times the fp32 state's were measured), and so
 *                  does m with beta1 of 0.94 or more. At random it follows on average.
 */
typedef struct lmhead_adamw {
    double lr;
    double beta1;
    double beta2;
    double eps;
    double weight_decay;
    int64_t step;
    const int32_t* device_step;
    const float* device_lr;
    const float* grad_scale;
    int32_t stochastic;
    uint32_t seed;
} lmhead_adamw;

/*
 * With g = grad_scale grad and t = step, in fp32:
 *   m' = beta1 m + (1 - beta1) g;  v' = beta2 v + (1 - beta2) g^2;
 *   param' = param (1 - lr weight_decay)
 *            - lr / (1 - beta1^t) * m' / (sqrt(v') / sqrt(1 - beta2^t) + eps).
 * The parameter is updated from the fp32 m' and v'; states in 8 bits are
 * rounded after that, over blocks of 128 consecutive elements of a tensor as
 * lmhead_quantize_fp8 rounds (the scale is the largest magnitude times 1 / 448 in
 * fp32, and every operation on the way to a code is rounded by itself, so that
 * elementwise fp32 programs get the same codes), except that a sqrt(v') > 0 becomes
 * no zero (at least 2^-9 of its scale): a vanishing denominator would let m' loose.
 * States of zeros start (any finite scales).
 * Stochastic: with y = value / scale and u the upper 16 of 20 random bits, as a
 * fraction, |y| + u step(y) is cut to the code below, step(y) being the distance
 * of the codes around y.
 *   tensors  host, [count]; count 0 .. 2^20. numel 0 .. 2^35 - 2^24.
 *   table    device, 8-byte aligned, or NULL: what lmhead_adamw_table wrote for
 *            these tensors, copied there. With it any number of tensors shares one
 *            launch (up to 16,777,215 workgroups of 2048 elements, or 4096 in 8
 *            bits), without it 48 do; 48 or fewer need none. Bits do not differ.
 */
int lmhead_adamw_step(const lmhead_adamw* p, const lmhead_adamw_tensor* tensors, int64_t count, const void* table,
                      void* stream);

/* Bytes of a table of count tensors (0 for a count out of range), and the table
 * itself, written to host memory (8-byte aligned). Pure host functions. A table
 * holds the tensors' addresses: other addresses need another table. A shape
 * error where the tensors are too large for one launch. */
size_t lmhead_adamw_table_size(int64_t count);
int lmhead_adamw_table(const lmhead_adamw_tensor* tensors, int64_t count, void* table, size_t table_bytes);

#ifdef __cplusplus
}
#endif

#endif /* LMHEAD_TRAIN_H */
