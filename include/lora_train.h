/*
 * lora_train.h -- C ABI of liblora.so, training operators around the adapter
 * product of lora.h: what lies between a model's logits and the next value of
 * the adapters' A and B.
 *
 *   lora_token_logps, lora_token_logps_backward   log-probabilities of the labels, and their gradient
 *   lora_preference_loss                          paired log-ratio loss, and its gradient
 *   lora_policy_loss                              clipped policy loss with a KL term, and its gradient
 *   lora_scale_gradient                           a gradient times a device scalar, in place
 *   lora_adamw_build, lora_grad_norm, lora_adamw  an AdamW step over many tensors at once
 *
 * The conventions of lora.h hold: device pointers owned by the caller, scratch
 * passed in as ws (256-byte aligned), strides in elements, work enqueued on
 * `stream` (of the current device) without a host sync, host-checkable errors
 * returned before anything is launched, results independent of the run (no float
 * atomics).  Logits rows need only the alignment of their element type: any row
 * stride, any V.
 *
 * The loss operators work on T rows of logits, element (t, v) at
 * logits[t*ldl + v], LORA_BF16 or LORA_F32, 0 <= T < 2^31, 0 <= V <= 2^30
 * (above: LORA_ERR_UNSUPPORTED), ldl >= V, and on labels[t] (int64): row t scores
 * label labels[t].  (A causal model's caller
 * passes the labels already moved by one.)  A label outside [0, V) marks an
 * IGNORED row: it contributes nothing, its log-probability and its gradient are
 * zero, and its logits are not read (they may hold anything, NaN included).
 * Softmax statistics and sums are held in 32 bits or more; a gradient stored in
 * bf16 is rounded once, to nearest even (lora_scale_gradient rounds it again).  Logits of minus infinity or of the
 * type's lowest value have probability zero as long as the row has a larger
 * one; a NaN, a plus infinity or a row of nothing but minus infinity gives NaN
 * in that row, as the formula does.
 *
 * `temperature` (finite, > 0, log2(e) / temperature finite in fp32) divides the
 * logits: z = logits / temperature.
 * `dlogits`, where an operator takes it, is written whole (every row, V
 * columns); it is either `logits` itself (same pointer, same stride: the
 * gradient replaces the logits) or shares no element with them.
 */
#ifndef LORA_TRAIN_H_
#define LORA_TRAIN_H_

#include "lora.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of workspace of the operators below (0: none, or arguments out of range).
 *   LORA_TRAIN_PREFERENCE_LOSS  (T, P)
 *   LORA_TRAIN_POLICY_LOSS      (T, bytes of a row of logits; 0: a bound for any) */
typedef enum {
    LORA_TRAIN_PREFERENCE_LOSS = 0,
    LORA_TRAIN_POLICY_LOSS = 1
} lora_train_op_t;
LORA_API size_t lora_train_workspace_size(lora_train_op_t op, int64_t n, int64_t m);

/* --------------------------------------------------------------------------------
 * lora_token_logps:  logps[t] = z[t][label] - ln sum_v exp(z[t][v])
 *   logps  float [T] (0 for an ignored row)
 *   stats  NULL, or float [T][2]: the row's largest logit and the sum of
 *          exp(z - largest z), for lora_token_logps_backward (8-byte aligned).
 * -------------------------------------------------------------------------------- */
LORA_API lora_status_t lora_token_logps(lora_dtype_t dtype, int64_t T, int64_t V, const void *logits, int64_t ldl,
                           const int64_t *labels, float temperature, float *logps, float *stats, void *stream);

/* --------------------------------------------------------------------------------
 * lora_token_logps_backward:
 *   dlogits[t][v] = dlogps[t] / temperature * ((v == label) - exp(z[t][v]) / sum_u exp(z[t][u]))
 *   stats   float [T][2] as lora_token_logps wrote them for the same logits,
 *           labels and temperature;  dlogps  float [T].
 * A row that is ignored, or whose dlogps is zero, gets zeros and is not read.
 * -------------------------------------------------------------------------------- */
LORA_API lora_status_t lora_token_logps_backward(lora_dtype_t dtype, int64_t T, int64_t V, const void *logits,
                           int64_t ldl, const int64_t *labels, float temperature, const float *stats,
                           const float *dlogps, void *dlogits, int64_t lddl, void *stream);

/* --------------------------------------------------------------------------------
 * lora_preference_loss: P pairs of packed sequences.  Sequence i (0 <= i < 2P)
 * holds the rows cu_seqlens[i] .. cu_seqlens[i+1]; pair p prefers sequence p
 * (chosen) to sequence P + p (rejected).  S_i is the sum of the sequence's
 * token log-probabilities (ignored rows count nothing), divided by the number
 * of rows that count if LORA_PREF_LENGTH_NORMALIZE is set; R_i = ref_logps[i] is
 * the same of the reference model (with an adapter off: one lora_preference_loss
 * call without dlogits on its logits gives seq_logps).
 *     d = (S_p - S_{P+p}) - (R_p - R_{P+p})
 *     LORA_PREF_SIGMOID  -(1 - label_smoothing) ln sigmoid(beta d) - label_smoothing ln sigmoid(-beta d)
 *     LORA_PREF_HINGE    max(0, 1 - beta d)
 *     LORA_PREF_IPO      (d - 1 / (2 beta))^2
 *     loss = mean over the pairs (0 for P = 0)
 *   cu_seqlens  device int32 [2P + 1], ascending; values are clamped to [0, T].
 *               A sequence may be empty (S = 0).  Rows in no sequence have a
 *               log-probability and no gradient.
 *   ref_logps   device float [2P], or NULL for R = 0.
 *   token_logps float [T];  seq_logps float [2P];  pair_loss float [P];  loss float [1]
 *   dlogits     NULL, or grad_scale * d loss / d logits
 *   beta        finite, > 0;  label_smoothing in [0, 1], used by LORA_PREF_SIGMOID alone
 *   ws          lora_train_workspace_size(LORA_TRAIN_PREFERENCE_LOSS, T, P) bytes
 * -------------------------------------------------------------------------------- */
typedef enum { LORA_PREF_SIGMOID = 0, LORA_PREF_HINGE = 1, LORA_PREF_IPO = 2 } lora_pref_kind_t;
#define LORA_PREF_LENGTH_NORMALIZE 1u
LORA_API lora_status_t lora_preference_loss(lora_dtype_t dtype, int64_t T, int64_t V, int32_t P, const void *logits,
                           int64_t ldl, const int64_t *labels, const int32_t *cu_seqlens, const float *ref_logps,
                           lora_pref_kind_t kind, float beta, float label_smoothing, uint32_t flags,
                           float temperature, float *token_logps, float *seq_logps, float *pair_loss, float *loss,
                           void *dlogits, int64_t lddl, float grad_scale, void *ws, size_t ws_bytes, void *stream);

/* --------------------------------------------------------------------------------
 * lora_policy_loss: with logp the row's token log-probability, over the rows that count
 *     r  = exp(logp - old_logps)         (old_logps NULL: r = 1, its gradient that of logp)
 *     pg = -min(r * A, clip(r, 1 - clip_low, 1 + clip_high) * A)
 *     kl = exp(d) - d - 1, d = ref_logps - logp        (ref_logps NULL: 0)
 *     loss = sum_t weights[t] * (pg + kl_beta * kl)
 * with the gradient  d loss / d logp = weights * (clipped ? 0 : -A r) + weights * kl_beta * (1 - exp(d)),
 * where a row is clipped when A > 0 and r > 1 + clip_high, or A < 0 and r < 1 - clip_low.
 *   old_logps, ref_logps  device float [T] or NULL;  advantages  device float [T]
 *   weights     device float [T] or NULL for 1: the caller's mean (1 / number of
 *               rows that count, 1 / (sequences * rows of the sequence), ...)
 *   token_logps float [T], none of the inputs;  metrics float [3]: the loss,
 *               sum weights * kl, and sum of weights over the clipped rows
 *   dlogits     NULL, or grad_scale * d loss / d logits
 *   clip_low in [0, 1], clip_high >= 0, kl_beta >= 0, all finite
 *   ws          lora_train_workspace_size(LORA_TRAIN_POLICY_LOSS, T, row bytes) bytes:
 *               none for rows up to 768 KB, or without dlogits
 * -------------------------------------------------------------------------------- */
LORA_API lora_status_t lora_policy_loss(lora_dtype_t dtype, int64_t T, int64_t V, const void *logits, int64_t ldl,
                           const int64_t *labels, const float *old_logps, const float *ref_logps,
                           const float *advantages, const float *weights, float clip_low, float clip_high,
                           float kl_beta, float temperature, float *token_logps, float *metrics, void *dlogits,
                           int64_t lddl, float grad_scale, void *ws, size_t ws_bytes, void *stream);

/* --------------------------------------------------------------------------------
 * lora_scale_gradient:  x[t][v] *= *factor (device float), rounded once.  Returns
 * to the stream at once when *factor is 1: the gradient that a loss operator
 * wrote ahead of time then needs no second pass.  Otherwise a bf16 gradient has
 * been rounded twice (exactly, once, where the factor is a power of two); grad_scale
 * of the loss operators scales before the one rounding.
 * -------------------------------------------------------------------------------- */
LORA_API lora_status_t lora_scale_gradient(lora_dtype_t dtype, int64_t T, int64_t V, void *x, int64_t ldx,
                           const float *factor, void *stream);

/* --------------------------------------------------------------------------------
 * AdamW over many tensors.  lora_adamw_build lays the tensors' addresses out
 * once in a caller's device buffer (the table), in chunks of
 * LORA_ADAMW_CHUNK elements of one tensor; lora_grad_norm and lora_adamw then
 * run over all tensors in one launch each.  The caller rebuilds the table when an
 * address changes, keeps the tensors alive while it is in use, and lets calls on
 * one table run one after the other (the table holds the norm's partial sums).
 * Tensors share no memory with each other: their chunks are worked on at once.
 *
 * Element i of tensor k, all in 32-bit arithmetic (g is read in its own type):
 *     g' = g * *grad_factor
 *     m  = beta1 m + (1 - beta1) g'
 *     v  = beta2 v + (1 - beta2) g'^2
 *     p  = p (1 - lr weight_decay) - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * With `master` the update is taken on master[i] (float) and p is its rounding.
 * The quotient is off by some 2^-22; a divisor below the smallest normal number
 * (eps = 0 and v = 0) counts as that number, so that 0 / 0 gives 0.
 *
 * States in 32 bits: exp_avg (m) and exp_avg_sq (v) are float [numel].
 * States in 8 bits (LORA_ADAMW_STATE_8BIT): blocks of LORA_ADAMW_BLOCK
 * consecutive elements (the last one of a tensor may be short) share a float
 * scale.  exp_avg holds m and exp_avg_sq holds u = sqrt(v) as e4m3 codes:
 *     a = max(max |m|, 1e-30) over the block, code = e4m3(m * (448 / a)), scale = a * (1 / 448)
 * rounded to nearest even, m = code * scale; likewise u, except that a positive
 * u never rounds to zero (it gets the smallest code: with m kept and u lost the
 * next step would be huge).  p's update uses m and u before they are rounded.
 * The states follow IEEE single rounding step by step in the order written, so
 * equal inputs give equal codes everywhere.
 *   Rounding to nearest keeps a state for a few steps, not for thousands: e4m3
 * values lie 6 to 12 % apart, a step with beta2 = 0.999 lowers u by 0.05 % at most,
 * so codes stay where they are relative to the block's largest one, and each u
 * follows that element instead of its own gradients (one outlier in a block leaves
 * the others' u at 0.3 of their value, steps three times too large, for thousands
 * of steps).  LORA_ADAMW_STOCHASTIC rounds both states at random instead, up with
 * the probability of how far up a value is, so that each follows its gradients on
 * average (u then scatters by some 17 % about its value).  The random bits are a
 * function of the step, the chunk's number in the table and the element's place in
 * the chunk, so a step is reproducible all the same:
 *     mix(x): x ^= x >> 16; x *= A; x ^= x >> 15; x *= B; x ^= x >> 16; x *= A; x ^= x >> 15
 *     x = (mix(mix(step + mix(step >> 32)) + chunk) + place) * A; x ^= x >> 15; x *= B; x ^= x >> 16
 * in 32 bits, A = 0x9E3779B9, B = 0xBB67AE85; m takes the low 16 bits of x, u the
 * high ones, and q = value * (448 / a) goes up when its distance from the value
 * below, in 2^-20 of the distance between the two (below 2^-6 on q + 2^-6 rounded to
 * fp32), and 16 * bits + 8 add up to 2^20 or more.
 *   p, g    dtype param_dtype / grad_dtype of the plan, contiguous [numel]
 *   codes   uint8 (e4m3) [numel];  scales  float [ceil(numel / LORA_ADAMW_BLOCK)]
 * Elements need only the alignment of their type; tensors whose pointers are all
 * 16-byte aligned take wide loads (codes: 4-byte).
 * -------------------------------------------------------------------------------- */
#define LORA_ADAMW_BLOCK 256
#define LORA_ADAMW_CHUNK 2048
#define LORA_ADAMW_STATE_8BIT 1u
#define LORA_ADAMW_MASTER 2u
#define LORA_ADAMW_STOCHASTIC 16u      /* with LORA_ADAMW_STATE_8BIT only */

typedef struct {
    void *param;
    const void *grad;
    void *exp_avg;
    void *exp_avg_sq;
    float *exp_avg_scale;      /* 8-bit states only, else ignored */
    float *exp_avg_sq_scale;
    float *master;             /* LORA_ADAMW_MASTER only, else ignored */
    int64_t numel;
} lora_adamw_tensor_t;

/* What the calls below need to know of a table; filled by lora_adamw_build. */
typedef struct {
    const void *table;         /* device */
    int64_t chunks;
    int32_t param_dtype;       /* lora_dtype_t */
    int32_t grad_dtype;
    uint32_t flags;
    uint32_t reserved;
} lora_adamw_plan_t;

/* Bytes of the table of n tensors (0 if an argument is out of range). */
LORA_API size_t lora_adamw_table_size(const lora_adamw_tensor_t *tensors, int32_t n);

/* Writes the table (256-byte aligned device buffer of lora_adamw_table_size() bytes)
 * and *plan.  `tensors` is a HOST array, read before the call returns; tensors of
 * zero elements are skipped.  Errors: NULL or misaligned pointers of a tensor with
 * elements -> LORA_ERR_INVALID_ARG / LORA_ERR_ALIGNMENT, a bad dtype or flag ->
 * LORA_ERR_UNSUPPORTED / LORA_ERR_INVALID_ARG, the buffer -> LORA_ERR_WORKSPACE. */
LORA_API lora_status_t lora_adamw_build(const lora_adamw_tensor_t *tensors, int32_t n, lora_dtype_t param_dtype,
                           lora_dtype_t grad_dtype, uint32_t flags, void *table, size_t table_bytes,
                           lora_adamw_plan_t *plan, void *stream);

/* out[0] = sqrt(sum of all g^2), out[1] = min(1, max_norm / (out[0] + 1e-6)); out is
 * device float [2], max_norm >= 0. */
LORA_API lora_status_t lora_grad_norm(const lora_adamw_plan_t *plan, float max_norm, float *out, void *stream);

/* One step.  step >= 1 counts this step; grad_factor: device float [1], or NULL for 1.
 * lr, weight_decay, eps >= 0 and beta1, beta2 in [0, 1), all finite.  These are host
 * values: a step captured in a graph replays the same count, rate and random bits. */
typedef struct {
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;
} lora_adamw_hyper_t;
LORA_API lora_status_t lora_adamw(const lora_adamw_plan_t *plan, const lora_adamw_hyper_t *hyper,
                           const float *grad_factor, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_TRAIN_H_ */
