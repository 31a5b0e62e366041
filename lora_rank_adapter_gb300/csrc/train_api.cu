// train_api.cu -- the extern "C" entry points of include/lora_train.h: argument
// validation, workspace sizes, and dispatch to the loss and optimizer kernels.
#include <cuda_runtime.h>
#include <math.h>

#include "adamw.h"
#include "host_common.h"
#include "loss.h"

namespace lora {
namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxVocab = (int64_t)1 << 30;      // places within a row are 32-bit ints in the kernels

bool size_ok(int64_t v) { return v >= 0 && v < kMaxDim; }
bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A pointer that the call reads or writes n elements of e bytes through.
lora_status_t check_ptr(const void *p, int64_t n, int e) {
  if (n == 0) return LORA_OK;
  if (p == nullptr) return LORA_ERR_INVALID_ARG;
  return aligned(p, e) ? LORA_OK : LORA_ERR_ALIGNMENT;
}
lora_status_t check_opt(const void *p, int e) { return aligned(p, e) ? LORA_OK : LORA_ERR_ALIGNMENT; }

lora_status_t check_ws(const void *ws, size_t ws_bytes, size_t need) {
  if (need == 0) return LORA_OK;
  if (ws == nullptr || !aligned(ws, 256) || ws_bytes < need) return LORA_ERR_WORKSPACE;
  return LORA_OK;
}

lora_status_t check_rows(lora_dtype_t dtype, int64_t T, int64_t V, const void *logits, int64_t ldl,
                         const int64_t *labels, float temperature, const void *dlogits, int64_t lddl) {
  if (dtype != LORA_F32 && dtype != LORA_BF16) return LORA_ERR_UNSUPPORTED;
  if (!size_ok(T) || !size_ok(V)) return LORA_ERR_INVALID_ARG;
  if (V > kMaxVocab) return LORA_ERR_UNSUPPORTED;
  // the kernels scale by log2(e) / temperature
  if (!(temperature > 0.f) || !isfinite(temperature) || !isfinite(1.f / temperature * 1.4426950408889634f))
    return LORA_ERR_INVALID_ARG;
  const int e = dtype == LORA_BF16 ? 2 : 4;
  if (T > 0 && V > 0) {
    if (ldl < V) return LORA_ERR_INVALID_ARG;
    if (dlogits != nullptr && lddl < V) return LORA_ERR_INVALID_ARG;
    LORA_TRY(check_ptr(logits, 1, e));
    LORA_TRY(check_opt(dlogits, e));
    if (dlogits == logits && lddl != ldl) return LORA_ERR_INVALID_ARG;
  }
  return check_ptr(labels, T, 8);
}

LossArgs loss_args(lora_dtype_t dtype, int64_t T, int64_t V, const void *logits, int64_t ldl, const int64_t *labels,
                   float temperature, float *logps, void *dlogits, int64_t lddl, float grad_scale) {
  LossArgs a;
  a.dtype = dtype; a.T = T; a.V = V; a.logits = logits; a.ldl = ldl; a.labels = labels; a.temperature = temperature;
  a.logps = logps; a.dlogits = dlogits; a.lddl = lddl; a.grad_scale = grad_scale;
  return a;
}

bool flags_ok(uint32_t flags) {
  if (flags & ~(LORA_ADAMW_STATE_8BIT | LORA_ADAMW_MASTER | LORA_ADAMW_STOCHASTIC)) return false;
  return !(flags & LORA_ADAMW_STOCHASTIC) || (flags & LORA_ADAMW_STATE_8BIT);
}

lora_status_t check_plan(const lora_adamw_plan_t *plan) {
  if (plan == nullptr || plan->chunks < 0 || plan->chunks >= kMaxDim) return LORA_ERR_INVALID_ARG;
  if (plan->table == nullptr || !aligned(plan->table, 256)) return LORA_ERR_INVALID_ARG;
  if ((plan->param_dtype != LORA_F32 && plan->param_dtype != LORA_BF16) ||
      (plan->grad_dtype != LORA_F32 && plan->grad_dtype != LORA_BF16))
    return LORA_ERR_UNSUPPORTED;
  return flags_ok(plan->flags) ? LORA_OK : LORA_ERR_INVALID_ARG;
}

// Chunks of the tensors, or -1 if a size is out of range.
int64_t count_chunks(const lora_adamw_tensor_t *tensors, int32_t n) {
  if (n < 0 || (n > 0 && tensors == nullptr)) return -1;
  int64_t chunks = 0;
  for (int32_t i = 0; i < n; ++i) {
    const int64_t k = tensors[i].numel;
    if (k < 0 || k > kMaxDim * LORA_ADAMW_CHUNK) return -1;
    chunks += ceil_div(k, LORA_ADAMW_CHUNK);
    if (chunks >= kMaxDim) return -1;
  }
  return chunks;
}

// Nothing is thrown across the C boundary: the launch helpers keep small tables
// that may have to allocate.
template <typename F>
lora_status_t guarded(F &&f) {
  try {
    return f();
  } catch (...) {
    return LORA_ERR_CUDA;
  }
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

size_t lora_train_workspace_size(lora_train_op_t op, int64_t n, int64_t m) {
  if (!size_ok(n) || m < 0 || m > 4 * kMaxVocab) return 0;
  switch (op) {
    case LORA_TRAIN_PREFERENCE_LOSS: return size_ok(m) ? preference_ws_bytes(n, m) : 0;
    case LORA_TRAIN_POLICY_LOSS: return policy_ws_bytes(n, m == 0 ? 4 * kMaxVocab : m, true);
  }
  return 0;
}

lora_status_t lora_token_logps(lora_dtype_t dtype, int64_t T, int64_t V, const void *logits, int64_t ldl,
                               const int64_t *labels, float temperature, float *logps, float *stats, void *stream) {
  LORA_TRY(check_rows(dtype, T, V, logits, ldl, labels, temperature, nullptr, 0));
  LORA_TRY(check_ptr(logps, T, 4));
  LORA_TRY(check_opt(stats, 8));
  return guarded([&] {
    return token_logps(loss_args(dtype, T, V, logits, ldl, labels, temperature, logps, nullptr, 0, 1.f), stats,
                       (cudaStream_t)stream);
  });
}

lora_status_t lora_token_logps_backward(lora_dtype_t dtype, int64_t T, int64_t V, const void *logits, int64_t ldl,
                                        const int64_t *labels, float temperature, const float *stats,
                                        const float *dlogps, void *dlogits, int64_t lddl, void *stream) {
  LORA_TRY(check_rows(dtype, T, V, logits, ldl, labels, temperature, dlogits, lddl));
  LORA_TRY(check_ptr(dlogits, T * V, 1));
  LORA_TRY(check_ptr(stats, T, 8));
  LORA_TRY(check_ptr(dlogps, T, 4));
  return guarded([&] {
    return token_logps_backward(loss_args(dtype, T, V, logits, ldl, labels, temperature, nullptr, dlogits, lddl, 1.f),
                                stats, dlogps, (cudaStream_t)stream);
  });
}

lora_status_t lora_preference_loss(lora_dtype_t dtype, int64_t T, int64_t V, int32_t P, const void *logits,
                                   int64_t ldl, const int64_t *labels, const int32_t *cu_seqlens,
                                   const float *ref_logps, lora_pref_kind_t kind, float beta, float label_smoothing,
                                   uint32_t flags, float temperature, float *token_logps, float *seq_logps,
                                   float *pair_loss, float *loss, void *dlogits, int64_t lddl, float grad_scale,
                                   void *ws, size_t ws_bytes, void *stream) {
  LORA_TRY(check_rows(dtype, T, V, logits, ldl, labels, temperature, dlogits, lddl));
  if (P < 0 || P >= (1 << 30)) return LORA_ERR_INVALID_ARG;
  if (kind != LORA_PREF_SIGMOID && kind != LORA_PREF_HINGE && kind != LORA_PREF_IPO) return LORA_ERR_UNSUPPORTED;
  if (!(beta > 0.f) || !isfinite(beta) || !isfinite(grad_scale)) return LORA_ERR_INVALID_ARG;
  if (!(label_smoothing >= 0.f && label_smoothing <= 1.f)) return LORA_ERR_INVALID_ARG;
  if (flags & ~LORA_PREF_LENGTH_NORMALIZE) return LORA_ERR_INVALID_ARG;
  LORA_TRY(check_ptr(cu_seqlens, P, 4));
  LORA_TRY(check_opt(ref_logps, 4));
  LORA_TRY(check_ptr(token_logps, T, 4));
  LORA_TRY(check_ptr(seq_logps, P, 4));
  LORA_TRY(check_ptr(pair_loss, P, 4));
  LORA_TRY(check_ptr(loss, 1, 4));
  LORA_TRY(check_ws(ws, ws_bytes, preference_ws_bytes(T, P)));
  PreferenceArgs p;
  p.P = P; p.cu = cu_seqlens; p.ref = ref_logps; p.kind = kind; p.beta = beta; p.smoothing = label_smoothing;
  p.normalize = (flags & LORA_PREF_LENGTH_NORMALIZE) != 0;
  p.seq_logps = seq_logps; p.pair_loss = pair_loss; p.loss = loss;
  return guarded([&] {
    return preference_loss(loss_args(dtype, T, V, logits, ldl, labels, temperature, token_logps, dlogits, lddl,
                                     grad_scale), p, ws, ws_bytes, (cudaStream_t)stream);
  });
}

lora_status_t lora_policy_loss(lora_dtype_t dtype, int64_t T, int64_t V, const void *logits, int64_t ldl,
                               const int64_t *labels, const float *old_logps, const float *ref_logps,
                               const float *advantages, const float *weights, float clip_low, float clip_high,
                               float kl_beta, float temperature, float *token_logps, float *metrics, void *dlogits,
                               int64_t lddl, float grad_scale, void *ws, size_t ws_bytes, void *stream) {
  LORA_TRY(check_rows(dtype, T, V, logits, ldl, labels, temperature, dlogits, lddl));
  if (!(clip_low >= 0.f && clip_low <= 1.f) || !(clip_high >= 0.f) || !isfinite(clip_high) || !(kl_beta >= 0.f) ||
      !isfinite(kl_beta) || !isfinite(grad_scale))
    return LORA_ERR_INVALID_ARG;
  LORA_TRY(check_opt(old_logps, 4));
  LORA_TRY(check_opt(ref_logps, 4));
  LORA_TRY(check_opt(weights, 4));
  LORA_TRY(check_ptr(advantages, T, 4));
  LORA_TRY(check_ptr(token_logps, T, 4));
  LORA_TRY(check_ptr(metrics, 1, 4));
  // the metrics take these values once more, after the log-probabilities have been written
  for (const float *in : {old_logps, ref_logps, advantages, weights})
    if (T > 0 && token_logps == in) return LORA_ERR_INVALID_ARG;
  LORA_TRY(check_ws(ws, ws_bytes, policy_ws_bytes(T, V * (dtype == LORA_BF16 ? 2 : 4), dlogits != nullptr)));
  PolicyArgs p;
  p.old_logps = old_logps; p.ref_logps = ref_logps; p.advantages = advantages; p.weights = weights;
  p.clip_low = clip_low; p.clip_high = clip_high; p.kl_beta = kl_beta; p.metrics = metrics;
  return guarded([&] {
    return policy_loss(loss_args(dtype, T, V, logits, ldl, labels, temperature, token_logps, dlogits, lddl,
                                 grad_scale), p, ws, ws_bytes, (cudaStream_t)stream);
  });
}

lora_status_t lora_scale_gradient(lora_dtype_t dtype, int64_t T, int64_t V, void *x, int64_t ldx,
                                  const float *factor, void *stream) {
  if (dtype != LORA_F32 && dtype != LORA_BF16) return LORA_ERR_UNSUPPORTED;
  if (!size_ok(T) || !size_ok(V)) return LORA_ERR_INVALID_ARG;
  if (V > kMaxVocab) return LORA_ERR_UNSUPPORTED;
  if (T == 0 || V == 0) return LORA_OK;
  if (ldx < V) return LORA_ERR_INVALID_ARG;
  LORA_TRY(check_ptr(x, 1, dtype == LORA_BF16 ? 2 : 4));
  LORA_TRY(check_ptr(factor, 1, 4));
  return guarded([&] { return scale_gradient(dtype, T, V, x, ldx, factor, (cudaStream_t)stream); });
}

size_t lora_adamw_table_size(const lora_adamw_tensor_t *tensors, int32_t n) {
  const int64_t chunks = count_chunks(tensors, n);
  return chunks < 0 ? 0 : table_bytes(chunks);
}

lora_status_t lora_adamw_build(const lora_adamw_tensor_t *tensors, int32_t n, lora_dtype_t param_dtype,
                               lora_dtype_t grad_dtype, uint32_t flags, void *table, size_t bytes,
                               lora_adamw_plan_t *plan, void *stream) {
  if (plan == nullptr) return LORA_ERR_INVALID_ARG;
  const int64_t chunks = count_chunks(tensors, n);
  if (chunks < 0) return LORA_ERR_INVALID_ARG;
  lora_adamw_plan_t made = {table, chunks, (int32_t)param_dtype, (int32_t)grad_dtype, flags, 0};
  if ((param_dtype != LORA_F32 && param_dtype != LORA_BF16) || (grad_dtype != LORA_F32 && grad_dtype != LORA_BF16))
    return LORA_ERR_UNSUPPORTED;
  if (!flags_ok(flags)) return LORA_ERR_INVALID_ARG;
  const bool s8 = (flags & LORA_ADAMW_STATE_8BIT) != 0;
  for (int32_t i = 0; i < n; ++i) {
    const lora_adamw_tensor_t &t = tensors[i];
    LORA_TRY(check_ptr(t.param, t.numel, param_dtype == LORA_BF16 ? 2 : 4));
    LORA_TRY(check_ptr(t.grad, t.numel, grad_dtype == LORA_BF16 ? 2 : 4));
    LORA_TRY(check_ptr(t.exp_avg, t.numel, s8 ? 1 : 4));
    LORA_TRY(check_ptr(t.exp_avg_sq, t.numel, s8 ? 1 : 4));
    if (s8) {
      LORA_TRY(check_ptr(t.exp_avg_scale, t.numel, 4));
      LORA_TRY(check_ptr(t.exp_avg_sq_scale, t.numel, 4));
    }
    if (flags & LORA_ADAMW_MASTER) LORA_TRY(check_ptr(t.master, t.numel, 4));
  }
  LORA_TRY(check_ws(table, bytes, table_bytes(chunks)));
  LORA_TRY(guarded([&] {
    return adamw_build(tensors, n, made, static_cast<AdamChunk *>(table), (cudaStream_t)stream);
  }));
  *plan = made;
  return LORA_OK;
}

lora_status_t lora_grad_norm(const lora_adamw_plan_t *plan, float max_norm, float *out, void *stream) {
  LORA_TRY(check_plan(plan));
  if (!(max_norm >= 0.f)) return LORA_ERR_INVALID_ARG;
  LORA_TRY(check_ptr(out, 1, 4));
  return guarded([&] { return grad_norm(*plan, max_norm, out, (cudaStream_t)stream); });
}

lora_status_t lora_adamw(const lora_adamw_plan_t *plan, const lora_adamw_hyper_t *h, const float *grad_factor,
                         void *stream) {
  LORA_TRY(check_plan(plan));
  if (h == nullptr || h->step < 1) return LORA_ERR_INVALID_ARG;
  auto ok = [](double v) { return v >= 0.0 && isfinite(v); };
  if (!ok(h->lr) || !ok(h->eps) || !ok(h->weight_decay) || !ok(h->beta1) || !ok(h->beta2) || h->beta1 >= 1.0 ||
      h->beta2 >= 1.0)
    return LORA_ERR_INVALID_ARG;
  LORA_TRY(check_opt(grad_factor, 4));
  return guarded([&] { return adamw(*plan, *h, grad_factor, (cudaStream_t)stream); });
}

}  // extern "C"
