// loss.h -- internal interface of the loss operators (loss.cu): log-probabilities
// of labels, preference loss and policy loss, with their gradients.
#pragma once

#include "../../include/lora_train.h"
#include "host_common.h"

namespace lora {

// Rows of logits and what is asked of them.
struct LossArgs {
  lora_dtype_t dtype;
  int64_t T, V;
  const void *logits;
  int64_t ldl;
  const int64_t *labels;
  float temperature;
  float *logps;           // [T]
  void *dlogits;          // NULL: no gradient
  int64_t lddl;
  float grad_scale;
};

struct PreferenceArgs {
  int32_t P;
  const int32_t *cu;      // [2P + 1]
  const float *ref;       // [2P] or NULL
  int kind;
  float beta, smoothing;
  int normalize;
  float *seq_logps, *pair_loss, *loss;
};

struct PolicyArgs {
  const float *old_logps, *ref_logps, *advantages, *weights;
  float clip_low, clip_high, kl_beta;
  float *metrics;         // [3]
};

// Reads and clears the error word of the waits in loss.cu (-1: the read failed).
int read_clear_error_loss();

size_t preference_ws_bytes(int64_t T, int64_t P);
// Rows of `row_bytes`; none where a row is held on chip, or without a gradient.
size_t policy_ws_bytes(int64_t T, int64_t row_bytes, bool grad);

lora_status_t token_logps(const LossArgs &a, float *stats, cudaStream_t st);
lora_status_t token_logps_backward(const LossArgs &a, const float *stats, const float *dlogps, cudaStream_t st);
lora_status_t preference_loss(const LossArgs &a, const PreferenceArgs &p, void *ws, size_t ws_bytes, cudaStream_t st);
lora_status_t policy_loss(const LossArgs &a, const PolicyArgs &p, void *ws, size_t ws_bytes, cudaStream_t st);
lora_status_t scale_gradient(lora_dtype_t dtype, int64_t T, int64_t V, void *x, int64_t ldx, const float *factor,
                             cudaStream_t st);

}  // namespace lora
