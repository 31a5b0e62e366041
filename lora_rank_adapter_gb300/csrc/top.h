// top.h -- internal interface of the operators over a row's most probable tokens:
// log-probabilities with entropy and alternatives (top.cu) and the distillation loss
// from a teacher's record of them (distill.cu).
#pragma once

#include "../../include/lora_train.h"
#include "host_common.h"

namespace lora {

struct TopArgs {
  lora_dtype_t dtype;
  int64_t T, V;
  int K;
  const void *logits;
  int64_t ldl;
  const int64_t *labels;      // NULL: every row counts
  double temperature;
  float *logps, *entropy;     // [T], NULL: not wanted
  int64_t *top_ids;           // [T][K]
  float *top_logps;           // [T][K]
  float *rest_logps;          // [T] or NULL
  float *stats;               // [T][2] or NULL
};

struct TopGradArgs {
  const int64_t *top_ids;     // [T][K]
  const float *stats, *entropy;
  const float *dlogps, *dentropy, *dtop_logps;      // NULL: zero
  void *dlogits;
  int64_t lddl;
};

struct DistillArgs {
  lora_dtype_t dtype;
  int64_t T, V;
  int K;
  const void *logits;
  int64_t ldl;
  const int64_t *ids;         // [T][K]
  const float *teacher;       // [T][K]
  const float *rest;          // [T] or NULL
  const float *weights;       // [T] or NULL
  bool reverse;
  double temperature;
  float *row_loss, *loss;     // [T], [1]
  void *dlogits;              // NULL: no gradient
  int64_t lddl;
  float grad_scale;
};

// Read and clear the error words of the waits in top.cu and distill.cu (-1: the read failed).
int read_clear_error_distill();

lora_status_t top_logps(const TopArgs &a, cudaStream_t st);
lora_status_t top_logps_backward(const TopArgs &a, const TopGradArgs &g, cudaStream_t st);
lora_status_t distill_loss(const DistillArgs &a, cudaStream_t st);

}  // namespace lora
