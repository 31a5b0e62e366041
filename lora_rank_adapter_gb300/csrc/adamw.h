// adamw.h -- internal interface of the optimizer step over many tensors (adamw.cu).
#pragma once

#include "../../include/lora_train.h"
#include "host_common.h"

namespace lora {

// One chunk of one tensor: its first element's addresses.  64 bytes, read whole
// by the block that takes the chunk.
struct AdamChunk {
  void *p;
  const void *g;
  void *m, *v;
  float *m_scale, *v_scale, *master;
  uint32_t count;     // elements, 1 .. LORA_ADAMW_CHUNK
  uint32_t wide;      // every address allows wide loads
};
static_assert(sizeof(AdamChunk) == 64, "a chunk is one 64-byte record");

// The chunks' records, and room for the gradient norm's partial sums.
size_t table_bytes(int64_t chunks);

lora_status_t adamw_build(const lora_adamw_tensor_t *tensors, int32_t n, const lora_adamw_plan_t &plan,
                          AdamChunk *table, cudaStream_t st);
lora_status_t grad_norm(const lora_adamw_plan_t &plan, float max_norm, float *out, cudaStream_t st);
lora_status_t adamw(const lora_adamw_plan_t &plan, const lora_adamw_hyper_t &h, const float *grad_factor,
                    cudaStream_t st);

}  // namespace lora
