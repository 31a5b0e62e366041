// adamw.cu -- the AdamW step over an adapter's many tensors, with states in 32 or
// in 8 bits, and the global norm of their gradients (include/lora_train.h).
//
// An adapter has some hundred tensors of ten thousand to a million elements, so
// the work is laid out once as a table of chunks (adamw_build) and a step is one
// launch over all of them: a block takes a chunk of 2048 elements, a warp a block
// of 256 (one scale of an 8-bit state), a lane 8 consecutive elements.
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>

#include "adamw.h"
#include "common.cuh"
#include "host_common.h"
#include "sum2.cuh"

namespace lora {
namespace {

constexpr int kThreads = 256;
constexpr int kLane = 8;                 // elements of a lane
constexpr int kNormBlocks = 2048;        // partial sums at most
static_assert(kThreads * kLane == LORA_ADAMW_CHUNK && 32 * kLane == LORA_ADAMW_BLOCK, "a warp holds one block");

// ----------------------------------------------------------------------------- the table
constexpr int kBuildTensors = 256;
struct BuildArgs {
  lora_adamw_tensor_t t[kBuildTensors];
  int64_t first[kBuildTensors + 1];      // chunks before tensor i, of this group
  int n;
  int e_p, e_g, e_s;                     // bytes of an element: parameter, gradient, state
};

__global__ void build_kernel(const __grid_constant__ BuildArgs a, AdamChunk *table) {
  pdl_wait();
  const int64_t c = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (c >= a.first[a.n]) return;
  int lo = 0, hi = a.n - 1;              // the tensor with first[lo] <= c < first[lo + 1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.first[mid] <= c) lo = mid; else hi = mid - 1;
  }
  const lora_adamw_tensor_t &t = a.t[lo];
  const int64_t at = (c - a.first[lo]) * LORA_ADAMW_CHUNK, left = t.numel - at;
  auto shift = [](const void *p, int64_t bytes) { return (void *)((char *)const_cast<void *>(p) + bytes); };
  AdamChunk r;
  r.p = shift(t.param, at * a.e_p);
  r.g = shift(t.grad, at * a.e_g);
  r.m = shift(t.exp_avg, at * a.e_s);
  r.v = shift(t.exp_avg_sq, at * a.e_s);
  r.m_scale = t.exp_avg_scale ? t.exp_avg_scale + at / LORA_ADAMW_BLOCK : nullptr;
  r.v_scale = t.exp_avg_sq_scale ? t.exp_avg_sq_scale + at / LORA_ADAMW_BLOCK : nullptr;
  r.master = t.master ? t.master + at : nullptr;
  r.count = (uint32_t)(left < LORA_ADAMW_CHUNK ? left : LORA_ADAMW_CHUNK);
  const uintptr_t state = reinterpret_cast<uintptr_t>(t.exp_avg) | reinterpret_cast<uintptr_t>(t.exp_avg_sq);
  const uintptr_t rest = reinterpret_cast<uintptr_t>(t.param) | reinterpret_cast<uintptr_t>(t.grad) |
                         reinterpret_cast<uintptr_t>(t.master);
  r.wide = (rest & 15u) == 0 && (state & (a.e_s == 1 ? 7u : 15u)) == 0;
  table[c] = r;
}

// ----------------------------------------------------------------------------- 8 elements of a lane
__device__ __forceinline__ void load8(const float *p, float *v) {
  const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float *v) {
  const uint4 q = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_bf16(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void store8(float *p, const float *v) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *v) {
  *reinterpret_cast<uint4 *>(p) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// Elements [0, n) of a lane's eight; the others read as zero and are not written.
template <typename E>
__device__ __forceinline__ void load_lane(const E *p, float *v, int n, bool wide) {
  if (wide && n == kLane) {
    load8(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < kLane; ++i) v[i] = i < n ? load1(p + i) : 0.f;
  }
}
template <typename E>
__device__ __forceinline__ void store_lane(E *p, const float *v, int n, bool wide) {
  if (wide && n == kLane) {
    store8(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < kLane; ++i)
      if (i < n) store1(p + i, v[i]);
  }
}

// e4m3 codes: eight of a lane are 8 bytes.
__device__ __forceinline__ void decode8(const uint8_t *c, float *v, float scale) {
#pragma unroll
  for (int i = 0; i < kLane; i += 2) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c[i] | (c[i + 1] << 8)), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    v[i] = __fmul_rn(f.x, scale);
    v[i + 1] = __fmul_rn(f.y, scale);
  }
}
__device__ __forceinline__ void load_codes(const uint8_t *p, float *v, float scale, int n, bool wide) {
  uint8_t c[kLane];
  if (wide && n == kLane) {
    *reinterpret_cast<uint2 *>(c) = *reinterpret_cast<const uint2 *>(p);
  } else {
#pragma unroll
    for (int i = 0; i < kLane; ++i) c[i] = i < n ? p[i] : 0;
  }
  decode8(c, v, scale);
}

// The warp's 256 values as codes and one scale.  The largest magnitude is taken
// on the bit patterns, whose order is that of the magnitudes with NaN above
// infinity: a NaN makes the block's scale NaN.
template <bool kRoot>
__device__ __forceinline__ void store_codes(uint8_t *p, float *scale, const float *v, int n, bool wide) {
  uint32_t top = __float_as_uint(1e-30f);
#pragma unroll
  for (int i = 0; i < kLane; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  top = __reduce_max_sync(0xffffffffu, top);
  const float a = __uint_as_float(top), up = __fdiv_rn(448.f, a);
  uint8_t c[kLane];
#pragma unroll
  for (int i = 0; i < kLane; i += 2) {
    float q[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      q[j] = __fmul_rn(v[i + j], up);
      // the smallest positive code, 2^-9, for a root that would round to zero
      if (kRoot && v[i + j] > 0.f) q[j] = fmaxf(q[j], 0.001953125f);
    }
    const __nv_fp8x2_storage_t two = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
    c[i] = (uint8_t)(two & 0xff);
    c[i + 1] = (uint8_t)(two >> 8);
  }
  if (wide && n == kLane) {
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<uint2 *>(c);
  } else {
#pragma unroll
    for (int i = 0; i < kLane; ++i)
      if (i < n) p[i] = c[i];
  }
  if (lane_id() == 0) *scale = __fmul_rn(a, (float)(1.0 / 448.0));
}

// ----------------------------------------------------------------------------- the step
struct StepArgs {
  const AdamChunk *table;
  const float *factor;
  float b1, b1c, b2, b2c;      // beta1, 1 - beta1, beta2, 1 - beta2
  float decay;                 // 1 - lr * weight_decay
  float rate;                  // lr / (1 - beta1^step)
  float root;                  // 1 / sqrt(1 - beta2^step)
  float eps;
};

// The states' arithmetic is written in single IEEE roundings (no contraction to
// multiply-add): equal inputs give equal 8-bit codes, whoever computes them.
template <typename P, typename G, bool k8, bool kMaster>
__global__ void __launch_bounds__(kThreads) adamw_kernel(StepArgs a) {
  pdl_wait();
  const AdamChunk c = a.table[blockIdx.x];
  const int warp = threadIdx.x >> 5;
  const int at = (int)threadIdx.x * kLane;
  if (warp * LORA_ADAMW_BLOCK >= (int)c.count) return;      // whole warps: a block's scale needs all 32 lanes
  const int n = min(max((int)c.count - at, 0), kLane);
  const bool wide = c.wide != 0;
  const float factor = a.factor ? *a.factor : 1.f;
  P *p = static_cast<P *>(c.p) + at;
  float w[kLane], g[kLane], m[kLane], v[kLane];
  load_lane(static_cast<const G *>(c.g) + at, g, n, wide);
  if (kMaster)
    load_lane(c.master + at, w, n, wide);
  else
    load_lane(p, w, n, wide);
  if (k8) {
    load_codes(static_cast<uint8_t *>(c.m) + at, m, c.m_scale[warp], n, wide);
    load_codes(static_cast<uint8_t *>(c.v) + at, v, c.v_scale[warp], n, wide);
  } else {
    load_lane(static_cast<float *>(c.m) + at, m, n, wide);
    load_lane(static_cast<float *>(c.v) + at, v, n, wide);
  }
#pragma unroll
  for (int i = 0; i < kLane; ++i) {
    const float gi = __fmul_rn(g[i], factor);
    if (k8) v[i] = __fmul_rn(v[i], v[i]);
    m[i] = __fadd_rn(__fmul_rn(m[i], a.b1), __fmul_rn(gi, a.b1c));
    v[i] = __fadd_rn(__fmul_rn(v[i], a.b2), __fmul_rn(__fmul_rn(gi, gi), a.b2c));
    const float u = __fsqrt_rn(v[i]);
    if (k8) v[i] = u;
    w[i] = w[i] * a.decay - a.rate * (m[i] / (u * a.root + a.eps));
  }
  if (kMaster) store_lane(c.master + at, w, n, wide);
  store_lane(p, w, n, wide);
  if (k8) {
    store_codes<false>(static_cast<uint8_t *>(c.m) + at, c.m_scale + warp, m, n, wide);
    store_codes<true>(static_cast<uint8_t *>(c.v) + at, c.v_scale + warp, v, n, wide);
  } else {
    store_lane(static_cast<float *>(c.m) + at, m, n, wide);
    store_lane(static_cast<float *>(c.v) + at, v, n, wide);
  }
}

// ----------------------------------------------------------------------------- the norm
// Squares summed in fp32 over a lane's elements of a chunk, in two fp32 parts
// beyond that; the last block adds the blocks' sums in block order.
template <typename G>
__global__ void __launch_bounds__(kThreads) norm_kernel(const AdamChunk *table, int64_t chunks, Sum2 *part,
                                                        unsigned *ticket, float max_norm, float *out) {
  __shared__ Sum2 sh[kThreads / 32];
  __shared__ unsigned before;
  pdl_wait();
  Sum2 sum;
  for (int64_t k = blockIdx.x; k < chunks; k += gridDim.x) {
    const G *g = static_cast<const G *>(table[k].g);
    const int at = (int)threadIdx.x * kLane, n = min(max((int)table[k].count - at, 0), kLane);
    float v[kLane], s = 0.f;
    load_lane(g + at, v, n, (reinterpret_cast<uintptr_t>(g) & 15u) == 0);
#pragma unroll
    for (int i = 0; i < kLane; ++i) s += v[i] * v[i];
    sum.add(s);
  }
  sum = block_sum<kThreads / 32>(sum, sh);
  if (threadIdx.x == 0) {
    part[blockIdx.x] = sum;
    __threadfence();
    before = atomicAdd(ticket, 1u);
    __threadfence();
  }
  __syncthreads();
  if (before != gridDim.x - 1) return;
  sum = Sum2();
  for (int i = threadIdx.x; i < (int)gridDim.x; i += kThreads) {
    const float2 p = __ldcg(reinterpret_cast<const float2 *>(part) + i);
    Sum2 one;
    one.hi = p.x;
    one.lo = p.y;
    sum.add(one);
  }
  sum = block_sum<kThreads / 32>(sum, sh);
  if (threadIdx.x == 0) {
    const float norm = sqrtf(sum.value()), f = max_norm / (norm + 1e-6f);
    out[0] = norm;
    out[1] = f >= 1.f ? 1.f : f;      // a NaN norm gives a NaN factor
  }
}

template <typename P, typename G, bool k8>
cudaError_t run_step(const lora_adamw_plan_t &plan, const StepArgs &a, cudaStream_t st) {
  const dim3 grid((unsigned)plan.chunks), block(kThreads);
  return (plan.flags & LORA_ADAMW_MASTER) ? launch(adamw_kernel<P, G, k8, true>, grid, block, 0, st, 1, true, a)
                                          : launch(adamw_kernel<P, G, k8, false>, grid, block, 0, st, 1, true, a);
}
template <typename P, typename G>
cudaError_t run_step(const lora_adamw_plan_t &plan, const StepArgs &a, cudaStream_t st) {
  return (plan.flags & LORA_ADAMW_STATE_8BIT) ? run_step<P, G, true>(plan, a, st) : run_step<P, G, false>(plan, a, st);
}

}  // namespace

// ----------------------------------------------------------------------------- host side
// Blocks of the norm at most (no tensors: one block that writes the norm 0).
static int64_t norm_blocks(int64_t chunks) { return std::max<int64_t>(1, std::min<int64_t>(chunks, kNormBlocks)); }

size_t grad_norm_ws_bytes(int64_t chunks) {
  return ws_round(sizeof(unsigned)) + ws_round(sizeof(Sum2) * (size_t)norm_blocks(chunks));
}

lora_status_t adamw_build(const lora_adamw_tensor_t *tensors, int32_t n, const lora_adamw_plan_t &plan,
                          AdamChunk *table, cudaStream_t st) {
  BuildArgs a;
  a.e_p = plan.param_dtype == LORA_BF16 ? 2 : 4;
  a.e_g = plan.grad_dtype == LORA_BF16 ? 2 : 4;
  a.e_s = (plan.flags & LORA_ADAMW_STATE_8BIT) ? 1 : 4;
  for (int32_t i = 0; i < n;) {
    a.n = 0;
    a.first[0] = 0;
    for (; i < n && a.n < kBuildTensors; ++i) {
      if (tensors[i].numel == 0) continue;
      lora_adamw_tensor_t t = tensors[i];
      if (!(plan.flags & LORA_ADAMW_STATE_8BIT)) t.exp_avg_scale = t.exp_avg_sq_scale = nullptr;
      if (!(plan.flags & LORA_ADAMW_MASTER)) t.master = nullptr;
      a.t[a.n] = t;
      a.first[a.n + 1] = a.first[a.n] + ceil_div(t.numel, LORA_ADAMW_CHUNK);
      ++a.n;
    }
    if (a.n == 0) break;
    const int64_t chunks = a.first[a.n];
    LORA_CUDA(launch(build_kernel, dim3((unsigned)ceil_div(chunks, 128)), dim3(128), 0, st, 1, true, a, table));
    table += chunks;
  }
  return LORA_OK;
}

lora_status_t grad_norm(const lora_adamw_plan_t &plan, float max_norm, float *out, void *ws, size_t ws_bytes,
                        cudaStream_t st) {
  WsCarver c(ws, ws_bytes);
  unsigned *ticket = static_cast<unsigned *>(c.take(sizeof(unsigned)));
  const int blocks = (int)std::min<int64_t>(norm_blocks(plan.chunks), 8 * (int64_t)num_sms());
  Sum2 *part = static_cast<Sum2 *>(c.take(sizeof(Sum2) * (size_t)blocks));
  if (part == nullptr) return LORA_ERR_WORKSPACE;
  LORA_CUDA(cudaMemsetAsync(ticket, 0, sizeof(unsigned), st));
  const AdamChunk *table = static_cast<const AdamChunk *>(plan.table);
  if (plan.grad_dtype == LORA_BF16)
    LORA_CUDA(launch(norm_kernel<__nv_bfloat16>, dim3(blocks), dim3(kThreads), 0, st, 1, true, table, plan.chunks,
                     part, ticket, max_norm, out));
  else
    LORA_CUDA(launch(norm_kernel<float>, dim3(blocks), dim3(kThreads), 0, st, 1, true, table, plan.chunks, part,
                     ticket, max_norm, out));
  return LORA_OK;
}

lora_status_t adamw(const lora_adamw_plan_t &plan, const lora_adamw_hyper_t &h, const float *grad_factor,
                    cudaStream_t st) {
  if (plan.chunks == 0) return LORA_OK;
  StepArgs a;
  a.table = static_cast<const AdamChunk *>(plan.table);
  a.factor = grad_factor;
  a.b1 = (float)h.beta1;
  a.b1c = (float)(1.0 - h.beta1);
  a.b2 = (float)h.beta2;
  a.b2c = (float)(1.0 - h.beta2);
  a.decay = (float)(1.0 - h.lr * h.weight_decay);
  a.rate = (float)(h.lr / (1.0 - pow(h.beta1, (double)h.step)));
  a.root = (float)(1.0 / sqrt(1.0 - pow(h.beta2, (double)h.step)));
  a.eps = (float)h.eps;
  const bool p16 = plan.param_dtype == LORA_BF16, g16 = plan.grad_dtype == LORA_BF16;
  cudaError_t e;
  if (p16)
    e = g16 ? run_step<__nv_bfloat16, __nv_bfloat16>(plan, a, st) : run_step<__nv_bfloat16, float>(plan, a, st);
  else
    e = g16 ? run_step<float, __nv_bfloat16>(plan, a, st) : run_step<float, float>(plan, a, st);
  LORA_CUDA(e);
  return LORA_OK;
}

}  // namespace lora
