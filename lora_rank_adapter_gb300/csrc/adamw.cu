// adamw.cu -- the AdamW step over an adapter's many tensors, with states in 32 or
// in 8 bits, and the global norm of their gradients (include/lora_train.h).
//
// An adapter has some hundred tensors of ten thousand to a million elements, so
// the work is laid out once as a table of chunks (adamw_build) and a step is one
// launch over all of them: a block takes a chunk of 2048 elements, a warp a block
// of 256 (one scale of an 8-bit state), a lane 8 elements.
//
// States in 32 bits are bound by their bytes: 448 tensors, 168 M elements in bf16
// with fp32 gradients and masters (30 bytes an element): 705 us, 7.1 TB/s; with the
// norm's reading of the gradients 820 us.  States in 8 bits (10 bytes an element
// with bf16 gradients): 261 us, 6.5 TB/s, 95 % of the copy rate; single-value
// arithmetic and a division of full precision took 435 us.  Rounded at random they
// take 328 us where rounding to nearest takes 250 (back to back on the same data),
// 410 where it takes 393 with fp32 parameters and gradients: bound by its
// instructions, some 24 more an element (82 % of the issue slots, 68 to nearest).
// Tensors off 16-byte boundaries go element by element: the same fp32 step with
// masters 900 us (5.6 TB/s), 8-bit states 435; the norm of fp32 gradients 102
// (6.5 TB/s), of bf16 ones 84 (4.0 TB/s).
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "adamw.h"
#include "common.cuh"
#include "f32x2.cuh"
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
  r.wide = (rest & 15u) == 0 && (state & (a.e_s == 1 ? 3u : 15u)) == 0;
  table[c] = r;
}

// ----------------------------------------------------------------------------- 4 + 4 elements of a lane
// A warp's 256 elements in two halves of 128, four consecutive ones of each for a
// lane: every load and store of a warp covers whole stretches of memory, whatever
// the type (16 bytes a lane in fp32, 8 in bf16, 4 of codes).
template <typename T>
struct Four;      // four elements as they lie in memory; as two pairs of fp32 values
template <>
struct Four<float> {
  uint4 q;
  __device__ __forceinline__ void get(uint64_t *v) const {
    v[0] = pk2(__uint_as_float(q.x), __uint_as_float(q.y));
    v[1] = pk2(__uint_as_float(q.z), __uint_as_float(q.w));
  }
  __device__ __forceinline__ void set(const uint64_t *v) {
    const float2 a = unpk2(v[0]), b = unpk2(v[1]);
    q = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  }
};
template <>
struct Four<__nv_bfloat16> {
  uint2 q;
  __device__ __forceinline__ void get(uint64_t *v) const {
    v[0] = pk2(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u));
    v[1] = pk2(__uint_as_float(q.y << 16), __uint_as_float(q.y & 0xffff0000u));
  }
  __device__ __forceinline__ void set(const uint64_t *v) {
    const float2 a = unpk2(v[0]), b = unpk2(v[1]);
    q = make_uint2(pack_bf16(a.x, a.y), pack_bf16(b.x, b.y));
  }
};
template <>
struct Four<uint8_t> {      // e4m3 codes
  uint32_t q;
  __device__ __forceinline__ void get(uint64_t *v) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(i == 0 ? q : q >> 16), __NV_E4M3);
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
      v[i] = pk2(f.x, f.y);
    }
  }
  __device__ __forceinline__ void set(const uint64_t *v) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(unpk2(v[0]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(unpk2(v[1]), __NV_SATFINITE, __NV_E4M3);
    q = lo | (hi << 16);
  }
};

// Four elements, kWhole: all there and at an aligned address; else elements
// [0, n) one by one (n <= 4), the others read as zero and not written.
// kOnce: nobody reads it again.
template <bool kWhole, bool kOnce = true, typename T>
__device__ __forceinline__ Four<T> load4(const T *p, int n) {
  Four<T> r;
  if constexpr (kWhole) {
    const decltype(r.q) *q = reinterpret_cast<const decltype(r.q) *>(p);
    r.q = kOnce ? __ldcs(q) : *q;
  } else {
    T *e = reinterpret_cast<T *>(&r.q);
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = i < n ? p[i] : T(0.f);
  }
  return r;
}
template <bool kWhole, typename T>
__device__ __forceinline__ void store4(T *p, const Four<T> &r, int n) {
  if constexpr (kWhole) {
    __stcs(reinterpret_cast<decltype(r.q) *>(p), r.q);
  } else {
    const T *e = reinterpret_cast<const T *>(&r.q);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = e[i];
  }
}

// max(a, |b|), NaN if either is.
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// The factor 448 / a that brings the warp's 256 values to the codes' range, and
// their scale a / 448.  Across the warp the largest magnitude is taken on the bit
// patterns, whose order is that of the magnitudes with NaN above infinity: a NaN
// makes the block's scale NaN.
__device__ __forceinline__ float code_range(const uint64_t *v, float &scale) {
  float top = 1e-30f;
#pragma unroll
  for (int i = 0; i < kLane / 2; ++i) {
    const float2 f = unpk2(v[i]);
    top = max_abs(max_abs(top, f.x), f.y);
  }
  const float a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top) & 0x7fffffffu));
  scale = __fmul_rn(a, (float)(1.0 / 448.0));
  return __fdiv_rn(448.f, a);
}

// 1 / x to 2^-22 or so, for x of at least the smallest normal number (the step's
// divisor is taken up to it).
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(1.17549435e-38f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(r));
  return r;
}

// Bits for the rounding of 8-bit states, 16 for each of the two states of an element:
// multiplications by odd numbers and shifted exclusive ors (the golden ratio's and the
// square root of three's fractions of 2^32), as in multiplicative hashing.
constexpr uint32_t kMix1 = 0x9E3779B9u, kMix2 = 0xBB67AE85u;
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= kMix1;
  x ^= x >> 15;
  x *= kMix2;
  x ^= x >> 16;
  x *= kMix1;
  return x ^ (x >> 15);
}
// `x1`: a place times kMix1
__device__ __forceinline__ uint32_t place_bits(uint32_t x1) {
  x1 ^= x1 >> 15;
  x1 *= kMix2;
  return x1 ^ (x1 >> 16);
}

// q to one of the two e4m3 values around it, the upper one with the probability of how
// far up q is.  `bits` (20 of them, the lowest four 0) are added below the three bits
// of mantissa that stay; below 2^-6, where the values lie 2^-9 apart, after 2^-6 has
// been added.  Values at a code stay there.
__device__ __forceinline__ float to_code(float q, uint32_t bits) {
  const float base = fabsf(q) < 0.015625f ? copysignf(0.015625f, q) : 0.f;
  const uint32_t t = __float_as_uint(__fadd_rn(q, base)) + bits + 8u;
  return __fsub_rn(__uint_as_float(t & 0xfff00000u), base);
}

// ----------------------------------------------------------------------------- the step
struct StepArgs {
  const AdamChunk *table;
  const float *factor;
  float b1, b1c, b2, b2c;      // beta1, 1 - beta1, beta2, 1 - beta2
  float decay;                 // 1 - lr * weight_decay
  float rate;                  // -lr / (1 - beta1^step)
  float root;                  // 1 / sqrt(1 - beta2^step)
  float eps;
  float one;                   // 1
  uint32_t noise;              // of the step
};

// A warp's 256 elements as they lie in memory.
// kNoise: 8-bit states rounded at random.
template <typename P, typename G, bool k8, bool kNoise, bool kMaster>
struct Block {
  using S = std::conditional_t<k8, uint8_t, float>;
  using W = std::conditional_t<kMaster, float, P>;
  Four<G> g[2];
  Four<S> m[2], v[2];
  Four<W> w[2];
  float ms, vs;

  // `block`: its number in the chunk
  template <bool kWhole>
  __device__ __forceinline__ void load(const AdamChunk &c, int block) {
    const int at = block * LORA_ADAMW_BLOCK + 4 * lane_id();
    const W *wp = kMaster ? reinterpret_cast<const W *>(c.master) : static_cast<const W *>(c.p);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int o = at + 128 * h, n = min(max((int)c.count - o, 0), 4);
      g[h] = load4<kWhole>(static_cast<const G *>(c.g) + o, n);
      m[h] = load4<kWhole>(static_cast<const S *>(c.m) + o, n);
      v[h] = load4<kWhole>(static_cast<const S *>(c.v) + o, n);
      w[h] = load4<kWhole>(wp + o, n);
    }
    if (k8) {
      ms = c.m_scale[block];
      vs = c.v_scale[block];
    }
  }

  // The step, and its results back to memory.  The states' arithmetic is in
  // single IEEE roundings, on pairs of values; a sum of products is written
  // fma(x, 1, y) with the 1 from memory, because the compiler contracts a packed
  // product and sum to one rounding: equal inputs give equal 8-bit codes,
  // whoever computes them.
  // `key`: of the chunk and the step.
  template <bool kWhole>
  __device__ __forceinline__ void step(const StepArgs &a, float factor, const AdamChunk &c, int block, uint32_t key) {
    constexpr int kPairs = kLane / 2;
    auto both = [](float x) { return pk2(x, x); };
    uint64_t pw[kPairs], pg[kPairs], pm[kPairs], pv[kPairs];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      g[h].get(pg + 2 * h);
      m[h].get(pm + 2 * h);
      v[h].get(pv + 2 * h);
      w[h].get(pw + 2 * h);
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const uint64_t gi = mul2(pg[i], both(factor));
      if (k8) {
        pm[i] = mul2(pm[i], both(ms));
        pv[i] = mul2(pv[i], both(vs));
        pv[i] = mul2(pv[i], pv[i]);
      }
      pm[i] = fma2(mul2(pm[i], both(a.b1)), both(a.one), mul2(gi, both(a.b1c)));
      pv[i] = fma2(mul2(pv[i], both(a.b2)), both(a.one), mul2(mul2(gi, gi), both(a.b2c)));
      const float2 vv = unpk2(pv[i]);
      const uint64_t u = pk2(__fsqrt_rn(vv.x), __fsqrt_rn(vv.y));
      if (k8) pv[i] = u;
      // the quotient is off by some 2^-22: far below a parameter's own rounding
      const float2 d = unpk2(fma2(u, both(a.root), both(a.eps)));
      pw[i] = fma2(mul2(pm[i], pk2(reciprocal(d.x), reciprocal(d.y))), both(a.rate), mul2(pw[i], both(a.decay)));
    }
    if (k8) {
      const uint64_t mup = both(code_range(pm, ms)), vup = both(code_range(pv, vs));
      if (lane_id() == 0) {
        c.m_scale[block] = ms;
        c.v_scale[block] = vs;
      }
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        pm[i] = mul2(pm[i], mup);
        const float2 u = unpk2(pv[i]);
        float2 q = unpk2(mul2(pv[i], vup));
        if (kNoise) {
          const uint32_t x1 = (key + block * LORA_ADAMW_BLOCK + 4 * lane_id()) * kMix1;
          const uint32_t e = 128 * (i / 2) + 2 * (i % 2);
          const uint32_t r0 = place_bits(x1 + e * kMix1), r1 = place_bits(x1 + (e + 1) * kMix1);
          const float2 f = unpk2(pm[i]);
          pm[i] = pk2(to_code(f.x, (r0 << 4) & 0xffff0u), to_code(f.y, (r1 << 4) & 0xffff0u));
          q.x = to_code(q.x, (r0 >> 12) & 0xffff0u);
          q.y = to_code(q.y, (r1 >> 12) & 0xffff0u);
        }
        // the smallest positive code, 2^-9, for a root that would round to zero
        if (u.x > 0.f) q.x = fmaxf(q.x, 0.001953125f);
        if (u.y > 0.f) q.y = fmaxf(q.y, 0.001953125f);
        pv[i] = pk2(q.x, q.y);
      }
    }
    const int at = block * LORA_ADAMW_BLOCK + 4 * lane_id();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int o = at + 128 * h, n = min(max((int)c.count - o, 0), 4);
      Four<P> rp;
      rp.set(pw + 2 * h);
      store4<kWhole>(static_cast<P *>(c.p) + o, rp, n);
      if constexpr (kMaster) {
        w[h].set(pw + 2 * h);
        store4<kWhole>(c.master + o, w[h], n);
      }
      m[h].set(pm + 2 * h);
      store4<kWhole>(static_cast<S *>(c.m) + o, m[h], n);
      v[h].set(pv + 2 * h);
      store4<kWhole>(static_cast<S *>(c.v) + o, v[h], n);
    }
  }
};

// A block of threads takes a chunk; with states in 8 bits (few bytes a warp) each
// warp loads two blocks of it before it works on the first.  Eight blocks of 128
// threads an SM (64 registers) take 261 us where 72 registers took 273, nine blocks
// 273 and ten 297 (spills); four blocks of 256 threads for 32-bit states 820, five 865.
constexpr int kEach8 = 2, kEach32 = 1;
template <typename P, typename G, bool k8, bool kNoise, bool kMaster>
__global__ void __launch_bounds__(kThreads / (k8 ? kEach8 : kEach32), k8 ? 8 : 4) adamw_kernel(StepArgs a) {
  constexpr int kEach = k8 ? kEach8 : kEach32, kWarps = kThreads / 32 / kEach;
  pdl_wait();
  // last to first: the norm before this step has left the last gradients in L2
  const uint32_t chunk = gridDim.x - 1 - blockIdx.x;
  const AdamChunk c = a.table[chunk];
  const float factor = a.factor ? *a.factor : 1.f;
  const int warp = threadIdx.x >> 5;
  const uint32_t key = kNoise ? mix(a.noise + chunk) : 0;
  Block<P, G, k8, kNoise, kMaster> b[kEach];
  if (c.wide && c.count == LORA_ADAMW_CHUNK) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) b[i].template load<true>(c, warp + i * kWarps);
#pragma unroll
    for (int i = 0; i < kEach; ++i) b[i].template step<true>(a, factor, c, warp + i * kWarps, key);
  } else {
    // whole warps: a block's scale needs all 32 lanes
    for (int i = warp; i * LORA_ADAMW_BLOCK < (int)c.count; i += kWarps) {
      b[0].template load<false>(c, i);
      b[0].template step<false>(a, factor, c, i, key);
    }
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
  pdl_launch_dependents();      // the step's blocks may take their places and wait there
  Sum2 sum[1];
  for (int64_t k = blockIdx.x; k < chunks; k += gridDim.x) {
    const G *g = static_cast<const G *>(table[k].g);
    const int at = (int)(threadIdx.x >> 5) * LORA_ADAMW_BLOCK + 4 * lane_id(), count = (int)table[k].count;
    Four<G> r[2];
    uint64_t v[kLane / 2], s = 0;
    if ((reinterpret_cast<uintptr_t>(g) & 15u) == 0 && count == LORA_ADAMW_CHUNK) {
#pragma unroll
      for (int h = 0; h < 2; ++h) r[h] = load4<true, false>(g + at + 128 * h, 4);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) r[h] = load4<false>(g + at + 128 * h, min(max(count - at - 128 * h, 0), 4));
    }
    r[0].get(v);
    r[1].get(v + 2);
#pragma unroll
    for (int i = 0; i < kLane / 2; ++i) s = fma2(v[i], v[i], s);
    const float2 two = unpk2(s);
    sum[0].add(two.x + two.y);
  }
  block_sums<kThreads / 32, 1>(sum, sh);
  if (threadIdx.x == 0) {
    part[blockIdx.x] = sum[0];
    __threadfence();
    before = atomicInc(ticket, gridDim.x - 1);      // back to 0 with the last block
    __threadfence();
  }
  __syncthreads();
  if (before != gridDim.x - 1) return;
  sum[0] = Sum2();
  for (int i = threadIdx.x; i < (int)gridDim.x; i += kThreads) {
    const float2 p = __ldcg(reinterpret_cast<const float2 *>(part) + i);
    Sum2 one;
    one.hi = p.x;
    one.lo = p.y;
    sum[0].add(one);
  }
  block_sums<kThreads / 32, 1>(sum, sh);
  if (threadIdx.x == 0) {
    const float norm = sqrtf(sum[0].value()), f = max_norm / (norm + 1e-6f);
    out[0] = norm;
    out[1] = f >= 1.f ? 1.f : f;      // a NaN norm gives a NaN factor
  }
}

template <typename P, typename G, bool k8, bool kNoise>
cudaError_t run_step(const lora_adamw_plan_t &plan, const StepArgs &a, cudaStream_t st) {
  const dim3 grid((unsigned)plan.chunks), block(kThreads / (k8 ? kEach8 : kEach32));
  return (plan.flags & LORA_ADAMW_MASTER) ? launch(adamw_kernel<P, G, k8, kNoise, true>, grid, block, 0, st, 1, true, a)
                                          : launch(adamw_kernel<P, G, k8, kNoise, false>, grid, block, 0, st, 1, true, a);
}
template <typename P, typename G>
cudaError_t run_step(const lora_adamw_plan_t &plan, const StepArgs &a, cudaStream_t st) {
  if (plan.flags & LORA_ADAMW_STOCHASTIC) return run_step<P, G, true, true>(plan, a, st);
  return (plan.flags & LORA_ADAMW_STATE_8BIT) ? run_step<P, G, true, false>(plan, a, st)
                                              : run_step<P, G, false, false>(plan, a, st);
}

}  // namespace

// ----------------------------------------------------------------------------- host side
size_t table_bytes(int64_t chunks) {
  return ws_round(sizeof(AdamChunk) * (size_t)chunks) + ws_round(sizeof(unsigned)) + sizeof(Sum2) * kNormBlocks;
}
// Behind the chunks: the norm's ticket and partial sums.
static unsigned *norm_ticket(const void *table, int64_t chunks) {
  return reinterpret_cast<unsigned *>(static_cast<char *>(const_cast<void *>(table)) +
                                      ws_round(sizeof(AdamChunk) * (size_t)chunks));
}

lora_status_t adamw_build(const lora_adamw_tensor_t *tensors, int32_t n, const lora_adamw_plan_t &plan,
                          AdamChunk *table, cudaStream_t st) {
  BuildArgs a;
  a.e_p = plan.param_dtype == LORA_BF16 ? 2 : 4;
  a.e_g = plan.grad_dtype == LORA_BF16 ? 2 : 4;
  a.e_s = (plan.flags & LORA_ADAMW_STATE_8BIT) ? 1 : 4;
  LORA_CUDA(cudaMemsetAsync(norm_ticket(table, plan.chunks), 0, sizeof(unsigned), st));
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

lora_status_t grad_norm(const lora_adamw_plan_t &plan, float max_norm, float *out, cudaStream_t st) {
  // no tensors: one block that writes the norm 0
  const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>({plan.chunks, kNormBlocks, 8 * (int64_t)num_sms()}));
  unsigned *ticket = norm_ticket(plan.table, plan.chunks);
  Sum2 *part = reinterpret_cast<Sum2 *>(reinterpret_cast<char *>(ticket) + ws_round(sizeof(unsigned)));
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
  a.rate = (float)(-h.lr / (1.0 - pow(h.beta1, (double)h.step)));
  a.root = (float)(1.0 / sqrt(1.0 - pow(h.beta2, (double)h.step)));
  a.eps = (float)h.eps;
  a.one = 1.f;
  a.noise = mix((uint32_t)h.step + mix((uint32_t)(h.step >> 32)));
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
