// sum2.cuh -- sums in two fp32 parts, in a fixed order.
#pragma once

#include <math.h>

#include "common.cuh"

namespace lora {

// A sum in two fp32 parts, about 48 bits (64-bit arithmetic is slow on this
// chip: a block's sum in it took 10 us).  The rounding error of each addition,
// which is exact in fp32 (Knuth's two-sum), goes into `lo`.
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
    const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b));
    hi = s;
    // a sum that is infinite or NaN stays what it is
    lo = fabsf(s) < INFINITY ? __fadd_rn(lo, err) : 0.f;
  }
  __device__ __forceinline__ void add(const Sum2 &o) {
    add(o.hi);
    lo = fabsf(hi) < INFINITY ? __fadd_rn(lo, o.lo) : 0.f;
  }
  __device__ __forceinline__ float value() const { return hi + lo; }
};

// Sum over the warp's lanes, known to all of them.
__device__ __forceinline__ Sum2 warp_sum(Sum2 x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sum2 y;
    y.hi = __shfl_xor_sync(0xffffffffu, x.hi, o);
    y.lo = __shfl_xor_sync(0xffffffffu, x.lo, o);
    // both lanes of a pair add in the same order
    if (lane_id() & o) {
      y.add(x);
      x = y;
    } else {
      x.add(y);
    }
  }
  return x;
}

// K sums over the block in a fixed order, known to warp 0.  sh: K per warp, not in
// use by a call before this one.
template <int kWarps, int K>
__device__ __forceinline__ void block_sums(Sum2 (&v)[K], Sum2 *sh) {
#pragma unroll
  for (int i = 0; i < K; ++i) {
    v[i] = warp_sum(v[i]);
    if (lane_id() == 0) sh[i * kWarps + (threadIdx.x >> 5)] = v[i];
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = warp_sum(lane_id() < kWarps ? sh[i * kWarps + lane_id() % kWarps] : Sum2());
}

}  // namespace lora
