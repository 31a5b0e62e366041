// loss.cu -- log-probabilities of labels, the preference loss and the clipped
// policy loss over rows of logits, with their gradients (include/lora_train.h).
//
// Every operator is made of row passes over the logits and small kernels over
// the T per-token values between them:
//   stats_kernel   one read of a row: its largest logit m and S = sum exp(z - m),
//                  a softmax's running maximum and sum, and the label's logp;
//   pairs_kernel / tokens_kernel   the loss and each token's d loss / d logp;
//   grad_kernel    d = c * ((v == label) - exp(z - m) / S), the row read again.
#include <math.h>

#include "common.cuh"
#include "host_common.h"
#include "loss.h"

namespace lora {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename E>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float load(const float *p) { return *p; }
  static __device__ __forceinline__ void store(float *p, float v) { *p = v; }
  static __device__ __forceinline__ void unpack(const uint4 &q, float *v) {
    v[0] = __uint_as_float(q.x);
    v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z);
    v[3] = __uint_as_float(q.w);
  }
  static __device__ __forceinline__ uint4 pack(const float *v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float load(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
  static __device__ __forceinline__ void unpack(const uint4 &q, float *v) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float *v) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
};

// A row split at 16-byte boundaries: `head` elements before the first, `vecs`
// whole 16-byte pieces, and the rest.
template <typename E>
struct RowSpan {
  int64_t head, vecs;
  __device__ __forceinline__ RowSpan(const E *row, int64_t V) {
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
    head = ((16u - off) & 15u) / sizeof(E);
    if (head > V) head = V;
    vecs = (V - head) / Elem<E>::kVec;
  }
};

// Running (m, s): the largest value seen and s = sum exp((x - m) * inv_t), with
// k = inv_t * log2(e).  While m is minus infinity nothing but minus infinity has
// been seen and s is zero; the reference is then 0 instead of m, so that
// exp(-inf - ref) is 0 and not NaN.
__device__ __forceinline__ float ref_of(float m) { return m == kNegInf ? 0.f : m; }

__device__ __forceinline__ void merge(float &m, float &s, float m2, float s2, float k) {
  const float mm = fmaxf(m, m2), r = ref_of(mm);
  s = s * ex2((m - r) * k) + s2 * ex2((m2 - r) * k);
  m = mm;
}

// One element / one 16-byte piece into the running pair.
template <int N>
__device__ __forceinline__ void absorb(float &m, float &s, const float *v, float k) {
  float b = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) b = fmaxf(b, v[i]);
  const float mm = fmaxf(m, b), r = ref_of(mm);
  float add = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) add += ex2((v[i] - r) * k);
  s = s * ex2((m - r) * k) + add;
  m = mm;
}

// (m, s) of the whole block, known to every thread.  sh: 2 floats per warp.
template <int kWarps>
__device__ __forceinline__ void block_merge(float &m, float &s, float k, float *sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    merge(m, s, m2, s2, k);
  }
  const int w = threadIdx.x >> 5;
  if (lane_id() == 0) {
    sh[2 * w] = m;
    sh[2 * w + 1] = s;
  }
  __syncthreads();
  m = sh[0];
  s = sh[1];
#pragma unroll
  for (int i = 1; i < kWarps; ++i) merge(m, s, sh[2 * i], sh[2 * i + 1], k);
}

// ----------------------------------------------------------------------------- row passes
constexpr int kRowThreads = 256;

struct RowArgs {
  const void *logits;
  int64_t ldl;
  const int64_t *labels;
  int64_t T, V;
  float inv_t;
  float *logps;        // stats pass
  float2 *stats;       // written by the stats pass (NULL: not wanted), read by the gradient pass
  float *coef;         // stats pass: zeroed (NULL: none); gradient pass: d loss / d logp
  unsigned *ticket;    // zeroed for the kernel that follows (NULL: none)
  void *dlogits;
  int64_t lddl;
  float grad_scale;
};

template <typename E>
__global__ void __launch_bounds__(kRowThreads) stats_kernel(RowArgs a) {
  __shared__ float sh[2 * (kRowThreads / 32)];
  pdl_wait();
  const int64_t t = blockIdx.x;
  if (threadIdx.x == 0) {
    if (a.coef) a.coef[t] = 0.f;
    if (a.ticket && t == 0) *a.ticket = 0;
  }
  const int64_t label = a.labels[t];
  if (label < 0 || label >= a.V) {
    if (threadIdx.x == 0) {
      a.logps[t] = 0.f;
      if (a.stats) a.stats[t] = make_float2(0.f, 1.f);
    }
    return;
  }
  const E *row = static_cast<const E *>(a.logits) + t * a.ldl;
  const RowSpan<E> sp(row, a.V);
  const float k = a.inv_t * kLog2e;
  float m = kNegInf, s = 0.f;
  constexpr int N = Elem<E>::kVec;
  if (threadIdx.x < sp.head) {
    const float v = Elem<E>::load(row + threadIdx.x);
    absorb<1>(m, s, &v, k);
  }
  const uint4 *body = reinterpret_cast<const uint4 *>(row + sp.head);
  for (int64_t i = threadIdx.x; i < sp.vecs; i += kRowThreads) {
    float v[N];
    Elem<E>::unpack(body[i], v);
    absorb<N>(m, s, v, k);
  }
  const int64_t tail = sp.head + sp.vecs * N;
  if (tail + threadIdx.x < a.V) {
    const float v = Elem<E>::load(row + tail + threadIdx.x);
    absorb<1>(m, s, &v, k);
  }
  block_merge<kRowThreads / 32>(m, s, k, sh);
  if (threadIdx.x == 0) {
    a.logps[t] = (Elem<E>::load(row + label) - m) * a.inv_t - logf(s);
    if (a.stats) a.stats[t] = make_float2(m, s);
  }
}

template <typename E>
__global__ void __launch_bounds__(kRowThreads) grad_kernel(RowArgs a) {
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int64_t label = a.labels[t];
  E *out = static_cast<E *>(a.dlogits) + t * a.lddl;
  const E *row = static_cast<const E *>(a.logits) + t * a.ldl;
  constexpr int N = Elem<E>::kVec;
  const float c = a.coef[t] * a.grad_scale * a.inv_t;
  if (label < 0 || label >= a.V || c == 0.f) {
    const RowSpan<E> so(out, a.V);
    uint4 *body = reinterpret_cast<uint4 *>(out + so.head);
    if (threadIdx.x < so.head) Elem<E>::store(out + threadIdx.x, 0.f);
    for (int64_t i = threadIdx.x; i < so.vecs; i += kRowThreads) body[i] = make_uint4(0, 0, 0, 0);
    const int64_t tail = so.head + so.vecs * N;
    if (tail + threadIdx.x < a.V) Elem<E>::store(out + tail + threadIdx.x, 0.f);
    return;
  }
  const float2 st = a.stats[t];
  const float k = a.inv_t * kLog2e, m = st.x, q = -c / st.y;
  const RowSpan<E> sp(row, a.V);
  auto one = [&](int64_t i) {
    const float d = q * ex2((Elem<E>::load(row + i) - m) * k);
    Elem<E>::store(out + i, i == label ? d + c : d);
  };
  if (threadIdx.x < sp.head) one(threadIdx.x);
  const uint4 *body = reinterpret_cast<const uint4 *>(row + sp.head);
  const bool wide = (reinterpret_cast<uintptr_t>(out + sp.head) & 15u) == 0;
  for (int64_t i = threadIdx.x; i < sp.vecs; i += kRowThreads) {
    float v[N];
    Elem<E>::unpack(body[i], v);
    const int64_t first = sp.head + i * N;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      v[j] = q * ex2((v[j] - m) * k);
      if (first + j == label) v[j] += c;
    }
    if (wide) {
      *reinterpret_cast<uint4 *>(out + first) = Elem<E>::pack(v);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) Elem<E>::store(out + first + j, v[j]);
    }
  }
  const int64_t tail = sp.head + sp.vecs * N;
  if (tail + threadIdx.x < a.V) one(tail + threadIdx.x);
}

// ----------------------------------------------------------------------------- per-token steps
constexpr int kPairThreads = 256;

// Sum over the block in a fixed order, known to every thread.
template <int kWarps>
__device__ __forceinline__ double block_sum(double v, double *sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (lane_id() == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sh[0];
#pragma unroll
  for (int i = 1; i < kWarps; ++i) v += sh[i];
  return v;
}

// ln sigmoid(h) = min(h, 0) - ln(1 + exp(-|h|)), free of overflow and of cancellation
__device__ __forceinline__ float log_sigmoid(float h) { return fminf(h, 0.f) - log1pf(expf(-fabsf(h))); }

// The last block to get here, known to all its threads; the others' writes are visible to it.
__device__ __forceinline__ bool last_block(unsigned *ticket, unsigned blocks) {
  __shared__ unsigned before;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    before = atomicAdd(ticket, 1u);
    __threadfence();
  }
  __syncthreads();
  return before == blocks - 1;
}

// One block per pair: both sequences' sums (in 64 bits: their difference is what
// counts), the pair's loss, and each token's d loss / d logp.  The last block
// takes the mean.
__global__ void __launch_bounds__(kPairThreads) pairs_kernel(PreferenceArgs p, int64_t T, int64_t V,
                                                             const int64_t *labels, const float *logps, float *coef,
                                                             unsigned *ticket) {
  __shared__ double sh[kPairThreads / 32];
  pdl_wait();
  const int pair = blockIdx.x;
  int64_t lo[2], hi[2];
  float S[2], n[2];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int seq = pair + side * p.P;
    lo[side] = min(max((int64_t)p.cu[seq], (int64_t)0), T);
    hi[side] = min(max((int64_t)p.cu[seq + 1], (int64_t)0), T);
    double sum = 0.0, count = 0.0;
    for (int64_t t = lo[side] + threadIdx.x; t < hi[side]; t += kPairThreads) sum += logps[t];
    if (p.normalize)
      for (int64_t t = lo[side] + threadIdx.x; t < hi[side]; t += kPairThreads)
        count += labels[t] >= 0 && labels[t] < V ? 1.0 : 0.0;
    sum = block_sum<kPairThreads / 32>(sum, sh);
    n[side] = 1.f;
    if (p.normalize) n[side] = fmaxf(1.f, (float)block_sum<kPairThreads / 32>(count, sh));
    S[side] = (float)(sum / n[side]);
    if (threadIdx.x == 0) p.seq_logps[seq] = S[side];
  }
  float d = S[0] - S[1];
  if (p.ref) d -= p.ref[pair] - p.ref[pair + p.P];
  float loss, slope;
  if (p.kind == LORA_PREF_SIGMOID) {
    const float h = p.beta * d;
    loss = -(1.f - p.smoothing) * log_sigmoid(h) - p.smoothing * log_sigmoid(-h);
    // d loss / d h = sigmoid(h) - (1 - eps), written without cancellation at large |h|
    slope = p.beta * (p.smoothing / (1.f + expf(-h)) - (1.f - p.smoothing) / (1.f + expf(h)));
  } else if (p.kind == LORA_PREF_HINGE) {
    loss = fmaxf(0.f, 1.f - p.beta * d);
    if (d != d) loss = d;
    slope = 1.f - p.beta * d > 0.f ? -p.beta : 0.f;
    if (d != d) slope = d;
  } else {
    const float u = d - 0.5f / p.beta;
    loss = u * u;
    slope = 2.f * u;
  }
  if (coef) {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const float c = (side == 0 ? slope : -slope) / (float)p.P / n[side];
      for (int64_t t = lo[side] + threadIdx.x; t < hi[side]; t += kPairThreads) coef[t] = c;
    }
  }
  if (threadIdx.x == 0) p.pair_loss[pair] = loss;
  if (last_block(ticket, gridDim.x)) {
    double sum = 0.0;
    for (int i = threadIdx.x; i < p.P; i += kPairThreads) sum += __ldcg(p.pair_loss + i);
    sum = block_sum<kPairThreads / 32>(sum, sh);
    if (threadIdx.x == 0) p.loss[0] = (float)(sum / p.P);
  }
}

// A token's part of the policy loss: the terms of the three metrics, and its
// d loss / d logp.
struct PolicyTerm {
  float loss, kl, clipped, coef;
};
__device__ __forceinline__ PolicyTerm policy_term(const PolicyArgs &p, int64_t t, float logp) {
  const float A = p.advantages[t], w = p.weights ? p.weights[t] : 1.f;
  const float r = p.old_logps ? expf(logp - p.old_logps[t]) : expf(logp - logp);
  const float hi = 1.f + p.clip_high, lo = 1.f - p.clip_low;
  const bool clipped = (A > 0.f && r > hi) || (A < 0.f && r < lo);
  float pg = -A * r, coef = -A * r;
  if (clipped) {
    pg = -A * (A > 0.f ? hi : lo);
    coef = 0.f;
  }
  float kl = 0.f;
  if (p.ref_logps) {
    const float d = p.ref_logps[t] - logp, e = expm1f(d);
    kl = e - d;
    coef -= p.kl_beta * e;
  }
  return {w * (pg + p.kl_beta * kl), w * kl, clipped ? w : 0.f, w * coef};
}

// Sums of the blocks' three partial sums, in block order, by the last block.
__device__ __forceinline__ void policy_finish(const double *part, int blocks, float *metrics) {
  if (threadIdx.x < 3) {
    double s = 0.0;
    for (int i = 0; i < blocks; ++i) s += __ldcg(part + 3 * i + threadIdx.x);
    metrics[threadIdx.x] = (float)s;
  }
}

__global__ void __launch_bounds__(kPairThreads) tokens_kernel(PolicyArgs p, int64_t T, int64_t V,
                                                              const int64_t *labels, const float *logps, float *coef,
                                                              double *part, unsigned *ticket) {
  __shared__ double sh[kPairThreads / 32];
  pdl_wait();
  double s[3] = {0.0, 0.0, 0.0};
  const int64_t t = blockIdx.x * (int64_t)kPairThreads + threadIdx.x;
  if (t < T && labels[t] >= 0 && labels[t] < V) {
    const PolicyTerm x = policy_term(p, t, logps[t]);
    if (coef) coef[t] = x.coef;
    s[0] = x.loss;
    s[1] = x.kl;
    s[2] = x.clipped;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    s[i] = block_sum<kPairThreads / 32>(s[i], sh);
    if (threadIdx.x == 0) part[3 * (int64_t)blockIdx.x + i] = s[i];
  }
  if (last_block(ticket, gridDim.x)) policy_finish(part, gridDim.x, p.metrics);
}

template <typename E>
__global__ void __launch_bounds__(kRowThreads) scale_kernel(E *x, int64_t ldx, int64_t V, const float *factor) {
  pdl_wait();
  const float f = *factor;
  if (f == 1.f) return;
  E *row = x + (int64_t)blockIdx.x * ldx;
  const RowSpan<E> sp(row, V);
  constexpr int N = Elem<E>::kVec;
  if (threadIdx.x < sp.head) Elem<E>::store(row + threadIdx.x, Elem<E>::load(row + threadIdx.x) * f);
  uint4 *body = reinterpret_cast<uint4 *>(row + sp.head);
  for (int64_t i = threadIdx.x; i < sp.vecs; i += kRowThreads) {
    float v[N];
    Elem<E>::unpack(body[i], v);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] *= f;
    body[i] = Elem<E>::pack(v);
  }
  const int64_t tail = sp.head + sp.vecs * N;
  if (tail + threadIdx.x < V) Elem<E>::store(row + tail + threadIdx.x, Elem<E>::load(row + tail + threadIdx.x) * f);
}

RowArgs row_args(const LossArgs &a) {
  RowArgs r{};
  r.logits = a.logits;
  r.ldl = a.ldl;
  r.labels = a.labels;
  r.T = a.T;
  r.V = a.V;
  r.inv_t = 1.f / a.temperature;
  r.logps = a.logps;
  r.dlogits = a.dlogits;
  r.lddl = a.lddl;
  r.grad_scale = a.grad_scale;
  return r;
}

lora_status_t run_stats(lora_dtype_t dtype, const RowArgs &r, cudaStream_t st) {
  if (r.T == 0) return LORA_OK;
  if (dtype == LORA_BF16)
    LORA_CUDA(launch(stats_kernel<__nv_bfloat16>, dim3((unsigned)r.T), dim3(kRowThreads), 0, st, 1, true, r));
  else
    LORA_CUDA(launch(stats_kernel<float>, dim3((unsigned)r.T), dim3(kRowThreads), 0, st, 1, true, r));
  return LORA_OK;
}

lora_status_t run_grad(lora_dtype_t dtype, const RowArgs &r, cudaStream_t st) {
  if (r.T == 0 || r.V == 0) return LORA_OK;
  if (dtype == LORA_BF16)
    LORA_CUDA(launch(grad_kernel<__nv_bfloat16>, dim3((unsigned)r.T), dim3(kRowThreads), 0, st, 1, true, r));
  else
    LORA_CUDA(launch(grad_kernel<float>, dim3((unsigned)r.T), dim3(kRowThreads), 0, st, 1, true, r));
  return LORA_OK;
}

int64_t token_blocks(int64_t T) { return ceil_div(T, kPairThreads); }

}  // namespace

// ----------------------------------------------------------------------------- host side
size_t preference_ws_bytes(int64_t T, int64_t) { return ws_round(8 * T) + ws_round(4 * T) + ws_round(4); }
size_t policy_ws_bytes(int64_t T) {
  return ws_round(8 * T) + ws_round(4 * T) + ws_round(4) + ws_round(24 * token_blocks(T));
}

lora_status_t token_logps(const LossArgs &a, float *stats, cudaStream_t st) {
  RowArgs r = row_args(a);
  r.stats = reinterpret_cast<float2 *>(stats);
  return run_stats(a.dtype, r, st);
}

lora_status_t token_logps_backward(const LossArgs &a, const float *stats, const float *dlogps, cudaStream_t st) {
  RowArgs r = row_args(a);
  r.stats = reinterpret_cast<float2 *>(const_cast<float *>(stats));
  r.coef = const_cast<float *>(dlogps);
  return run_grad(a.dtype, r, st);
}

lora_status_t preference_loss(const LossArgs &a, const PreferenceArgs &p, void *ws, size_t ws_bytes,
                              cudaStream_t st) {
  if (p.P == 0) LORA_CUDA(cudaMemsetAsync(p.loss, 0, sizeof(float), st));
  WsCarver c(ws, ws_bytes);
  RowArgs r = row_args(a);
  float *coef = nullptr;
  if (a.T > 0) {
    r.stats = static_cast<float2 *>(c.take(8 * a.T));
    coef = static_cast<float *>(c.take(4 * a.T));
  }
  r.ticket = static_cast<unsigned *>(c.take(4));
  if (r.ticket == nullptr || (a.T > 0 && coef == nullptr)) return LORA_ERR_WORKSPACE;
  r.coef = coef;
  if (a.T == 0)
    LORA_CUDA(cudaMemsetAsync(r.ticket, 0, sizeof(unsigned), st));
  else
    LORA_TRY(run_stats(a.dtype, r, st));
  if (p.P > 0)
    LORA_CUDA(launch(pairs_kernel, dim3((unsigned)p.P), dim3(kPairThreads), 0, st, 1, true, p, a.T, a.V, a.labels,
                     (const float *)a.logps, a.dlogits ? coef : (float *)nullptr, r.ticket));
  return a.dlogits ? run_grad(a.dtype, r, st) : LORA_OK;
}

lora_status_t policy_loss(const LossArgs &a, const PolicyArgs &p, void *ws, size_t ws_bytes, cudaStream_t st) {
  if (a.T == 0) {
    LORA_CUDA(cudaMemsetAsync(p.metrics, 0, 3 * sizeof(float), st));
    return LORA_OK;
  }
  WsCarver c(ws, ws_bytes);
  RowArgs r = row_args(a);
  r.stats = static_cast<float2 *>(c.take(8 * a.T));
  r.coef = static_cast<float *>(c.take(4 * a.T));
  r.ticket = static_cast<unsigned *>(c.take(4));
  const int64_t blocks = token_blocks(a.T);
  double *part = static_cast<double *>(c.take(24 * blocks));
  if (part == nullptr) return LORA_ERR_WORKSPACE;
  LORA_TRY(run_stats(a.dtype, r, st));
  LORA_CUDA(launch(tokens_kernel, dim3((unsigned)blocks), dim3(kPairThreads), 0, st, 1, true, p, a.T, a.V, a.labels,
                   (const float *)a.logps, a.dlogits ? r.coef : (float *)nullptr, part, r.ticket));
  return a.dlogits ? run_grad(a.dtype, r, st) : LORA_OK;
}

lora_status_t scale_gradient(lora_dtype_t dtype, int64_t T, int64_t V, void *x, int64_t ldx, const float *factor,
                             cudaStream_t st) {
  if (T == 0 || V == 0) return LORA_OK;
  if (dtype == LORA_BF16)
    LORA_CUDA(launch(scale_kernel<__nv_bfloat16>, dim3((unsigned)T), dim3(kRowThreads), 0, st, 1, true,
                     (__nv_bfloat16 *)x, ldx, V, factor));
  else
    LORA_CUDA(launch(scale_kernel<float>, dim3((unsigned)T), dim3(kRowThreads), 0, st, 1, true, (float *)x, ldx, V,
                     factor));
  return LORA_OK;
}

}  // namespace lora
