// distill.cu -- the divergence of a model's rows from a teacher's record of its most
// probable tokens, with the gradient (include/lora_train.h).
//
// Mathematics.  The record lists tokens j with ln q_j, and perhaps the mass q_r that
// the teacher leaves to all others.  With a_j = ln p_j - ln q_j and p_r the student's
// mass outside the list (summed by itself: 1 - sum p_j would cancel for a sure student)
//     forward  L = -sum q_j a_j [- q_r a_r],   d L / d z_v = p_v Q - q_v,
//              and for a token outside the list p_v Q [- q_r p_v / p_r];  Q = sum q
//     reverse  L = sum p_j a_j [+ p_r a_r],    d L / d z_v = p_v (a_v - L)   with the rest,
//              p_v (a_v + 1 - L - P) and outside the list -p_v (L + P) without;  P = sum p_j
// So whatever the form, a token outside the list has f exp(z_v), one f for its row, and
// at most LORA_TOP_MAX tokens have a value of their own.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "f32x2.cuh"
#include "host_common.h"
#include "rows.cuh"
#include "sum2.cuh"
#include "top.h"

namespace lora {
namespace {

constexpr int kMaxTop = LORA_TOP_MAX;
constexpr int kEach = kMaxTop / 32;      // listed tokens of a lane

struct Distill {
  const void *logits;
  int64_t ldl;
  const int64_t *ids;
  const float *teacher, *rest, *weights;
  int64_t T, V;
  int K;
  bool reverse;
  Scale scale;
  float *row_loss;
  void *dlogits;
  int64_t lddl;
  float grad_scale;
};

__device__ __forceinline__ float warp_sum_f(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A row's record, the listed tokens over the lanes of a warp: place i of lane l is
// entry i * 32 + l.  id -1: no token (out of range, or listed before).
struct Record {
  int id[kEach];
  float z[kEach], lnq[kEach];      // the student's logit, the teacher's log-probability
};

// What a row's loss and gradient come to, by a warp, from the sums over the tokens that
// are not listed (m, s).  dz: c times the listed tokens' gradient; f: what exp((x - m) k)
// of all others is multiplied by.
struct RowTerms {
  float loss, f;
  float dz[kEach];
};
__device__ __forceinline__ RowTerms row_terms(const Distill &a, const Record &r, float ln_qr, float m, float s, float c) {
  const float k = a.scale.k;
  float top = kNegInf;
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (r.id[i] >= 0) top = fmaxf(top, r.z[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float M = fmaxf(top, m), ref = ref_of(M);
  float e[kEach], sum = 0.f;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    e[i] = r.id[i] >= 0 ? ex2((r.z[i] - ref) * k) : 0.f;
    sum += e[i];
  }
  const float rest = s * ex2((m - ref) * k), S = warp_sum_f(sum) + rest, ln_S = logf(S);
  const float p_r = rest / S, ln_pr = a.scale.gap(m, ref) + logf(s) - ln_S;
  float L = 0.f, Q = 0.f, P = 0.f, p[kEach], q[kEach], gap[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const bool there = r.id[i] >= 0;
    p[i] = e[i] / S;
    q[i] = there ? expf(r.lnq[i]) : 0.f;
    gap[i] = a.scale.gap(r.z[i], ref) - ln_S - r.lnq[i];
    if (!there) {
      p[i] = gap[i] = 0.f;
    } else if (a.reverse) {
      if (p[i] == 0.f) gap[i] = 0.f;      // no 0 * infinity
      L += p[i] * gap[i];
      P += p[i];
    } else {
      if (q[i] != 0.f) L -= q[i] * gap[i];
      Q += q[i];
    }
  }
  L = warp_sum_f(L);
  float F;      // the mass that the gradient leaves outside the list
  if (a.reverse) {
    if (a.rest) {
      const float gap_r = p_r == 0.f ? 0.f : ln_pr - ln_qr;
      L += p_r * gap_r;
      F = p_r * (gap_r - L);
      P = 1.f;
    } else {
      P = warp_sum_f(P);
      F = -p_r * (L + P);
    }
  } else {
    Q = warp_sum_f(Q);
    F = 0.f;
    if (a.rest) {
      const float qr = expf(ln_qr);
      if (qr != 0.f) L -= qr * (ln_pr - ln_qr);
      Q += qr;
      F = -qr;
    }
    F += p_r * Q;
  }
  RowTerms t;
  t.loss = L;
  t.f = s == 0.f ? 0.f : c * F / s;      // s is 0: nothing outside the list has any probability
  if (!(S > 0.f)) t.f = NAN;             // nor inside: no distribution
#pragma unroll
  for (int i = 0; i < kEach; ++i) t.dz[i] = c * (a.reverse ? p[i] * (gap[i] + 1.f - L - P) : p[i] * Q - q[i]);
  return t;
}

constexpr int kThreads = 256;

template <typename E, int kThreads>
__global__ void __launch_bounds__(kThreads) distill_kernel(Distill a, int C, int slice) {
  constexpr int kWarps = kThreads / 32, N = Elem<E>::kVec, U = 4;
  __shared__ int ids[kMaxTop], next[kMaxTop], head[kThreads];
  __shared__ float logit[kMaxTop], dz[kMaxTop];
  __shared__ float2 sh[kWarps], pair[kMaxCluster];
  __shared__ unsigned edges;                     // listed ones among the ragged ends
  __shared__ float weight, m_of, f_of;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = blockIdx.x / C;
  const int rank = (int)(blockIdx.x % C), tid = threadIdx.x, lane = lane_id(), warp = tid >> 5, K = a.K, V = (int)a.V;
  const E *row = static_cast<const E *>(a.logits) + t * a.ldl;
  E *out = static_cast<E *>(a.dlogits) + t * a.lddl;
  const RowSpan<E> sp(row, V);
  const int v0 = min(rank * slice, sp.vecs), v1 = min(v0 + slice, sp.vecs), tail = sp.tail();
  const int e0 = rank == 0 ? 0 : sp.head + v0 * N, e1 = rank == C - 1 ? V : sp.head + v1 * N;
  const float k = a.scale.k;
  if (tid < kMaxTop) {
    const int64_t id = tid < K ? a.ids[t * K + tid] : -1;
    ids[tid] = id >= 0 && id < V ? (int)id : -1;
  }
  if (C > 1) cluster_arrive();                   // no block is written to before it runs
  if (tid == 0) {
    weight = a.weights ? a.weights[t] : 1.f;     // read once for the block
    edges = 0;
  }
  head[tid] = -1;
  __syncthreads();
  int mark = tid < kMaxTop ? ids[tid] : -1;
  for (int j = 0; j < tid && mark >= 0; ++j)
    if (ids[j] == mark) mark = -1;               // listed before
  const float w = weight;
  const bool counts = __syncthreads_or(mark >= 0) && w != 0.f;
  if (tid < kMaxTop) {
    ids[tid] = mark;
    logit[tid] = mark >= 0 && counts ? Elem<E>::load(row + mark) : 0.f;
  }
  if (mark >= e0 && mark < e1) {
    if (mark < sp.head) {
      atomicOr(&edges, 1u << mark);
    } else if (mark >= tail) {
      atomicOr(&edges, 1u << (16 + mark - tail));
    } else {
      const int owner = ((mark - sp.head) / N - v0) % kThreads;
      next[tid] = atomicExch(&head[owner], tid);
    }
  }
  __syncthreads();
  float m = kNegInf, s = 0.f;
  if (counts) {
    const uint4 *src = reinterpret_cast<const uint4 *>(row + sp.head);
    const int mine = head[tid];
    uint64_t s2 = 0;
    for (int i = v0 + tid; i < v1; i += U * kThreads) {
      uint4 q[U];
#pragma unroll
      for (int u = 0; u < U; ++u) q[u] = i + u * kThreads < v1 ? src[i + u * kThreads] : Elem<E>::lowest();
      for (int j = mine; j >= 0; j = next[j]) {
        const int place = ids[j] - sp.head, p = place / N - i;
        if (p < 0 || p >= U * kThreads) continue;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (p == u * kThreads) Elem<E>::strike(q[u], place % N);
      }
      absorb<E, U>(m, s2, q, k);
    }
    const float2 both = unpk2(s2);
    s = both.x + both.y;
    if (rank == 0 && tid < sp.head && !(edges >> tid & 1u)) absorb_one(m, s, Elem<E>::load(row + tid), k);
    if (rank == C - 1 && tid < V - tail && !(edges >> (16 + tid) & 1u)) absorb_one(m, s, Elem<E>::load(row + tail + tid), k);
  }
  block_merge<kWarps>(m, s, k, sh);
  if (C > 1) {
    __syncwarp();
    cluster_wait();
    if (warp == 0 && lane < C) st_dsmem_f2(&pair[rank], lane, make_float2(m, s));
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (warp == 0) {
      const float2 v = lane < C ? pair[lane] : make_float2(kNegInf, 0.f);
      m = v.x;
      s = v.y;
      warp_merge(m, s, k);
    }
  }
  if (!counts) {
    if (rank == 0 && tid == 0) a.row_loss[t] = 0.f;
    if (a.dlogits) zero_span<E, kThreads>(out, e0, e1, tid);
    return;
  }
  if (warp == 0) {
    Record r;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int j = i * 32 + lane;
      r.id[i] = ids[j];
      r.z[i] = logit[j];
      r.lnq[i] = r.id[i] >= 0 ? a.teacher[t * K + j] : 0.f;
    }
    const RowTerms x = row_terms(a, r, a.rest ? a.rest[t] : 0.f, m, s, w * a.grad_scale * a.scale.hi);
#pragma unroll
    for (int i = 0; i < kEach; ++i) dz[i * 32 + lane] = x.dz[i];
    if (lane == 0) {
      m_of = ref_of(m);
      f_of = x.f;
      if (rank == 0) a.row_loss[t] = x.loss;
    }
  }
  __syncthreads();
  if (!a.dlogits) return;
  const RowGrad g = {m_of, k, 0.f, f_of};
  const bool same = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(row)) & 15u) == 0;
  if (!same) {
    grad_words<E, kThreads>(out, row, e0, e1, -1, g);
  } else {
    const uint4 *src = reinterpret_cast<const uint4 *>(row + sp.head);
    uint4 *dst = reinterpret_cast<uint4 *>(out + sp.head);
    for (int i = v0 + tid; i < v1; i += kThreads) __stcs(dst + i, g.piece<E>(src[i]));
    auto one = [&](int j) { Elem<E>::store(out + j, g(Elem<E>::load(row + j))); };
    if (rank == 0 && tid < sp.head) one(tid);
    if (rank == C - 1 && tid < V - tail) one(tail + tid);
  }
  __syncthreads();                               // the listed tokens' places come after the pieces
  if (mark >= e0 && mark < e1) Elem<E>::store(out + mark, dz[tid]);
}

// loss = sum of weights * row_loss, in a fixed order.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) loss_kernel(const float *row_loss, const float *weights, int64_t T,
                                                           float *loss) {
  __shared__ Sum2 sh[kSumThreads / 32];
  pdl_wait();
  Sum2 s[1];
#pragma unroll 2
  for (int64_t t = threadIdx.x; t < T; t += kSumThreads) {
    const float w = weights ? weights[t] : 1.f;
    if (w != 0.f) s[0].add(w * row_loss[t]);
  }
  block_sums<kSumThreads / 32, 1>(s, sh);
  if (threadIdx.x == 0) *loss = s[0].value();
}

int slice_of(int64_t bytes, int parts) { return (int)std::max<int64_t>(8, round_up(ceil_div(bytes / 16, parts), 8)); }

template <typename E>
cudaError_t launch_distill(const Distill &r, int64_t bytes, cudaStream_t st) {
  const int64_t sms = num_sms();
  int c = 1;
  if (2 * r.T < sms)
    c = (int)std::min<int64_t>({std::max<int64_t>(1, 4 * sms / r.T), std::max<int64_t>(1, bytes / (4 << 10)), kMaxCluster});
  return launch(distill_kernel<E, kThreads>, dim3((unsigned)(r.T * c)), dim3(kThreads), 0, st, c, true, r, c,
                slice_of(bytes, c));
}

}  // namespace

// ----------------------------------------------------------------------------- host side
int read_clear_error_distill() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)) != cudaSuccess) return -1;
  if (v) cudaMemcpyToSymbol(g_device_error, &z, sizeof(int));
  return v;
}

lora_status_t distill_loss(const DistillArgs &a, cudaStream_t st) {
  if (a.T == 0) {
    LORA_CUDA(cudaMemsetAsync(a.loss, 0, sizeof(float), st));
    return LORA_OK;
  }
  Distill r{};
  r.logits = a.logits; r.ldl = a.ldl; r.ids = a.ids; r.teacher = a.teacher; r.rest = a.rest; r.weights = a.weights;
  r.T = a.T; r.V = a.V; r.K = a.K; r.reverse = a.reverse; r.scale = Scale::of(a.temperature); r.row_loss = a.row_loss;
  r.dlogits = a.dlogits; r.lddl = a.lddl; r.grad_scale = a.grad_scale;
  LORA_CUDA(a.dtype == LORA_BF16 ? launch_distill<__nv_bfloat16>(r, a.V * 2, st) : launch_distill<float>(r, a.V * 4, st));
  LORA_CUDA(launch(loss_kernel, dim3(1), dim3(kSumThreads), 0, st, 1, true, (const float *)a.row_loss, a.weights, a.T,
                   a.loss));
  return LORA_OK;
}

}  // namespace lora
