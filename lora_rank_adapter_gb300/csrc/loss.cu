// loss.cu -- log-probabilities of labels, the preference loss and the clipped
// policy loss over rows of logits, with their gradients (include/lora_train.h).
//
// Mathematics.  With z = x / temperature, m = max z and S = sum exp(z - m), a
// row's logp is z_label - m - ln S, and for a coefficient c = d loss / d logp its
// gradient is d_v = (c / temperature) ((v == label) - exp(z_v - m) / S).  exp is
// 2^((x - m) k), k = log2(e) / temperature: x - m first, so that rows at the end
// of the type's range (masks of its lowest value) neither overflow nor cancel.
//
// Bytes decide: one or two exponentials and some ten operations an element, against
// 6.8 TB/s (the measured copy rate) and about 4.6 T exponentials a second.
//   stats_kernel    one reading of a row: (m, S) and logp;
//   grad_kernel     its gradient from (m, S) and c, the row read again;
//   held_kernel     the policy loss, whose c needs the row only: the row is held in
//                   the shared memory of a cluster and read once;
//   short_kernel    each of the three for rows of up to 32 KB, held in registers;
//   pairs_kernel    the preference loss, whose c needs every row of a pair: between
//                   a pass of statistics and one of gradients, 3 N bytes;
//   metrics_kernel, tokens_kernel   sums over, and coefficients of, T tokens.
#include <math.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "f32x2.cuh"
#include "host_common.h"
#include "loss.h"
#include "sum2.cuh"

namespace lora {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint64_t ex2_2(uint64_t v) {
  const float2 f = unpk2(v);
  return pk2(ex2(f.x), ex2(f.y));
}

template <typename E>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float load(const float *p) { return *p; }
  static __device__ __forceinline__ void store(float *p, float v) { *p = v; }
  // a 16-byte piece as kVec / 2 pairs, and its largest value
  static __device__ __forceinline__ void pairs(const uint4 &q, uint64_t *v) {
    v[0] = pk2(__uint_as_float(q.x), __uint_as_float(q.y));
    v[1] = pk2(__uint_as_float(q.z), __uint_as_float(q.w));
  }
  static __device__ __forceinline__ uint4 pack_pairs(const uint64_t *v) {
    const float2 a = unpk2(v[0]), b = unpk2(v[1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  }
  template <int U>
  static __device__ __forceinline__ float largest(const uint4 (&q)[U]) {
    float b = kNegInf;
#pragma unroll
    for (int u = 0; u < U; ++u)
      b = fmaxf(b, fmaxf(fmaxf(__uint_as_float(q[u].x), __uint_as_float(q[u].y)),
                         fmaxf(__uint_as_float(q[u].z), __uint_as_float(q[u].w))));
    return b;
  }
  static __device__ __forceinline__ uint4 lowest() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
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
  static __device__ __forceinline__ void pairs(const uint4 &q, uint64_t *v) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pk2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 pack_pairs(const uint64_t *v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpk2(v[i]);
      w[i] = pack_bf16(f.x, f.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  template <int U>
  static __device__ __forceinline__ float largest(const uint4 (&q)[U]) {
    auto two = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); };
    __nv_bfloat162 b = two(0xff80ff80u);
#pragma unroll
    for (int u = 0; u < U; ++u)
      b = __hmax2(b, __hmax2(__hmax2(two(q[u].x), two(q[u].y)), __hmax2(two(q[u].z), two(q[u].w))));
    const float2 f = __bfloat1622float2(b);
    return fmaxf(f.x, f.y);
  }
  static __device__ __forceinline__ uint4 lowest() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
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
// whole 16-byte pieces, and the rest.  (V <= 2^30: places within a row are ints.)
template <typename E>
struct RowSpan {
  int head, vecs;
  __device__ __forceinline__ RowSpan(const E *row, int V) {
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
    head = (int)(((16u - off) & 15u) / sizeof(E));
    if (head > V) head = V;
    vecs = (V - head) / Elem<E>::kVec;
  }
  __device__ __forceinline__ int tail() const { return head + vecs * Elem<E>::kVec; }
};

// Running (m, s): the largest value seen and s = sum exp((x - m) * inv_t), with
// k = inv_t * log2(e).  While m is minus infinity nothing but minus infinity has
// been seen and s is zero; the reference is then 0 instead of m, so that
// exp(-inf - ref) is 0 and not NaN.
__device__ __forceinline__ float ref_of(float m) { return m == kNegInf ? 0.f : m; }

// One element into the running pair.
__device__ __forceinline__ void absorb_one(float &m, float &s, float v, float k) {
  const float mm = fmaxf(m, v), r = ref_of(mm);
  s = s * ex2((m - r) * k) + ex2((v - r) * k);
  m = mm;
}

// U 16-byte pieces into a running maximum and a pair of partial sums.  The
// reference moves once for all of them.
template <typename E, int U>
__device__ __forceinline__ void absorb(float &m, uint64_t &s, const uint4 (&q)[U], float k) {
  const float mm = fmaxf(m, Elem<E>::largest(q)), r = ref_of(mm), f = ex2((m - r) * k);
  const uint64_t r2 = pk2(-r, -r), k2 = pk2(k, k);
  m = mm;
  s = mul2(s, pk2(f, f));
  uint64_t t = 0;      // a second chain of sums: (0, 0)
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint64_t v[Elem<E>::kVec / 2];
    Elem<E>::pairs(q[u], v);
#pragma unroll
    for (int j = 0; j < Elem<E>::kVec / 2; ++j) {
      const uint64_t e = ex2_2(mul2(add2(v[j], r2), k2));
      if (j & 1) t = add2(t, e); else s = add2(s, e);
    }
  }
  s = add2(s, t);
}

// Pieces [from, to) of a row, kThreads threads, U loads of each in flight.
template <typename E, int kThreads, int U>
__device__ __forceinline__ void absorb_span(float &m, uint64_t &s, const uint4 *p, int from, int to, float k) {
  int i = from + (int)threadIdx.x;
  for (; to - i > (U - 1) * kThreads; i += U * kThreads) {
    uint4 q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) q[u] = p[i + u * kThreads];
    absorb<E, U>(m, s, q, k);
  }
  if (U > 1 && i < to) {
    uint4 q[U > 1 ? U - 1 : 1];
#pragma unroll
    for (int u = 0; u < U - 1; ++u) q[u] = to - i > u * kThreads ? p[i + u * kThreads] : Elem<E>::lowest();
    absorb<E, U - 1>(m, s, q, k);
  }
}

// (m, s) of the warp's lanes: the largest m, then one rescaling of each s.
__device__ __forceinline__ void warp_merge(float &m, float &s, float k) {
  float mm;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(mm) : "f"(m));
  s *= ex2((m - ref_of(mm)) * k);
  m = mm;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
}

// (m, s) of the whole block, known to the threads of warp 0.
template <int kWarps>
__device__ __forceinline__ void block_merge(float &m, float &s, float k, float2 *sh) {
  warp_merge(m, s, k);
  if (lane_id() == 0) sh[threadIdx.x >> 5] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x >= 32) return;
  const float2 v = threadIdx.x < kWarps ? sh[threadIdx.x] : make_float2(kNegInf, 0.f);
  m = v.x;
  s = v.y;
  warp_merge(m, s, k);
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
  float *coef;         // d loss / d logp: zeroed by the statistics pass (NULL: none), read by the gradient pass
  unsigned *ticket;    // zeroed by the statistics pass (NULL: none)
  void *dlogits;
  int64_t lddl;
  float grad_scale;
};

constexpr int kMaxCluster = 8;

// (m, s) of the blocks of a cluster, by warp 0 of each, once.  Each block writes
// its pair to all the others; `ready` counts one arrival from each.  The caller
// has let the cluster arrive and wait after `ready` was set up, and lets no block
// leave before all have sent.
struct ClusterSlots {
  uint64_t ready;
  float2 pair[kMaxCluster];
  int64_t label;       // of the block's row, read once for all its threads
};
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_dsmem_f2(const void *local_ptr, uint32_t cta, float2 v) {
  uint32_t local = smem_u32(local_ptr), remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(cta));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote), "f"(v.x), "f"(v.y) : "memory");
}
// A pair stored to another block of the cluster, its bytes completing `bar` there
// (only in a kernel that was launched as clusters).
__device__ __forceinline__ void st_async_f2(const void *local_ptr, const uint64_t *local_bar, uint32_t cta, float2 v) {
  uint32_t p, b;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(smem_u32(local_ptr)), "r"(cta));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(smem_u32(local_bar)), "r"(cta));
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(p),
               "f"(v.x), "f"(v.y), "r"(b)
               : "memory");
}
__device__ __forceinline__ void cluster_send(float m, float s, int rank, int C, ClusterSlots *slots) {
  const int lane = lane_id();
  if (lane < C) {
    st_dsmem_f2(&slots->pair[rank], lane, make_float2(m, s));
    mbar_arrive_remote(&slots->ready, lane);
  }
  __syncwarp();
}
// False: the wait ran out.
__device__ __forceinline__ bool cluster_merge(float &m, float &s, float k, int C, ClusterSlots *slots) {
  const int lane = lane_id();
  if (!__all_sync(0xffffffffu, mbar_wait<true>(&slots->ready, 0))) return false;
  const float2 v = lane < C ? slots->pair[lane] : make_float2(kNegInf, 0.f);
  m = v.x;
  s = v.y;
  warp_merge(m, s, k);
  return true;
}

// The statistics of a row, read once from global memory by the C blocks of a
// cluster, a slice of `slice` 16-byte pieces each.  Bound by the reading: 5462 rows
// of 128256 bf16 (1.4 GB) take 213 us, 6.6 TB/s, four loads of a thread in flight.
// (Plain loads: through TMA copies into shared memory the same took 270 us.)  An
// ignored row is not read, but its blocks meet all the same, and a block whose wait
// ran out stays for the others: no block leaves before all have sent to it, whatever
// each has seen of labels that another stream may be writing.
template <typename E, int kThreads>
__global__ void __launch_bounds__(kThreads) stats_kernel(RowArgs a, int C, int slice) {
  __shared__ float2 sh[kThreads / 32];
  __shared__ ClusterSlots slots;
  pdl_wait();
  pdl_launch_dependents();      // the next kernel's blocks may take their places and wait there
  const int64_t t = blockIdx.x / C;
  const int rank = (int)(blockIdx.x % C), tid = threadIdx.x;
  int64_t label;
  if (C > 1) {
    if (tid == 0) {
      mbar_init(&slots.ready, C);
      fence_barrier_init();
      slots.label = a.labels[t];
    }
    __syncthreads();
    cluster_arrive();
    label = slots.label;
  } else {
    label = a.labels[t];
  }
  if (rank == 0 && tid == 0) {
    if (a.coef) a.coef[t] = 0.f;
    if (a.ticket && t == 0) *a.ticket = 0;
  }
  const bool counts = label >= 0 && label < a.V;
  const float k = a.inv_t * kLog2e;
  float picked = 0.f, m = kNegInf, s = 0.f;
  if (counts) {
    const E *row = static_cast<const E *>(a.logits) + t * a.ldl;
    const RowSpan<E> sp(row, (int)a.V);
    const int v0 = min(rank * slice, sp.vecs), v1 = min(v0 + slice, sp.vecs), tail = sp.tail();
    if (rank == 0 && tid == 0) picked = Elem<E>::load(row + label);
    uint64_t s2 = 0;
    absorb_span<E, kThreads, 4>(m, s2, reinterpret_cast<const uint4 *>(row + sp.head), v0, v1, k);
    const float2 both = unpk2(s2);
    s = both.x + both.y;
    if (rank == C - 1) {      // the ragged ends
      if (tid < sp.head) absorb_one(m, s, Elem<E>::load(row + tid), k);
      if (tid < (int)a.V - tail) absorb_one(m, s, Elem<E>::load(row + tail + tid), k);
    }
    block_merge<kThreads / 32>(m, s, k, sh);
  }
  bool whole = true;
  if (C > 1) {
    cluster_wait();
    if (tid < 32) cluster_send(m, s, rank, C, &slots);
    cluster_arrive();
    if (tid < 32) whole = cluster_merge(m, s, k, C, &slots);
  }
  if (rank == 0 && tid == 0 && whole) {
    a.logps[t] = counts ? (picked - m) * a.inv_t - logf(s) : 0.f;
    if (a.stats) a.stats[t] = counts ? make_float2(m, s) : make_float2(0.f, 1.f);
  }
  if (C > 1) {
    __syncwarp();
    cluster_wait();      // all have sent
  }
}

// Zeros over elements [from, to) of an output row.
template <typename E, int kThreads>
__device__ __forceinline__ void zero_span(E *out, int from, int to, int tid) {
  E *o = out + from;
  const RowSpan<E> so(o, to - from);
  if (tid < so.head) Elem<E>::store(o + tid, 0.f);
  uint4 *body = reinterpret_cast<uint4 *>(o + so.head);
  for (int i = tid; i < so.vecs; i += kThreads) __stcs(body + i, make_uint4(0, 0, 0, 0));
  if (tid < to - from - so.tail()) Elem<E>::store(o + so.tail() + tid, 0.f);
}

// A row's gradient d_v = c [v == label] + f exp(z_v - m), f = -c / S.
struct RowGrad {
  float m, k, c, f;
  __device__ __forceinline__ float operator()(float v) const { return f * ex2((v - m) * k); }
  // a 16-byte piece, as if it did not hold the label
  template <typename E>
  __device__ __forceinline__ uint4 piece(const uint4 &q) const {
    constexpr int N = Elem<E>::kVec;
    uint64_t v[N / 2];
    Elem<E>::pairs(q, v);
    const uint64_t m2 = pk2(-m, -m), k2 = pk2(k, k), f2 = pk2(f, f);
#pragma unroll
    for (int j = 0; j < N / 2; ++j) v[j] = mul2(ex2_2(mul2(add2(v[j], m2), k2)), f2);
    return Elem<E>::pack_pairs(v);
  }
};

// Elements [e0, e1) of the output row where it sits at another offset to a
// 16-byte boundary than the logits: 4-byte words of the output, their elements
// read one by one (src: element i of the row at src[i]).
template <typename E, int kThreads>
__device__ __forceinline__ void grad_words(E *out, const E *src, int e0, int e1, int label, const RowGrad &g) {
  auto one = [&](int i) { return g(Elem<E>::load(src + i)) + (i == label ? g.c : 0.f); };
  const int tid = threadIdx.x;
  if (sizeof(E) == 4) {
#pragma unroll 4
    for (int i = e0 + tid; i < e1; i += kThreads) Elem<E>::store(out + i, one(i));
  } else {
    const int w0 = e0 + (int)((reinterpret_cast<uintptr_t>(out + e0) >> 1) & 1);      // the first whole word
    const int words = e1 > w0 ? (e1 - w0) / 2 : 0;
#pragma unroll 4
    for (int i = tid; i < words; i += kThreads)
      __stcs(reinterpret_cast<unsigned *>(out + w0) + i, pack_bf16(one(w0 + 2 * i), one(w0 + 2 * i + 1)));
    if (tid == 0 && w0 > e0 && e0 < e1) Elem<E>::store(out + e0, one(e0));
    if (tid == 1 && w0 + 2 * words < e1) Elem<E>::store(out + e1 - 1, one(e1 - 1));
  }
}

// The gradient from saved statistics: `parts` blocks a row, a slice of `slice`
// 16-byte pieces each.  Rows go last to first: the pass over the logits before
// this one has left its last rows in L2.  Bound by its bytes: 7792 rows of 128256
// bf16, 30 % of them ignored (1.4 GB read, 2 GB written), take 497 us, 6.8 TB/s.
template <typename E>
__global__ void __launch_bounds__(kRowThreads) grad_kernel(RowArgs a, int parts, int slice) {
  pdl_wait();
  const int64_t t = a.T - 1 - blockIdx.x / parts;
  const int rank = (int)(blockIdx.x % parts);
  const int64_t label = a.labels[t];
  const float c = a.coef[t] * a.grad_scale * a.inv_t;
  const float2 st = a.stats[t];
  E *out = static_cast<E *>(a.dlogits) + t * a.lddl;
  const E *row = static_cast<const E *>(a.logits) + t * a.ldl;
  const RowSpan<E> sp(row, (int)a.V);
  constexpr int N = Elem<E>::kVec;
  const int tid = threadIdx.x, V = (int)a.V;
  const int v0 = min(rank * slice, sp.vecs), v1 = min(v0 + slice, sp.vecs), tail = sp.tail();
  const int e0 = rank == 0 ? 0 : sp.head + v0 * N, e1 = rank == parts - 1 ? V : sp.head + v1 * N;
  if (label < 0 || label >= V || c == 0.f) {
    zero_span<E, kRowThreads>(out, e0, e1, tid);
    return;
  }
  const RowGrad g = {st.x, a.inv_t * kLog2e, c, -c / st.y};
  const int mark = (int)label;
  if (((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(row)) & 15u) != 0) {
    grad_words<E, kRowThreads>(out, row, e0, e1, mark, g);
    return;
  }
  const uint4 *src = reinterpret_cast<const uint4 *>(row + sp.head);
  uint4 *dst = reinterpret_cast<uint4 *>(out + sp.head);
  // the label's element goes after its piece, by the thread that wrote that
  const int place = mark - sp.head - v0 * N;
  const bool mine = place >= 0 && place < (v1 - v0) * N && place / N % kRowThreads == tid;
  const float picked = mine ? Elem<E>::load(row + mark) : 0.f;
  int i = v0 + tid;
  for (; v1 - i > 3 * kRowThreads; i += 4 * kRowThreads) {
    uint4 q[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) q[u] = src[i + u * kRowThreads];
#pragma unroll
    for (int u = 0; u < 4; ++u) __stcs(dst + i + u * kRowThreads, g.piece<E>(q[u]));
  }
  for (; i < v1; i += kRowThreads) __stcs(dst + i, g.piece<E>(src[i]));
  if (mine) Elem<E>::store(out + mark, g(picked) + c);
  auto one = [&](int j) { Elem<E>::store(out + j, g(Elem<E>::load(row + j)) + (j == mark ? c : 0.f)); };
  if (rank == 0 && tid < sp.head) one(tid);
  if (rank == parts - 1 && tid < V - tail) one(tail + tid);
}

// ----------------------------------------------------------------------------- per-token steps
constexpr int kPairThreads = 256;

// ln sigmoid(h) = min(h, 0) - ln(1 + exp(-|h|)), free of overflow and of cancellation
__device__ __forceinline__ float log_sigmoid(float h) { return fminf(h, 0.f) - log1pf(expf(-fabsf(h))); }

// One block per pair: both sequences' sums (in two fp32 parts: their difference is
// what counts), the pair's loss, and each of its tokens' d loss / d logp.  The last
// block takes the mean.  A chain of short dependent steps: what can be on its way
// together is.
__global__ void __launch_bounds__(kPairThreads) pairs_kernel(PreferenceArgs p, int64_t T, int64_t V,
                                                             const int64_t *labels, const float *logps, float *coef,
                                                             unsigned *ticket) {
  __shared__ Sum2 sh[2 * (kPairThreads / 32)], sh_n[2 * (kPairThreads / 32)];
  __shared__ float slope_of[2];
  __shared__ unsigned before;
  const int pair = blockIdx.x, tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int32_t *cu = p.cu;
  const int32_t edge[4] = {cu[pair], cu[pair + 1], cu[pair + p.P], cu[pair + p.P + 1]};
  const float ref = p.ref ? p.ref[pair] - p.ref[pair + p.P] : 0.f;
  int64_t lo[2], n[2];
  Sum2 sum[2], counted[2];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    lo[side] = min(max((int64_t)edge[2 * side], (int64_t)0), T);
    n[side] = max(min((int64_t)edge[2 * side + 1], T) - lo[side], (int64_t)0);
  }
  for (int64_t i = tid; i < max(n[0], n[1]); i += kPairThreads)
#pragma unroll
    for (int side = 0; side < 2; ++side)
      if (i < n[side]) {
        const int64_t t = lo[side] + i;
        sum[side].add(logps[t]);
        if (p.normalize) counted[side].add(labels[t] >= 0 && labels[t] < V ? 1.f : 0.f);
      }
  if (p.normalize) block_sums<kPairThreads / 32, 2>(counted, sh_n);
  block_sums<kPairThreads / 32, 2>(sum, sh);
  if (tid == 0) {
    float S[2], count[2];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      count[side] = p.normalize ? fmaxf(1.f, counted[side].value()) : 1.f;
      S[side] = sum[side].value() / count[side];
      p.seq_logps[pair + side * p.P] = S[side];
    }
    const float d = S[0] - S[1] - ref;
    float loss, slope;
    if (p.kind == LORA_PREF_SIGMOID) {
      const float h = p.beta * d;
      loss = -(1.f - p.smoothing) * log_sigmoid(h);
      if (p.smoothing > 0.f) loss -= p.smoothing * log_sigmoid(-h);      // no 0 * infinity at an infinite h
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
    p.pair_loss[pair] = loss;
    slope_of[0] = slope / (float)p.P / count[0];
    slope_of[1] = -slope / (float)p.P / count[1];
    if (gridDim.x == 1) {
      p.loss[0] = loss;
    } else {
      __threadfence();
      before = atomicAdd(ticket, 1u);
      __threadfence();
    }
  }
  __syncthreads();
  if (coef)
#pragma unroll
    for (int side = 0; side < 2; ++side)
      for (int64_t i = tid; i < n[side]; i += kPairThreads) coef[lo[side] + i] = slope_of[side];
  if (gridDim.x == 1 || before != gridDim.x - 1) return;
  Sum2 all[1];
  for (int i = tid; i < p.P; i += kPairThreads) all[0].add(__ldcg(p.pair_loss + i));
  block_sums<kPairThreads / 32, 1>(all, sh);
  if (tid == 0) p.loss[0] = all[0].value() / (float)p.P;
}

// A token's part of the policy loss: the terms of the three metrics, and its
// d loss / d logp.
struct PolicyRow {
  float A, w, old, ref;
};
__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs &p, int64_t t) {
  return {p.advantages[t], p.weights ? p.weights[t] : 1.f, p.old_logps ? p.old_logps[t] : 0.f,
          p.ref_logps ? p.ref_logps[t] : 0.f};
}
struct PolicyTerm {
  float loss, kl, clipped, coef;
};
__device__ __forceinline__ PolicyTerm policy_term(const PolicyArgs &p, const PolicyRow &in, float logp) {
  const float A = in.A, w = in.w;
  // on the policy itself r is 1, also for a label that is masked out (a NaN stays one)
  const float r = expf(p.old_logps ? logp - in.old : logp == kNegInf ? 0.f : logp - logp);
  const float hi = 1.f + p.clip_high, lo = 1.f - p.clip_low;
  const bool clipped = (A > 0.f && r > hi) || (A < 0.f && r < lo);
  float pg = -A * r, coef = -A * r;
  if (clipped) {
    pg = -A * (A > 0.f ? hi : lo);
    coef = 0.f;
  }
  float kl = 0.f;
  if (p.ref_logps) {
    const float d = in.ref - logp, e = expm1f(d);
    kl = e - d;
    coef -= p.kl_beta * e;
  }
  return {w * (pg + p.kl_beta * kl), w * kl, clipped ? w : 0.f, w * coef};
}

// The policy loss where a row does not fit on chip: the coefficients from the
// log-probabilities of the statistics pass.
__global__ void __launch_bounds__(kPairThreads) tokens_kernel(PolicyArgs p, int64_t T, int64_t V,
                                                              const int64_t *labels, const float *logps, float *coef) {
  pdl_wait();
  const int64_t t = blockIdx.x * (int64_t)kPairThreads + threadIdx.x;
  if (t >= T) return;
  coef[t] = labels[t] >= 0 && labels[t] < V ? policy_term(p, policy_row(p, t), logps[t]).coef : 0.f;
}

// ----------------------------------------------------------------------------- short rows
// A row of some KB is held in the registers of one warp, or of four that make up a
// block: its loads are all on their way at once, and no row waits for another.
// Statistics, policy loss or gradient of it in one go.
enum ShortMode { kShortStats, kShortPolicy, kShortGrad };

template <typename E, int kPieces, int kTeam, int kMode>
__global__ void __launch_bounds__(kTeam == 1 ? 256 : 32 * kTeam) short_kernel(RowArgs a, PolicyArgs p) {
  constexpr int kLanes = 32 * kTeam, kRows = kTeam == 1 ? 8 : 1, N = Elem<E>::kVec;
  __shared__ float2 sh[kTeam];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = blockIdx.x * (int64_t)kRows + threadIdx.x / kLanes;
  if (t >= a.T) return;                                  // whole teams
  const int tid = threadIdx.x % kLanes, V = (int)a.V;
  if (kMode == kShortStats && tid == 0) {
    if (a.coef) a.coef[t] = 0.f;
    if (a.ticket && t == 0) *a.ticket = 0;
  }
  const int64_t label = a.labels[t];
  E *out = static_cast<E *>(a.dlogits) + t * a.lddl;
  bool counts = label >= 0 && label < V;
  float c = 0.f, m = kNegInf, s = 0.f;
  if (kMode == kShortGrad) {
    const float2 st = a.stats[t];
    c = a.coef[t] * a.grad_scale * a.inv_t;
    m = st.x;
    s = st.y;
    counts = counts && c != 0.f;
  }
  if (!counts) {
    if (kMode != kShortGrad && tid == 0) {
      a.logps[t] = 0.f;
      if (kMode == kShortStats && a.stats) a.stats[t] = make_float2(0.f, 1.f);
    }
    if (kMode != kShortStats && a.dlogits) zero_span<E, kLanes>(out, 0, V, tid);
    return;
  }
  const int mark = (int)label;
  const E *row = static_cast<const E *>(a.logits) + t * a.ldl;
  const RowSpan<E> sp(row, V);
  const uint4 *src = reinterpret_cast<const uint4 *>(row + sp.head);
  uint4 q[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) q[u] = tid + u * kLanes < sp.vecs ? src[tid + u * kLanes] : Elem<E>::lowest();
  // the ragged ends, at most seven elements each
  const int tail = sp.tail();
  const bool at_head = tid < sp.head, at_tail = tid >= 16 && tid - 16 < V - tail;
  const int edge_at = at_head ? tid : tail + tid - 16;
  float edge = kNegInf;
  if (at_head || at_tail) edge = Elem<E>::load(row + edge_at);
  const float picked = Elem<E>::load(row + mark);
  const float k = a.inv_t * kLog2e;
  if (kMode != kShortGrad) {
    PolicyRow in;
    if (kMode == kShortPolicy) in = policy_row(p, t);
    uint64_t s2 = 0;
    constexpr int U = kPieces < 4 ? kPieces : 4;
#pragma unroll
    for (int u = 0; u < kPieces; u += U) {
      if (u * kLanes >= sp.vecs) break;
      uint4 some[U];
#pragma unroll
      for (int i = 0; i < U; ++i) some[i] = q[u + i];
      absorb<E, U>(m, s2, some, k);
    }
    const float2 both = unpk2(s2);
    s = both.x + both.y;
    if (edge != kNegInf) absorb_one(m, s, edge, k);
    warp_merge(m, s, k);
    // past this point the gradient may replace the row: all reads of it come before
    if (kTeam == 1) __syncwarp();
    if (kTeam > 1) {
      if (lane_id() == 0) sh[tid >> 5] = make_float2(m, s);
      __syncthreads();
      const float2 v = lane_id() < kTeam ? sh[lane_id() % kTeam] : make_float2(kNegInf, 0.f);
      m = v.x;
      s = v.y;
      warp_merge(m, s, k);
    }
    const float logp = (picked - m) * a.inv_t - logf(s);
    if (tid == 0) {
      a.logps[t] = logp;
      if (kMode == kShortStats && a.stats) a.stats[t] = make_float2(m, s);
    }
    if (kMode == kShortStats || a.dlogits == nullptr) return;
    c = policy_term(p, in, logp).coef * a.grad_scale * a.inv_t;
    if (c == 0.f) {
      zero_span<E, kLanes>(out, 0, V, tid);
      return;
    }
  }
  const RowGrad g = {m, k, c, -c / s};
  const bool same = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(row)) & 15u) == 0;
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int i = tid + u * kLanes;
    if (i >= sp.vecs) break;
    q[u] = g.piece<E>(q[u]);
    E *to = out + sp.head + i * N;
    if (same) {
      __stcs(reinterpret_cast<uint4 *>(to), q[u]);
    } else {
      const E *e = reinterpret_cast<const E *>(&q[u]);
#pragma unroll
      for (int j = 0; j < N; ++j) to[j] = e[j];
    }
  }
  // the label's element after its piece, by the lane that wrote that
  const int place = mark - sp.head;
  if (place >= 0 && place < sp.vecs * N && place / N % kLanes == tid) Elem<E>::store(out + mark, g(picked) + c);
  if (at_head || at_tail) Elem<E>::store(out + edge_at, g(edge) + (edge_at == mark ? c : 0.f));
}

// ----------------------------------------------------------------------------- a row held on chip
// One row is read once: the C blocks of a cluster take a slice each, hold it in
// shared memory, and share their (m, s) through each other's shared memory.  The
// policy loss's coefficient needs that row only, so its gradient is formed from
// the held slice and the row is never read again (2 N bytes instead of 3 N).
//
// The clusters stay for row after row.  A loader warp copies the slices, chunk by
// chunk, through a ring of slots; a slot is free again when its chunk's gradient
// has been formed, so the next rows' chunks are on their way all the time.  The
// other warps go through the rows without a barrier of the block: each
// sends its (m, s) to every block of the cluster, waits for all of them, and
// works out the row's coefficient by itself.
//
// 8699 rows of 128256 bf16, 20 % ignored (1.8 GB read, 2.2 GB written): 632 us,
// 6.35 TB/s, 93 % of the copy rate; two passes over the row took 860 us.  What it
// came from: 1026 us with one row for a cluster at a time, 759 us with the ring,
// and 630 us when the warps' sums went by asynchronous stores instead of arrivals
// with release semantics, which waited for the last row's gradient to reach
// memory.  Two blocks of eight warps an SM beat one of sixteen (646 us), three of
// four (776 us) and slices of 32 KB (893 us).
constexpr int kHeldWarps = 8;                           // that sum and write
constexpr int kHeldWork = 32 * kHeldWarps;
constexpr int kHeldThreads = kHeldWork + 32;             // and the loader warp
constexpr int kPer = 4;                                  // 16-byte pieces of a chunk for each thread
constexpr int kChunk = kPer * kHeldWork;
constexpr int kSlots = 6;                                // 96 KB: two blocks on an SM
constexpr int kHeldBlocks = 2;
constexpr int kSliceBytes = 64 << 10;                    // of a row for a block, where eight blocks suffice
constexpr int kHeldSmem = kSlots * kChunk * 16;

struct HeldArgs {
  RowArgs r;
  PolicyArgs p;
  int cluster;
  int slice;           // 16-byte pieces of a block at most, up to kSlots chunks
  uint32_t zero;       // 0, which the compiler does not know
};

// A block's slice of a row.
template <typename E>
struct HeldSlice {
  const E *row;
  int head, vecs, v0, nv;
  __device__ __forceinline__ HeldSlice(const HeldArgs &h, int64_t t, int rank) {
    row = static_cast<const E *>(h.r.logits) + t * h.r.ldl;
    const RowSpan<E> sp(row, (int)h.r.V);
    head = sp.head;
    vecs = sp.vecs;
    v0 = min(rank * h.slice, vecs);
    nv = min(v0 + h.slice, vecs) - v0;
  }
};

// A place in the ring, counting chunks: its slot, and the parity of the slot's phase.
struct RingAt {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == kSlots) {
      slot = 0;
      parity ^= 1;
    }
  }
};

template <typename E>
__global__ void __launch_bounds__(kHeldThreads, kHeldBlocks) held_kernel(HeldArgs h) {
  extern __shared__ __align__(128) uint4 ring[];
  __shared__ uint64_t full[kSlots], empty[kSlots], ready[2], done;
  __shared__ float2 pairs[2][kMaxCluster * kHeldWarps];  // (m, s) of every warp of the cluster, two exchanges
  const RowArgs &a = h.r;
  constexpr int N = Elem<E>::kVec;
  const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5, C = h.cluster;
  const int rank = (int)(blockIdx.x % C);
  const int64_t clusters = gridDim.x / C;
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kHeldWarps);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&ready[i], C == 1 ? kHeldWarps : 1);
    mbar_init(&done, C * kHeldWarps);
    fence_barrier_init();
  }
  __syncthreads();
  if (C > 1) {                                           // every block's barriers stand before any is written to
    cluster_arrive();
    cluster_wait();
  }
  pdl_wait();
  pdl_launch_dependents();
  int64_t t = blockIdx.x / C;
  int64_t label = t < a.T ? a.labels[t] : -1;
  auto advance = [&](int64_t &mark) {                    // this row's label, with the next one's on its way
    mark = label;
    if (t + clusters < a.T) label = a.labels[t + clusters];
    return mark >= 0 && mark < a.V;
  };
  RingAt at;

  if (warp == kHeldWarps) {                              // the loader
    if (lane != 0) return;
    bool ok = true, again = false;                       // again: the ring has been filled once
    int64_t mark;
    for (; t < a.T && ok; t += clusters) {
      if (!advance(mark)) continue;
      const HeldSlice<E> sl(h, t, rank);
      const uint4 *src = reinterpret_cast<const uint4 *>(sl.row + sl.head) + sl.v0;
      for (int from = 0; from < sl.nv && ok; from += kChunk) {
        const uint32_t bytes = (uint32_t)min(kChunk, sl.nv - from) * 16;
        ok = !again || mbar_wait(&empty[at.slot], at.parity ^ 1);
        if (!ok) break;
        mbar_arrive_expect_tx(&full[at.slot], bytes);
        bulk_load(ring + at.slot * kChunk, src + from, bytes, &full[at.slot]);
        at.next();
        again = again || at.parity;
      }
    }
    // The last copies land before the block ends, whoever else waits for them.
    for (int i = 0; i < kSlots; ++i)
      if (again || i < at.slot) mbar_wait(&full[i], i < at.slot ? at.parity : at.parity ^ 1);
    // And the block does not end before every warp of the cluster has sent its last
    // pair here, also where a wait ran out, or where another stream wrote the labels and
    // warps took different rows for ignored: for as many limits as may lie ahead of a
    // warp, whose rows in the ring are kSlots at most, of kSlots chunks and an exchange
    // each.  (At most 1 % of the rows above: 632 us, 641 with a barrier of the
    // cluster at the end, 630 where the block just leaves.)
    if (C > 1)
      for (int i = 0; i < kSlots * (kSlots + 1) && !mbar_wait<true>(&done, 0); ++i) {}
    return;
  }

  uint32_t count = 0;                                    // exchanges so far
  const float k = a.inv_t * kLog2e;
  for (; t < a.T; t += clusters) {
    int64_t mark64;
    const bool valid = advance(mark64);
    const HeldSlice<E> sl(h, t, rank);
    E *out = static_cast<E *>(a.dlogits) + t * a.lddl;
    const int V = (int)a.V, nv = sl.nv, tail = sl.head + sl.vecs * N, first = sl.head + sl.v0 * N, mark = (int)mark64;
    if (!valid) {
      if (rank == 0 && tid == 0) a.logps[t] = 0.f;
      if (a.dlogits) zero_span<E, kHeldWork>(out, rank == 0 ? 0 : first, rank == C - 1 ? V : first + nv * N, tid);
      continue;
    }
    // on their way while the row is summed (read before this warp's arrival lets
    // any other write the row, where the gradient replaces it)
    const PolicyRow in = policy_row(h.p, t);
    const float picked = Elem<E>::load(sl.row + mark);
    // the ragged ends, at most seven elements each: the first block's and the last one's
    const bool at_head = rank == 0 && tid < sl.head, at_tail = rank == C - 1 && tid >= 16 && tid - 16 < V - tail;
    const int edge_at = at_head ? tid : tail + tid - 16;
    float edge = kNegInf;
    if (at_head || at_tail) edge = Elem<E>::load(sl.row + edge_at);

    float m = kNegInf;
    uint64_t s2 = 0;
    RingAt here = at;
    bool ok = true;
    for (int from = 0; from < nv; from += kChunk, here.next()) {
      ok = mbar_wait(&full[here.slot], here.parity) && ok;
      absorb_span<E, kHeldWork, kPer>(m, s2, ring + here.slot * kChunk, 0, min(kChunk, nv - from), k);
    }
    const float2 both = unpk2(s2);
    float s = both.x + both.y;
    if (edge != kNegInf) absorb_one(m, s, edge, k);
    warp_merge(m, s, k);
    const uint32_t set = count & 1;
    // In a cluster the pair's own bytes complete the others' barriers: an arrival
    // with release semantics there would first wait for the last row's gradient to
    // reach memory.  It is sent when `picked` has come (h.zero is 0): past the
    // exchange any warp may write that element.
    if (C == 1) {
      __syncwarp();                                      // every lane's reads of the row come before the arrival
      if (lane == 0) {
        pairs[set][warp] = make_float2(m, s);
        mbar_arrive(&ready[set]);
      }
    } else {
      if (tid == 0) mbar_arrive_expect_tx(&ready[set], C * kHeldWarps * 8);
      if (lane < C)
        st_async_f2(&pairs[set][rank * kHeldWarps + warp], &ready[set], lane + (__float_as_uint(picked) & h.zero),
                    make_float2(m, s));
    }
    ok = mbar_wait<true>(&ready[set], (count >> 1) & 1) && ok;
    if (!__all_sync(0xffffffffu, ok)) break;             // a wait ran out: the error word is set
    ++count;
    m = kNegInf;
    s = 0.f;
    for (int i = lane; i < C * kHeldWarps; i += 32) {
      const float2 v = pairs[set][i];
      const float mm = fmaxf(m, v.x), r = ref_of(mm);
      s = s * ex2((m - r) * k) + v.y * ex2((v.x - r) * k);
      m = mm;
    }
    warp_merge(m, s, k);
    const float logp = (picked - m) * a.inv_t - logf(s);
    if (rank == 0 && tid == 0) a.logps[t] = logp;
    const float c = policy_term(h.p, in, logp).coef * a.grad_scale * a.inv_t;
    const RowGrad g = {m, k, c, -c / s};
    const bool write = a.dlogits != nullptr && c != 0.f;
    const bool same = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(sl.row)) & 15u) == 0;
    uint4 *dst = reinterpret_cast<uint4 *>(out + sl.head) + sl.v0;
    for (int from = 0; from < nv; from += kChunk, at.next()) {
      const int n = min(kChunk, nv - from);
      const uint4 *src = ring + at.slot * kChunk;
      if (write && same) {
        if (n == kChunk) {
#pragma unroll
          for (int u = 0; u < kPer; ++u) __stcs(dst + from + tid + u * kHeldWork, g.piece<E>(src[tid + u * kHeldWork]));
        } else {
          for (int i = tid; i < n; i += kHeldWork) __stcs(dst + from + i, g.piece<E>(src[i]));
        }
      } else if (write) {
        const int e = first + from * N;                  // the chunk's first element
        grad_words<E, kHeldWork>(out, reinterpret_cast<const E *>(src) - e, e, e + n * N, mark, g);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[at.slot]);
    }
    if (write) {
      if (at_head || at_tail) Elem<E>::store(out + edge_at, g(edge) + (edge_at == mark ? c : 0.f));
      // the label's element, by the thread that wrote its piece
      const int place = mark - first;
      if (same && place >= 0 && place < nv * N && place / N % kHeldWork == tid) Elem<E>::store(out + mark, g(picked) + c);
    } else if (a.dlogits) {
      zero_span<E, kHeldWork>(out, rank == 0 ? 0 : first, rank == C - 1 ? V : first + nv * N, tid);
    }
  }
  if (C > 1 && lane < C) mbar_arrive_remote(&done, lane);
}

// The three metrics from the log-probabilities, in a fixed order.  (The terms are
// worked out again: they need a few values of a token, and no scratch memory.)
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) metrics_kernel(PolicyArgs p, int64_t T, int64_t V, const int64_t *labels,
                                                              const float *logps) {
  __shared__ Sum2 sh[3 * (kSumThreads / 32)];
  pdl_wait();
  Sum2 s[3];
#pragma unroll 2
  for (int64_t t = threadIdx.x; t < T; t += kSumThreads) {
    const int64_t label = labels[t];
    if (label < 0 || label >= V) continue;
    const PolicyTerm x = policy_term(p, policy_row(p, t), logps[t]);
    s[0].add(x.loss);
    s[1].add(x.kl);
    s[2].add(x.clipped);
  }
  block_sums<kSumThreads / 32, 3>(s, sh);
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < 3; ++i) p.metrics[i] = s[i].value();
  }
}

template <typename E>
__global__ void __launch_bounds__(kRowThreads) scale_kernel(E *x, int64_t ldx, int V, const float *factor) {
  pdl_wait();
  const float f = *factor;
  if (f == 1.f) return;
  E *row = x + (int64_t)blockIdx.x * ldx;
  const RowSpan<E> sp(row, V);
  constexpr int N = Elem<E>::kVec;
  const int tid = threadIdx.x, tail = sp.tail();
  if (tid < sp.head) Elem<E>::store(row + tid, Elem<E>::load(row + tid) * f);
  uint4 *body = reinterpret_cast<uint4 *>(row + sp.head);
  for (int i = tid; i < sp.vecs; i += kRowThreads) {
    float v[N];
    Elem<E>::unpack(body[i], v);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] *= f;
    body[i] = Elem<E>::pack(v);
  }
  if (tid < V - tail) Elem<E>::store(row + tail + tid, Elem<E>::load(row + tail + tid) * f);
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

// How a row is cut for the held kernel: slices of at most four chunks (64 KB), so
// that a third of the ring is always ahead; few rows are cut finer, down to 4 KB
// a block, as long as all blocks run at once.  A row that eight blocks' rings
// do not hold (cluster 0) goes by the two-pass kernels.
struct HeldPlan {
  int cluster, slice;
};
HeldPlan plan_held(int64_t T, int64_t bytes) {
  int64_t c = std::max<int64_t>(1, ceil_div(bytes, kSliceBytes));
  c = std::max(c, std::min(kHeldBlocks * num_sms() / std::max<int64_t>(T, 1), bytes / 4096));
  c = std::min<int64_t>(c, kMaxCluster);
  const int64_t slice = std::max<int64_t>(8, round_up(ceil_div(bytes / 16, c), 8));
  if (slice > kSlots * kChunk) return {0, 0};
  return {(int)c, (int)slice};
}

// Clusters of a kernel that the device holds at once; the last answers are kept.
int max_clusters(const void *kernel, int cluster) {
  struct Known {
    const void *kernel;
    int dev, cluster, n;
  };
  static Known known[32];
  static int used = 0;
  static std::mutex mu;
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lk(mu);
  for (const Known &k : known)
    if (k.n > 0 && k.kernel == kernel && k.dev == dev && k.cluster == cluster) return k.n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(kHeldThreads);
  cfg.dynamicSmemBytes = kHeldSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) n = 1;
  known[used++ % 32] = {kernel, dev, cluster, n};
  return n;
}

template <typename E>
cudaError_t launch_held(const HeldArgs &h, cudaStream_t st) {
  const void *kernel = reinterpret_cast<const void *>(held_kernel<E>);
  cudaError_t e = ensure_smem(kernel, kHeldSmem);
  if (e != cudaSuccess) return e;
  const int64_t clusters = std::min<int64_t>(h.r.T, max_clusters(kernel, h.cluster));
  return launch(held_kernel<E>, dim3((unsigned)(clusters * h.cluster)), dim3(kHeldThreads), kHeldSmem, st, h.cluster,
                true, h);
}

// Blocks for each row of the gradient pass: enough that the grid fills
// the SMs (eight blocks each) some eight times over, so that the last blocks to
// run leave few SMs idle, with at least 16 KB a block; few rows are cut down to
// 4 KB a block until the grid fills the SMs once.
int parts_of(int64_t T, int64_t bytes) {
  const int64_t once = 8 * (int64_t)num_sms();
  int64_t c = std::min(ceil_div(8 * once, T), bytes / (16 << 10));
  c = std::max(c, std::min(ceil_div(once, T), bytes / (4 << 10)));
  return (int)std::min<int64_t>(std::max<int64_t>(c, 1), 64);
}
// 16-byte pieces of one of `parts` slices of a row.
int slice_of(int64_t bytes, int parts) { return (int)std::max<int64_t>(8, round_up(ceil_div(bytes / 16, parts), 8)); }

// Rows of up to kShortest bytes go to a warp's registers, four pieces a lane, up to
// kShort bytes sixteen, and for sums up to kShortTeam bytes to those of four warps.
// Against a block of 256 threads (sums, gradient) or a cluster's ring (policy loss)
// for a row: sums of 4000 rows of 1003 fp32 5.2 us (10.3), of 16000 bf16 21.4 (25.4);
// gradient of 4000 rows of 300 fp32 2.9 (7.5); policy loss with gradient of 5655 rows
// of 300 fp32 9.2 (36.3), of 8192 bf16 36.6 (52.1), of 16000 bf16 56.3 (74.3).
constexpr int64_t kShortest = 2 << 10, kShort = 8 << 10, kShortTeam = 32 << 10;
template <typename E, int kMode>
cudaError_t launch_short_as(const RowArgs &r, const PolicyArgs &p, int64_t bytes, cudaStream_t st) {
  const dim3 grid((unsigned)ceil_div(r.T, 8));
  if (bytes <= kShortest) return launch(short_kernel<E, 4, 1, kMode>, grid, dim3(256), 0, st, 1, true, r, p);
  if (bytes <= kShort) return launch(short_kernel<E, 16, 1, kMode>, grid, dim3(256), 0, st, 1, true, r, p);
  if constexpr (kMode != kShortGrad)
    return launch(short_kernel<E, 16, 4, kMode>, dim3((unsigned)r.T), dim3(128), 0, st, 1, true, r, p);
  return cudaErrorInvalidValue;
}
template <int kMode>
bool short_rows(int64_t bytes) {
  return bytes <= (kMode == kShortGrad ? kShort : kShortTeam);
}
template <int kMode>
cudaError_t launch_short(lora_dtype_t dtype, const RowArgs &r, const PolicyArgs &p, cudaStream_t st) {
  return dtype == LORA_BF16 ? launch_short_as<__nv_bfloat16, kMode>(r, p, r.V * 2, st)
                            : launch_short_as<float, kMode>(r, p, r.V * 4, st);
}

// The statistics pass: one block a row, with more threads to it the fewer rows
// there are to fill the SMs; rows for less than half of the SMs are cut over
// clusters, down to 4 KB a block.  Rows of 128256 bf16, 256 / 512 / 1024 threads:
// 2000 rows 81.9 / 79.2 / 93.3 us, 200 rows 15.7 / 12.0 / 13.8, 100 rows 14.0 / 9.2
// / 7.5; 40 rows over clusters of eight blocks of 256 threads 4.8 us, whole 5.8.
// Clusters cost where blocks abound: 4000 rows of 32000 bf16 42.0 us with one
// block each, 80 with four.
template <typename E>
cudaError_t launch_stats(const RowArgs &r, int64_t bytes, cudaStream_t st) {
  const int64_t sms = num_sms();
  if (2 * r.T < sms) {
    const int c = (int)std::min<int64_t>({std::max<int64_t>(1, 4 * sms / r.T), std::max<int64_t>(1, bytes / (4 << 10)),
                                          kMaxCluster});
    return launch(stats_kernel<E, kRowThreads>, dim3((unsigned)(r.T * c)), dim3(kRowThreads), 0, st, c, true, r, c,
                  slice_of(bytes, c));
  }
  const int slice = slice_of(bytes, 1);
  const dim3 grid((unsigned)r.T);
  if (bytes >= (32 << 10) && r.T <= sms) return launch(stats_kernel<E, 1024>, grid, dim3(1024), 0, st, 1, true, r, 1, slice);
  if (bytes >= (32 << 10) && r.T <= 2 * sms) return launch(stats_kernel<E, 512>, grid, dim3(512), 0, st, 1, true, r, 1, slice);
  return launch(stats_kernel<E, kRowThreads>, grid, dim3(kRowThreads), 0, st, 1, true, r, 1, slice);
}

lora_status_t run_stats(lora_dtype_t dtype, const RowArgs &r, cudaStream_t st) {
  if (r.T == 0) return LORA_OK;
  if (short_rows<kShortStats>(r.V * (dtype == LORA_BF16 ? 2 : 4))) {
    LORA_CUDA(launch_short<kShortStats>(dtype, r, PolicyArgs{}, st));
    return LORA_OK;
  }
  LORA_CUDA(dtype == LORA_BF16 ? launch_stats<__nv_bfloat16>(r, r.V * 2, st) : launch_stats<float>(r, r.V * 4, st));
  return LORA_OK;
}

lora_status_t run_grad(lora_dtype_t dtype, const RowArgs &r, cudaStream_t st) {
  if (r.T == 0 || r.V == 0) return LORA_OK;
  const int64_t bytes = r.V * (dtype == LORA_BF16 ? 2 : 4);
  if (short_rows<kShortGrad>(bytes)) {
    LORA_CUDA(launch_short<kShortGrad>(dtype, r, PolicyArgs{}, st));
    return LORA_OK;
  }
  const int c = parts_of(r.T, bytes), slice = slice_of(bytes, c);
  const dim3 grid((unsigned)(r.T * c)), block(kRowThreads);
  LORA_CUDA(dtype == LORA_BF16 ? launch(grad_kernel<__nv_bfloat16>, grid, block, 0, st, 1, true, r, c, slice)
                               : launch(grad_kernel<float>, grid, block, 0, st, 1, true, r, c, slice));
  return LORA_OK;
}

int64_t token_blocks(int64_t T) { return ceil_div(T, kPairThreads); }

}  // namespace

// ----------------------------------------------------------------------------- host side
size_t preference_ws_bytes(int64_t T, int64_t) { return ws_round(8 * T) + ws_round(4 * T) + ws_round(4); }
size_t policy_ws_bytes(int64_t T, int64_t row_bytes, bool grad) {
  if (T == 0 || !grad || row_bytes <= (int64_t)kMaxCluster * kSlots * kChunk * 16) return 0;
  return ws_round(8 * T) + ws_round(4 * T);
}
int read_clear_error_loss() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)) != cudaSuccess) return -1;
  if (v) cudaMemcpyToSymbol(g_device_error, &z, sizeof(int));
  return v;
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
  unsigned *ticket = static_cast<unsigned *>(c.take(4));
  if (ticket == nullptr || (a.T > 0 && coef == nullptr)) return LORA_ERR_WORKSPACE;
  r.coef = coef;
  r.ticket = ticket;
  if (a.T == 0)
    LORA_CUDA(cudaMemsetAsync(ticket, 0, sizeof(unsigned), st));
  else
    LORA_TRY(run_stats(a.dtype, r, st));
  if (p.P > 0)
    LORA_CUDA(launch(pairs_kernel, dim3((unsigned)p.P), dim3(kPairThreads), 0, st, 1, true, p, a.T, a.V, a.labels,
                     (const float *)a.logps, a.dlogits ? coef : (float *)nullptr, ticket));
  return a.dlogits ? run_grad(a.dtype, r, st) : LORA_OK;
}

lora_status_t policy_loss(const LossArgs &a, const PolicyArgs &p, void *ws, size_t ws_bytes, cudaStream_t st) {
  if (a.T == 0) {
    LORA_CUDA(cudaMemsetAsync(p.metrics, 0, 3 * sizeof(float), st));
    return LORA_OK;
  }
  RowArgs r = row_args(a);
  const int64_t bytes = a.V * (a.dtype == LORA_BF16 ? 2 : 4);
  if (short_rows<kShortPolicy>(bytes)) {
    LORA_CUDA(launch_short<kShortPolicy>(a.dtype, r, p, st));
  } else if (const HeldPlan hp = plan_held(a.T, bytes); hp.cluster > 0) {
    const HeldArgs h = {r, p, hp.cluster, hp.slice, 0u};
    LORA_CUDA(a.dtype == LORA_BF16 ? launch_held<__nv_bfloat16>(h, st) : launch_held<float>(h, st));
  } else if (a.dlogits == nullptr) {
    LORA_TRY(run_stats(a.dtype, r, st));
  } else {
    WsCarver c(ws, ws_bytes);
    r.stats = static_cast<float2 *>(c.take(8 * a.T));
    float *coef = static_cast<float *>(c.take(4 * a.T));
    if (coef == nullptr) return LORA_ERR_WORKSPACE;
    LORA_TRY(run_stats(a.dtype, r, st));
    r.coef = coef;
    LORA_CUDA(launch(tokens_kernel, dim3((unsigned)token_blocks(a.T)), dim3(kPairThreads), 0, st, 1, true, p, a.T, a.V,
                     a.labels, (const float *)a.logps, coef));
    LORA_TRY(run_grad(a.dtype, r, st));
  }
  LORA_CUDA(launch(metrics_kernel, dim3(1), dim3(kSumThreads), 0, st, 1, true, p, a.T, a.V, a.labels,
                   (const float *)a.logps));
  return LORA_OK;
}

lora_status_t scale_gradient(lora_dtype_t dtype, int64_t T, int64_t V, void *x, int64_t ldx, const float *factor,
                             cudaStream_t st) {
  if (T == 0 || V == 0) return LORA_OK;
  if (dtype == LORA_BF16)
    LORA_CUDA(launch(scale_kernel<__nv_bfloat16>, dim3((unsigned)T), dim3(kRowThreads), 0, st, 1, true,
                     (__nv_bfloat16 *)x, ldx, (int)V, factor));
  else
    LORA_CUDA(launch(scale_kernel<float>, dim3((unsigned)T), dim3(kRowThreads), 0, st, 1, true, (float *)x, ldx, (int)V,
                     factor));
  return LORA_OK;
}

}  // namespace lora
