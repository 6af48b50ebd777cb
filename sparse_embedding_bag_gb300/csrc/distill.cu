// Distillation from a teacher's top logits: loss per row, gradient of the
// student's logits, and both in one step.
//
// With z a row of student logits, p = softmax(z / tau), and the teacher's list
// (id_k, t_k), q_k = exp(t_k / tau - L):
//   L given (tail): r = max(0, 1 - sum q), u = mass of p off the list, and
//     loss = tau^2 [ sum_k q_k (log q_k - log p_{id_k}) + r (log r - log u) ]
//   L not given: L = log sum exp(t_k / tau), r = 0.
//   dloss/dz_v = tau [ p_v - sum_{k: id_k = v} q_k ]   for v on the list,
//                tau p_v (1 - r / u)                   off it.
// u is summed over the tokens off the list, never as 1 - (mass on it): it would
// cancel for a student that agrees with its teacher. Entries with id -1 are
// padding; a row without entries, or whose teacher has no mass (L = -infinity), has
// loss 0 and gradient 0.
//
// Exponentials are base 2: p_v = 2^((z_v - M) c) / S with c = log2(e) / tau and M the
// row's largest logit. The difference comes first, so that rows masked with the type's
// lowest value neither overflow nor lose their maximum. Sums are held in fp32.
//
// Forward and step: a cluster of CTAs holds a row in shared memory, brought there by bulk
// copies: the row is read from HBM once and its gradient, computed in place, written once.
// Its largest logit and sums are exchanged through distributed shared memory in one round.
// Backward (its sums are known): blocks over pieces of the rows, one read and one write.
#include <cmath>

#include "sm103.cuh"

namespace embbwd {
namespace {

constexpr int kMaxList = 1024;   // longest teacher list
constexpr int kRowThreads = 512;
constexpr int kMaxCluster = 8;
constexpr uint32_t kLoadBytes = 16384;              // of a bulk load with a barrier of its own
constexpr uint32_t kSliceMost = 200 * 1024;         // bytes of a row that a CTA can hold
constexpr uint32_t kSliceWanted = 66 * 1024;        // three CTAs an SM
constexpr uint32_t kSliceLeast = 4 * 1024;
constexpr int kLoads = kSliceMost / kLoadBytes + 1;
constexpr int32_t kMaxDistillRows = 1 << 23;        // (rows x pieces of a row stay below 2^31)
constexpr int kPiece = 8192;                        // elements of a block of the backward

enum { kForward = 0, kBackward = 1, kStep = 2 };

struct DistillArgs {
  const void* z;
  int64_t z_stride;
  int32_t N, V, K;
  const int64_t* ids;
  const void* t;
  int t_dtype;
  int64_t t_stride;
  const float* lse;      // nullable: renormalise over the list
  const float* weight;   // nullable: 1
  float tau, c2;         // c2 = log2(e) / tau
  float* loss;
  float4* stats;         // written by the forward, read by the backward
  void* dz;
  int64_t dz_stride;
  uint32_t* status;
};

// The teacher's list of a row in shared memory.
struct List {
  int32_t* id;   // [K], -1: no entry
  float* q;      // [K]
  float* z;      // [K] the student's logit there
  int repeated;  // some id occurs more than once
};

// Is entry k the first with its id? Only looked for in rows where ids repeat.
__device__ __forceinline__ bool is_first(const List& l, int k) {
  if (l.repeated)
    for (int j = 0; j < k; ++j)
      if (l.id[j] == l.id[k]) return false;
  return true;
}
// The teacher's probability of entry k's token: repeated entries add in list order.
__device__ __forceinline__ float q_of_token(const List& l, int k, int K) {
  if (!l.repeated) return l.q[k];
  float q = 0.f;
  for (int j = k; j < K; ++j)
    if (l.id[j] == l.id[k]) q += l.q[j];
  return q;
}

// Reads the ids of row n's list; returns whether there is any, to every thread.
__device__ __forceinline__ bool read_ids(const DistillArgs& a, int32_t n, List& l) {
  int any = 0;
  for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
    const int64_t id = a.ids[n * a.t_stride + k];
    if (id < -1 || id >= a.V) report(a.status, kErrIndex);
    const bool ok = id >= 0 && id < a.V;
    l.id[k] = ok ? (int32_t)id : -1;
    any |= ok;
  }
  return __syncthreads_or(any);
}

// The rest of the list (the student's logits of entries in [lo, hi)), each thread its own
// entries; returns whether the row takes part. Sets l.q, *L and the sum of q. L is found
// here unless the caller knows it.
template <typename T>
__device__ __forceinline__ bool read_list(const DistillArgs& a, int32_t n, List& l, float* scratch, int32_t lo,
                                          int32_t hi, float known_L, bool known, float* L, float* qsum) {
  const T* z = static_cast<const T*>(a.z) + n * a.z_stride;
  float big = -INFINITY;
  for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
    const int32_t id = l.id[k];
    const float t = id >= 0 ? __fdiv_rn(load_as_float(a.t, a.t_dtype, n * a.t_stride + k), a.tau) : -INFINITY;
    l.z[k] = id >= lo && id < hi ? Elem<T>::get(z[id]) : 0.f;
    l.q[k] = t;
    big = fmaxf(big, t);
  }
  *L = known_L;
  if (!known) {
    big = block_all<true>(big, scratch);
    float s = 0.f;
    for (int k = threadIdx.x; k < a.K; k += blockDim.x) s += expf(l.q[k] - (isinf(big) ? 0.f : big));
    s = block_all<false>(s, scratch);
    *L = s == 0.f ? -INFINITY : (isinf(big) ? 0.f : big) + logf(s);
  }
  if (*L == -INFINITY) return false;
  float s = 0.f;
  for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
    const float q = l.id[k] >= 0 ? expf(l.q[k] - *L) : 0.f;
    l.q[k] = q;
    s += q;
  }
  *qsum = block_all<false>(s, scratch);
  return true;
}

// The loss of a row (without tau^2) and the coefficient of its gradient off the list,
// from M, S and the sum off the list. All threads of a block that read the whole list.
__device__ __forceinline__ float loss_of(const DistillArgs& a, int32_t n, const List& l, float* scratch, float M,
                                         float S, float L) {
  const float logS = logf(S);
  float ls = 0.f;
  for (int k = threadIdx.x; k < a.K; k += blockDim.x)
    if (l.q[k] > 0.f) {
      const float logp = (l.z[k] - M) * (a.c2 * kLn2) - logS;
      ls += l.q[k] * ((__fdiv_rn(load_as_float(a.t, a.t_dtype, n * a.t_stride + k), a.tau) - L) - logp);
    } else if (!(l.q[k] == 0.f)) {
      ls = NAN;
    }
  return block_all<false>(ls, scratch);
}
__device__ __forceinline__ float tail_of(float qsum, float rest, float S, float* coef) {
  const float r = fmaxf(0.f, 1.f - qsum), u = rest / S;
  *coef = r > 0.f ? 1.f - r / u : 1.f;
  return r > 0.f ? r * (logf(r) - logf(u)) : 0.f;
}

// Rows too wide for a cluster: one block a row, which is read for its largest logit, for
// its sums and for its gradient. A bitmap of the vocabulary marks the list.
template <typename T, bool kGrad>
__global__ void __launch_bounds__(kRowThreads) k_distill_wide(DistillArgs a) {
  extern __shared__ uint32_t on_list[];
  __shared__ List l;
  __shared__ float scratch[64];
  const int32_t n = blockIdx.x;
  const int32_t words = (a.V + 31) / 32;
  const T* z = static_cast<const T*>(a.z) + n * a.z_stride;
  T* dz = static_cast<T*>(a.dz) + n * a.dz_stride;
  for (int i = threadIdx.x; i < words; i += kRowThreads) on_list[i] = 0;
  if (threadIdx.x == 0) {
    l.id = reinterpret_cast<int32_t*>(on_list + words), l.q = reinterpret_cast<float*>(l.id + a.K), l.z = l.q + a.K;
    l.repeated = 0;
  }
  __syncthreads();
  float L = 0.f, qsum = 0.f;
  if (!read_ids(a, n, l) || !read_list<T>(a, n, l, scratch, 0, a.V, a.lse ? a.lse[n] : 0.f, a.lse != nullptr, &L, &qsum)) {
    if (threadIdx.x == 0) {
      a.loss[n] = 0.f;
      if (!kGrad) a.stats[n] = make_float4(0.f, 1.f, 0.f, L);
    }
    if (kGrad)
      for (int32_t v = threadIdx.x; v < a.V; v += kRowThreads) dz[v] = Elem<T>::put(0.f);
    return;
  }
  for (int k = threadIdx.x; k < a.K; k += kRowThreads)
    if (l.id[k] >= 0) {
      const uint32_t bit = 1u << (l.id[k] & 31);
      if (atomicOr(&on_list[l.id[k] >> 5], bit) & bit) l.repeated = 1;
    }
  float M = -INFINITY;
  for (int32_t v = threadIdx.x; v < a.V; v += kRowThreads) M = fmaxf(M, Elem<T>::get(z[v]));
  M = block_all<true>(M, scratch);
  float rest = 0.f, top = 0.f;
  for (int32_t v = threadIdx.x; v < a.V; v += kRowThreads)
    if (!(on_list[v >> 5] >> (v & 31) & 1u)) rest += ex2((Elem<T>::get(z[v]) - M) * a.c2);
  rest = block_all<false>(rest, scratch);
  for (int k = threadIdx.x; k < a.K; k += kRowThreads)
    if (l.id[k] >= 0 && is_first(l, k)) top += ex2((l.z[k] - M) * a.c2);
  const float S = rest + block_all<false>(top, scratch);
  float coef = 1.f, loss = loss_of(a, n, l, scratch, M, S, L);
  if (a.lse) loss += tail_of(qsum, rest, S, &coef);
  if (threadIdx.x == 0) {
    a.loss[n] = a.tau * a.tau * loss;
    if (!kGrad) a.stats[n] = make_float4(M, S, coef, L);
  }
  if (!kGrad) return;
  const float scale = (a.weight ? a.weight[n] : 1.f) * a.tau;
  for (int32_t v = threadIdx.x; v < a.V; v += kRowThreads)
    if (!(on_list[v >> 5] >> (v & 31) & 1u))
      dz[v] = Elem<T>::put(scale * coef / S * ex2((Elem<T>::get(z[v]) - M) * a.c2));
  for (int k = threadIdx.x; k < a.K; k += kRowThreads)
    if (l.id[k] >= 0 && is_first(l, k))
      dz[l.id[k]] = Elem<T>::put(scale * (ex2((l.z[k] - M) * a.c2) / S - q_of_token(l, k, a.K)));
}

// 16 bytes of a row, as pairs of floats.
template <typename T>
struct Unit;
template <>
struct Unit<float> {
  static constexpr int n = 4;
  __device__ __forceinline__ static float max_of(uint4 v) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  __device__ __forceinline__ static void widen(uint4 v, F2 (&x)[2]) {
    x[0] = F2::of(__uint_as_float(v.x), __uint_as_float(v.y));
    x[1] = F2::of(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  __device__ __forceinline__ static uint4 narrow(const float2 (&x)[2]) {
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x), __float_as_uint(x[1].y));
  }
};
template <>
struct Unit<__nv_bfloat16> {
  static constexpr int n = 8;
  __device__ __forceinline__ static float max_of(uint4 v) {
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v);
    const float2 m = __bfloat1622float2(__hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3])));
    return fmaxf(m.x, m.y);
  }
  __device__ __forceinline__ static void widen(uint4 v, F2 (&x)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = F2::of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ __forceinline__ static uint4 narrow(const float2 (&x)[4]) {
    uint4 v;
    __nv_bfloat162* p = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __float22bfloat162_rn(x[i]);
    return v;
  }
};
template <>
struct Unit<__half> {
  static constexpr int n = 8;
  __device__ __forceinline__ static float max_of(uint4 v) {
    const __half2* p = reinterpret_cast<const __half2*>(&v);
    const float2 m = __half22float2(__hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3])));
    return fmaxf(m.x, m.y);
  }
  __device__ __forceinline__ static void widen(uint4 v, F2 (&x)[4]) {
    const __half2* p = reinterpret_cast<const __half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(p[i]);
      x[i] = F2::of(f.x, f.y);
    }
  }
  __device__ __forceinline__ static uint4 narrow(const float2 (&x)[4]) {
    uint4 v;
    __half2* p = reinterpret_cast<__half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __float22half2_rn(x[i]);
    return v;
  }
};

// Sizes of a cluster CTA's shared memory: the slice, its bitmap, the list.
template <typename T>
__host__ __device__ constexpr uint32_t slice_bytes(int32_t slice) {
  return (uint32_t)(slice + Unit<T>::n) * sizeof(T);
}
__host__ __device__ constexpr uint32_t bitmap_bytes(int32_t slice) { return ((uint32_t)slice / 8 + 4 + 15) / 16 * 16; }
template <typename T>
constexpr size_t cluster_smem(int32_t slice, int K) {
  return slice_bytes<T>(slice) + bitmap_bytes(slice) + (size_t)K * 12;
}

// A cluster a row, `slice` elements (a multiple of 64) a CTA. Element e of the slice lies
// at position shift + e of the buffer, shift its place in 16 bytes of global memory, so that
// whole 16-byte units are copied in bulk; the few elements beside them one by one.
template <typename T, bool kGrad>
__global__ void __launch_bounds__(kRowThreads, 3) k_distill_cluster(DistillArgs a, int32_t slice, int log_ctas) {
  using U = Unit<T>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ List l;
  __shared__ float scratch[64];
  __shared__ float parts[3][kMaxCluster];  // of every CTA: largest logit, sums off and on the list
  __shared__ uint64_t bars[kLoads];
  __shared__ int abort;
  const uint32_t ctas = 1u << log_ctas, rank = blockIdx.x & (ctas - 1);
  const int32_t n = blockIdx.x >> log_ctas;
  const int32_t r0 = min((int64_t)a.V, (int64_t)rank * slice), len = min(a.V - r0, slice);
  const T* z = static_cast<const T*>(a.z) + n * a.z_stride + r0;
  T* dz = static_cast<T*>(a.dz) + n * a.dz_stride + r0;
  T* data = reinterpret_cast<T*>(smem);
  uint4* units4 = reinterpret_cast<uint4*>(smem);
  uint32_t* bitmap = reinterpret_cast<uint32_t*>(smem + slice_bytes<T>(slice));
  const int32_t shift = (int32_t)(reinterpret_cast<uintptr_t>(z) / sizeof(T) % U::n);
  const int32_t units = len ? (shift + len + U::n - 1) / U::n : 0;
  const int32_t u0 = min(units, shift ? 1 : 0), u1 = max(u0, (shift + len) / U::n);  // units that are copied whole
  const int32_t edge0 = min(len, u0 * U::n - shift), edge1 = max(edge0, min(len, u1 * U::n - shift));

  for (int i = threadIdx.x; i < (int)bitmap_bytes(slice) / 4; i += kRowThreads) bitmap[i] = 0;
  if (threadIdx.x == 0) {
    l.id = reinterpret_cast<int32_t*>(smem + slice_bytes<T>(slice) + bitmap_bytes(slice));
    l.q = reinterpret_cast<float*>(l.id + a.K), l.z = l.q + a.K;
    l.repeated = 0;
    abort = 0;
    for (int i = 0; i < kLoads; ++i) mbar_init(smem_u32(&bars[i]), 1);
    mbar_init_fence();
  }
  __syncthreads();
  // The row is asked for as soon as it is known to have a list.
  const uint32_t bytes = (uint32_t)(u1 - u0) * 16;
  bool part = read_ids(a, n, l);
  if (part && threadIdx.x == 0)
    for (uint32_t i = 0; i * kLoadBytes < bytes; ++i) {
      const uint32_t at = i * kLoadBytes, some = min(kLoadBytes, bytes - at);
      mbar_expect(smem_u32(&bars[i]), some);
      bulk_load(smem_u32(smem) + u0 * 16 + at, reinterpret_cast<const char*>(z + (u0 * U::n - shift)) + at, some,
                smem_u32(&bars[i]));
    }
  const int32_t lo = rank == 0 ? 0 : r0, hi = rank == 0 ? a.V : r0 + len;  // CTA 0 finds the loss: it needs every entry's logit
  float L = 0.f, qsum = 0.f, M = -INFINITY, S = 0.f, tail = 0.f;
  if (part) {
    part = read_list<T>(a, n, l, scratch, lo, hi, a.lse ? a.lse[n] : 0.f, a.lse != nullptr, &L, &qsum);
    if (!part)  // a teacher without mass: the copies under way end first
      for (uint32_t i = 0; i * kLoadBytes < bytes; ++i) mbar_wait(smem_u32(&bars[i]), 0, &abort);
  }
  if (!part) {  // the same for the whole cluster
    if (rank == 0 && threadIdx.x == 0) {
      a.loss[n] = 0.f;
      if (!kGrad) a.stats[n] = make_float4(0.f, 1.f, 0.f, L);
    }
    if constexpr (!kGrad) return;
    __syncthreads();
    for (int32_t u = threadIdx.x; u < units; u += kRowThreads) units4[u] = make_uint4(0, 0, 0, 0);
  } else {
    for (int32_t q = threadIdx.x; q < (u0 + units - u1) * U::n; q += kRowThreads) {  // the edge units
      const int32_t p = q < u0 * U::n ? q : q + (u1 - u0) * U::n, e = p - shift;
      data[p] = e >= 0 && e < len ? z[e] : Elem<T>::put(-INFINITY);
    }
    for (int k = threadIdx.x; k < a.K; k += kRowThreads) {
      const int32_t e = l.id[k] - r0;
      if (l.id[k] < 0 || e < 0 || e >= len) continue;
      const uint32_t p = shift + e, bit = 1u << (p & 31);
      if (atomicOr(&bitmap[p >> 5], bit) & bit) l.repeated = 1;
    }
    __syncthreads();
    float m = -INFINITY;
    for (int32_t u = threadIdx.x; u < units; u += kRowThreads) {
      if (u >= u0 && u < u1) mbar_wait(smem_u32(&bars[(uint32_t)(u - u0) * 16 / kLoadBytes]), 0, &abort);
      m = fmaxf(m, U::max_of(units4[u]));
    }
    m = block_all<true>(m, scratch);
    const float ref = m == -INFINITY ? 0.f : m;
    const F2 minus = F2::of(-ref, -ref), c2 = F2::of(a.c2, a.c2);
    F2 sum = F2::of(0.f, 0.f);
    const uint8_t* on_list = reinterpret_cast<const uint8_t*>(bitmap);
#pragma unroll 2
    for (int32_t u = threadIdx.x; u < units; u += kRowThreads) {
      F2 x[U::n / 2];
      U::widen(units4[u], x);
      const uint32_t bits = U::n == 8 ? on_list[u] : on_list[u >> 1] >> (u & 1) * 4 & 15u;
#pragma unroll
      for (int i = 0; i < U::n / 2; ++i) {
        const float2 y = ((x[i] + minus) * c2).get();
        float2 e = make_float2(ex2(y.x), ex2(y.y));
        if (bits >> 2 * i & 1u) e.x = 0.f;
        if (bits >> 2 * i & 2u) e.y = 0.f;
        sum = sum + F2::of(e.x, e.y);
      }
    }
    float rest = sum.get().x + sum.get().y, top = 0.f;
    for (int k = threadIdx.x; k < a.K; k += kRowThreads) {
      const int32_t e = l.id[k] - r0;
      if (l.id[k] >= 0 && e >= 0 && e < len && is_first(l, k)) top += ex2((l.z[k] - ref) * a.c2);
    }
    block_sums(rest, top, scratch);
    if (threadIdx.x < ctas) {
      cluster_store(cluster_map(smem_u32(&parts[0][rank]), threadIdx.x), m);
      cluster_store(cluster_map(smem_u32(&parts[1][rank]), threadIdx.x), rest);
      cluster_store(cluster_map(smem_u32(&parts[2][rank]), threadIdx.x), top);
    }
    cluster_sync();
    float off = 0.f;
    for (uint32_t i = 0; i < ctas; ++i) M = fmaxf(M, parts[0][i]);
    for (uint32_t i = 0; i < ctas; ++i) {
      const float f = parts[0][i] == M ? 1.f : ex2((parts[0][i] - M) * a.c2);
      off += parts[1][i] * f;
      S += parts[2][i] * f;
    }
    S += off;
    float coef = 1.f;
    if (a.lse) tail = tail_of(qsum, off, S, &coef);
    if (threadIdx.x == 0 && abort) report(a.status, kErrTimeout);
    if constexpr (!kGrad) {
      if (rank != 0) return;
      const float loss = loss_of(a, n, l, scratch, M, S, L) + tail;
      if (threadIdx.x == 0) {
        a.loss[n] = a.tau * a.tau * loss;
        a.stats[n] = make_float4(M, S, coef, L);
      }
      return;
    }
    const float scale = (a.weight ? a.weight[n] : 1.f) * a.tau, g = scale * coef / S;
    const F2 minus_M = F2::of(-M, -M), g2 = F2::of(g, g);
#pragma unroll 2
    for (int32_t u = threadIdx.x; u < units; u += kRowThreads) {
      F2 x[U::n / 2];
      U::widen(units4[u], x);
      float2 e[U::n / 2];
#pragma unroll
      for (int i = 0; i < U::n / 2; ++i) {
        const float2 y = ((x[i] + minus_M) * c2).get();
        e[i] = (F2::of(ex2(y.x), ex2(y.y)) * g2).get();
      }
      units4[u] = U::narrow(e);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < a.K; k += kRowThreads) {
      const int32_t e = l.id[k] - r0;
      if (l.id[k] >= 0 && e >= 0 && e < len && is_first(l, k))
        data[shift + e] = Elem<T>::put(scale * (ex2((l.z[k] - M) * a.c2) / S - q_of_token(l, k, a.K)));
    }
  }
  proxy_fence();
  __syncthreads();
  if (reinterpret_cast<uintptr_t>(dz) / sizeof(T) % U::n == (uintptr_t)shift) {
    if (threadIdx.x == 0 && u1 > u0) {
      bulk_store(dz + (u0 * U::n - shift), smem_u32(smem) + u0 * 16, bytes);
      bulk_commit();
    }
    for (int32_t q = threadIdx.x; q < edge0 + len - edge1; q += kRowThreads) {
      const int32_t e = q < edge0 ? q : q - edge0 + edge1;
      dz[e] = data[shift + e];
    }
  } else {
    for (int32_t e = threadIdx.x; e < len; e += kRowThreads) dz[e] = data[shift + e];
  }
  if (rank == 0 && part) {
    const float loss = loss_of(a, n, l, scratch, M, S, L) + tail;
    if (threadIdx.x == 0) a.loss[n] = a.tau * a.tau * loss;
  }
  if (threadIdx.x == 0) bulk_wait_read();
}

// The gradient from the forward's sums: a block takes kPiece elements of a row.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_distill_backward(DistillArgs a, int32_t pieces) {
  using U = Unit<T>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t on_list[kPiece / 32];
  __shared__ List l;
  const int32_t n = blockIdx.x / pieces, r0 = (blockIdx.x - n * pieces) * kPiece, len = min(a.V - r0, kPiece);
  const T* z = static_cast<const T*>(a.z) + n * a.z_stride + r0;
  T* dz = static_cast<T*>(a.dz) + n * a.dz_stride + r0;
  // units start `head` elements into the piece: stores 16-byte aligned, and loads too where both can be
  const int32_t z_at = reinterpret_cast<uintptr_t>(z) / sizeof(T) % U::n;
  const int32_t dz_at = reinterpret_cast<uintptr_t>(dz) / sizeof(T) % U::n;
  const int32_t head = min(len, (U::n - dz_at) % U::n), units = (len - head) / U::n;
  constexpr int kBatch = 4;
  uint4 raw[kBatch];
  const bool wide_loads = z_at == dz_at;
  const uint4* zu = reinterpret_cast<const uint4*>(z + head);
  auto load = [&](int k, int32_t u) {
    if (wide_loads && u < units) raw[k] = zu[u];
  };
#pragma unroll
  for (int k = 0; k < kBatch; ++k) load(k, threadIdx.x + k * kThreads);
  const float4 st = a.stats[n];
  for (int i = threadIdx.x; i < kPiece / 32; i += kThreads) on_list[i] = 0;
  if (threadIdx.x == 0) {
    l.id = reinterpret_cast<int32_t*>(smem), l.q = reinterpret_cast<float*>(l.id + a.K), l.z = l.q + a.K;
    l.repeated = 0;
  }
  __syncthreads();
  int any = 0;
  for (int k = threadIdx.x; k < a.K; k += kThreads) {
    const int64_t id = a.ids[n * a.t_stride + k];
    const bool ok = id >= 0 && id < a.V;
    if (id < -1 || id >= a.V) report(a.status, kErrIndex);
    any |= ok;
    const int32_t e = ok ? (int32_t)id - r0 : -1;
    const bool here = e >= 0 && e < len;
    l.id[k] = here ? e : -1;
    if (!here) continue;
    l.q[k] = expf(__fdiv_rn(load_as_float(a.t, a.t_dtype, n * a.t_stride + k), a.tau) - st.w);
    l.z[k] = Elem<T>::get(z[e]);
    const uint32_t bit = 1u << (e & 31);
    if (atomicOr(&on_list[e >> 5], bit) & bit) l.repeated = 1;
  }
  any = __syncthreads_or(any);
  const bool part = any && st.w != -INFINITY;
  const float scale = (a.weight ? a.weight[n] : 1.f) * a.tau, g = scale * st.z / st.y;
  const F2 minus = F2::of(-st.x, -st.x), c2 = F2::of(a.c2, a.c2), g2 = F2::of(g, g);
  for (int32_t i0 = threadIdx.x; i0 < units; i0 += kBatch * kThreads) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int32_t u = i0 + k * kThreads;
      if (u >= units) break;
      if (!wide_loads) {
        T* e = reinterpret_cast<T*>(&raw[k]);
#pragma unroll
        for (int i = 0; i < U::n; ++i) e[i] = z[head + u * U::n + i];
      }
      F2 x[U::n / 2];
      U::widen(raw[k], x);
      load(k, u + kBatch * kThreads);
      float2 e[U::n / 2];
#pragma unroll
      for (int i = 0; i < U::n / 2; ++i) {
        const float2 y = ((x[i] + minus) * c2).get();
        e[i] = (F2::of(ex2(y.x), ex2(y.y)) * g2).get();
      }
      uint4 w = part ? U::narrow(e) : make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(dz + head)[u] = w;
    }
  }
  for (int32_t o = threadIdx.x; o < len - units * U::n; o += kThreads) {
    const int32_t e = o < head ? o : o + units * U::n;
    dz[e] = Elem<T>::put(part ? g * ex2((Elem<T>::get(z[e]) - st.x) * a.c2) : 0.f);
  }
  if (!part) return;
  __syncthreads();
  for (int k = threadIdx.x; k < a.K; k += kThreads)
    if (l.id[k] >= 0 && is_first(l, k))
      dz[l.id[k]] = Elem<T>::put(scale * (ex2((l.z[k] - st.x) * a.c2) / st.y - q_of_token(l, k, a.K)));
}

template <typename T>
cudaError_t launch_rows(int device, bool grad, DistillArgs& a, cudaStream_t s) {
  // The smallest cluster whose slices leave room for three CTAs an SM; more CTAs for few
  // rows, while the GPU has not one each and slices stay above kSliceLeast.
  int log_ctas = 0;
  auto slice_of = [&] { return (int32_t)((((int64_t)a.V + (1 << log_ctas) - 1) / (1 << log_ctas) + 63) / 64 * 64); };
  while ((1 << log_ctas) < kMaxCluster && slice_bytes<T>(slice_of()) > kSliceWanted) ++log_ctas;
  while ((1 << log_ctas) < kMaxCluster && ((int64_t)a.N << log_ctas) < sm_count(device) &&
         slice_bytes<T>(slice_of()) > kSliceLeast)
    ++log_ctas;
  int32_t slice = slice_of();
  if (slice_bytes<T>(slice) <= kSliceMost && ((int64_t)a.N << log_ctas) <= INT32_MAX) {
    const void* fn = grad ? reinterpret_cast<const void*>(&k_distill_cluster<T, true>)
                          : reinterpret_cast<const void*>(&k_distill_cluster<T, false>);
    static bool ready[2][64];
    constexpr size_t most = kSliceMost + bitmap_bytes(kSliceMost / sizeof(T)) + kMaxList * 12;
    static_assert(most < 225 * 1024, "");
    const cudaError_t e = allow_smem(fn, most, device, ready[grad]);
    if (e != cudaSuccess) return e;
    void* args[] = {&a, &slice, &log_ctas};
    return launch_clusters(fn, dim3((unsigned)a.N << log_ctas), dim3(kRowThreads), 1 << log_ctas,
                           cluster_smem<T>(slice, a.K), s, args);
  }
  const void* fn = grad ? reinterpret_cast<const void*>(&k_distill_wide<T, true>)
                        : reinterpret_cast<const void*>(&k_distill_wide<T, false>);
  static bool ready[2][64];
  const cudaError_t e = allow_smem(fn, kMaxVocab / 8 + kMaxList * 12, device, ready[grad]);
  if (e != cudaSuccess) return e;
  void* args[] = {&a};
  return launch_kernel(fn, dim3(a.N), dim3(kRowThreads), (size_t)((a.V + 31) / 32) * 4 + (size_t)a.K * 12, s, args, false);
}

template <typename T>
cudaError_t launch_mode(int device, int mode, DistillArgs& a, cudaStream_t s) {
  if (mode != kBackward) return launch_rows<T>(device, mode == kStep, a, s);
  int32_t pieces = (a.V + kPiece - 1) / kPiece;
  void* args[] = {&a, &pieces};
  return launch_kernel(reinterpret_cast<const void*>(&k_distill_backward<T>), dim3((unsigned)a.N * pieces),
                       dim3(kThreads), (size_t)a.K * 12, s, args, false);
}

emb_status distill(int device, int mode, int dtype, DistillArgs a, void* stream) {
  if (device < 0 || a.N < 0 || a.N > kMaxDistillRows || a.V < 1 || a.V > kMaxVocab || a.K < 0 || a.K > kMaxList) return EMB_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || !dtype_ok(a.t_dtype)) return EMB_ERR_INVALID_ARG;
  if (!(a.tau > 0.f) || !std::isfinite(a.tau)) return EMB_ERR_INVALID_ARG;
  if (!aligned(a.ids, 8) || !aligned(a.t, dtype_size(a.t_dtype)) || !aligned(a.lse, 4) || !aligned(a.weight, 4) ||
      !aligned(a.loss, 4) || !aligned(a.stats, 16) || !aligned(a.status, 4))
    return EMB_ERR_INVALID_ARG;
  if (a.N == 0) return EMB_OK;
  if (!a.z || !aligned(a.z, dtype_size(dtype)) || (a.K > 0 && (!a.ids || !a.t))) return EMB_ERR_INVALID_ARG;
  if (a.N > 1 && (a.z_stride < a.V || a.t_stride < a.K)) return EMB_ERR_INVALID_ARG;
  if (mode != kBackward && !a.loss) return EMB_ERR_INVALID_ARG;
  if (mode != kStep && !a.stats) return EMB_ERR_INVALID_ARG;
  if (mode != kForward) {
    if (!a.dz || !aligned(a.dz, dtype_size(dtype)) || (a.N > 1 && a.dz_stride < a.V)) return EMB_ERR_INVALID_ARG;
    if (a.dz == a.z && a.N > 1 && a.dz_stride != a.z_stride) return EMB_ERR_INVALID_ARG;
  }
  a.c2 = (float)(1.4426950408889634 / (double)a.tau);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return on_device(device, [&] {
    switch (dtype) {
      case EMB_F32: return launch_mode<float>(device, mode, a, s);
      case EMB_F16: return launch_mode<__half>(device, mode, a, s);
      default: return launch_mode<__nv_bfloat16>(device, mode, a, s);
    }
  });
}

}  // namespace
}  // namespace embbwd

using namespace embbwd;

extern "C" emb_status emb_distill_forward(int device, const void* logits, emb_dtype logits_dtype, int64_t logits_stride,
                                          int32_t N, int32_t V, const int64_t* teacher_ids, const void* teacher_logits,
                                          emb_dtype teacher_dtype, int64_t teacher_stride, int32_t K,
                                          const float* teacher_lse, float temperature, float* loss, float* stats,
                                          uint32_t* device_status, void* stream) {
  DistillArgs a{};
  a.z = logits, a.z_stride = logits_stride, a.N = N, a.V = V, a.K = K, a.ids = teacher_ids, a.t = teacher_logits;
  a.t_dtype = teacher_dtype, a.t_stride = teacher_stride, a.lse = teacher_lse, a.tau = temperature, a.loss = loss;
  a.stats = reinterpret_cast<float4*>(stats), a.status = device_status;
  return distill(device, kForward, logits_dtype, a, stream);
}

extern "C" emb_status emb_distill_backward(int device, const void* logits, emb_dtype logits_dtype,
                                           int64_t logits_stride, int32_t N, int32_t V, const int64_t* teacher_ids,
                                           const void* teacher_logits, emb_dtype teacher_dtype, int64_t teacher_stride,
                                           int32_t K, const float* stats, const float* row_weight, float temperature,
                                           void* dlogits, int64_t dlogits_stride, uint32_t* device_status,
                                           void* stream) {
  DistillArgs a{};
  a.z = logits, a.z_stride = logits_stride, a.N = N, a.V = V, a.K = K, a.ids = teacher_ids, a.t = teacher_logits;
  a.t_dtype = teacher_dtype, a.t_stride = teacher_stride, a.weight = row_weight, a.tau = temperature;
  a.stats = reinterpret_cast<float4*>(const_cast<float*>(stats)), a.dz = dlogits, a.dz_stride = dlogits_stride;
  a.status = device_status;
  return distill(device, kBackward, logits_dtype, a, stream);
}

extern "C" emb_status emb_distill_step(int device, const void* logits, emb_dtype logits_dtype, int64_t logits_stride,
                                       int32_t N, int32_t V, const int64_t* teacher_ids, const void* teacher_logits,
                                       emb_dtype teacher_dtype, int64_t teacher_stride, int32_t K,
                                       const float* teacher_lse, const float* row_weight, float temperature, float* loss,
                                       void* dlogits, int64_t dlogits_stride, uint32_t* device_status, void* stream) {
  DistillArgs a{};
  a.z = logits, a.z_stride = logits_stride, a.N = N, a.V = V, a.K = K, a.ids = teacher_ids, a.t = teacher_logits;
  a.t_dtype = teacher_dtype, a.t_stride = teacher_stride, a.lse = teacher_lse, a.weight = row_weight;
  a.tau = temperature, a.loss = loss, a.dz = dlogits, a.dz_stride = dlogits_stride, a.status = device_status;
  return distill(device, kStep, logits_dtype, a, stream);
}
