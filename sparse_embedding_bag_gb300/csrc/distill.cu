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
// cancel for a student that agrees with its teacher. The sum is relative to a
// reference near the largest logit off the list: relative to the row's largest, which is
// usually a listed one, it underflows once the listed tokens lead by 87 tau. Entries with
// id -1 are padding; a row without entries, or whose teacher has no mass (L = -infinity),
// has loss 0 and gradient 0. With no finite logit off the list u is 0: an r that rounding
// explains counts as 0, a larger one makes the loss infinite; either way the gradient
// off the list is 0.
//
// Exponentials are base 2: 2^((z_v - ref) c), c = log2(e) / tau. Differences come first, so
// that rows masked with the type's lowest value neither overflow nor lose their maximum.
// Sums are held in fp32.
//
// Forward and step: a cluster of CTAs takes a row, a part of it each. It streams its part
// from HBM with a running reference (sums are rescaled when a value exceeds it by far, which
// is rare after the first), the cluster exchanges largest logits and sums through
// distributed shared memory in one round, and the step streams the part once more. Rows of
// 128256 16-bit logits are still in L2 then (49 MB under way of its 129): HBM reads 269 MB
// for 263 MB of rows. fp32 rows of that length mostly are not (97 MB under way, and their
// gradients: 972 MB for 525), nor are rows of 2^20, whose parts are longer (bf16 1075 MB for
// 537, fp32 2150 for 1074). 4096 x 128256 bf16 take 388 us (5.3 TB/s of one read and one
// write), fp32 905 (4.6); 256 x 2^20 bf16 249 (4.3), fp32 515 (4.2).
// Backward (its sums are known): blocks over pieces of the rows, one read and one write.
// Holding the rows in shared memory instead (bulk copies, three CTAs of 64 KB an SM) took
// 474 us a step at 4096 x 128256 bf16, against 388: a CTA does nothing else while its
// slice arrives, and reads it three times.
#include <cmath>

#include "sm103.cuh"

namespace embbwd {
namespace {

constexpr int kMaxList = 1024;   // longest teacher list
constexpr int kMaxCluster = 8;
constexpr int kRowBlocks = 5;                       // CTAs an SM of the row kernel
constexpr int kBatch = 4;                           // 16-byte loads a thread has in flight
constexpr int32_t kPartLeast = 2048;                // elements of a CTA's part of a row
constexpr int32_t kMaxDistillRows = 1 << 23;        // (rows x pieces of a row stay below 2^31)
constexpr int kPieceMost = 32768, kPieceLeast = 2048;      // elements of a block of the backward, a power of two

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
  float tau, inv_tau, c2;  // c2 = log2(e) / tau
  float* loss;
  float4* stats;         // written by the forward, read by the backward
  void* dz;
  int64_t dz_stride;
  uint32_t* status;
};

// t_k / tau, as a product with the reciprocal, rounded: what is subtracted from it later
// must not meet an unrounded product where L came from rounded ones.
__device__ __forceinline__ float teacher_logit(const DistillArgs& a, int32_t n, int k) {
  return __fmul_rn(load_as_float(a.t, a.t_dtype, n * a.t_stride + k), a.inv_tau);
}

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
    const float t = id >= 0 ? teacher_logit(a, n, k) : -INFINITY;
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
      const float logp = __fmul_rn(l.z[k] - M, a.inv_tau) - logS;
      ls += l.q[k] * ((teacher_logit(a, n, k) - L) - logp);
    } else if (!(l.q[k] == 0.f)) {
      ls = NAN;
    }
  return block_all<false>(ls, scratch);
}

// 2^((a - b) c), 1 for equal ones (infinities among them).
__device__ __forceinline__ float power_of(float a, float b, float c2) { return a == b ? 1.f : ex2((a - b) * c2); }

// r / u above 2^kLargeRatio is held by its binary logarithm: a coefficient above 1.
constexpr float kLargeRatio = 64.f;

// The remaining mass's part of the loss (without tau^2), and the coefficient off the list.
// `off` is the sum there relative to `ref`.
__device__ __forceinline__ float tail_of(const DistillArgs& a, float qsum, float L, float off, float ref, float S,
                                         float M, float* coef) {
  const float r = fmaxf(0.f, 1.f - qsum);
  *coef = 1.f;
  // Each q carries a few roundings of values up to |L| + |log q|, L the caller's as many.
  if (off == 0.f) return r > 0x1p-24f * (8.f * fabsf(L) + (float)a.K + 32.f) ? INFINITY : 0.f;
  if (!(r > 0.f)) return 0.f;
  const float ratio = logf(r) - (__fmul_rn(ref - M, a.inv_tau) + (logf(off) - logf(S)));  // log(r / u)
  const float lg = ratio * 1.44269504f;
  *coef = lg > kLargeRatio ? lg : 1.f - r / (off * power_of(ref, M, a.c2) / S);
  return r * ratio;
}

// The gradient off the list is g 2^((z - ref) c): (scale / S) coef 2^((z - M) c). The exponent
// takes up a coefficient far below 0, so that no power underflows whose product with it
// does not.
__device__ __forceinline__ void off_list(const DistillArgs& a, float coef, float scale, float M, float S, float* ref,
                                         float* g) {
  *ref = M, *g = scale * coef / S;
  if (coef > 1.f || coef < -65536.f) *ref = M - (coef > 1.f ? coef : log2f(-coef)) / a.c2, *g = -scale / S;
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

// How a part of a row at p is cut into 16-byte units: the first starts `head` elements into
// it, at a multiple of 16 bytes.
template <typename T>
struct Cut {
  int32_t head, units;
  __device__ __forceinline__ Cut(const T* p, int32_t len) {
    constexpr int n = Unit<T>::n;
    head = min(len, (int32_t)(-(reinterpret_cast<uintptr_t>(p) / sizeof(T)) % n)), units = (len - head) / n;
  }
  template <bool kWide>
  __device__ __forceinline__ uint4 load(const T* z, int32_t u) const {
    constexpr int n = Unit<T>::n;
    if (kWide) return reinterpret_cast<const uint4*>(z + head)[u];
    uint4 v;
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int i = 0; i < n; ++i) e[i] = z[head + u * n + i];
    return v;
  }
  // Elements beside the units, by number from 0 to len - units * n - 1.
  __device__ __forceinline__ int32_t beside(int32_t o) const { return o < head ? o : o + units * Unit<T>::n; }
};

// 2^((x - ref) c) of a unit.
template <int n>
__device__ __forceinline__ void powers(const F2 (&x)[n], F2 minus_ref, F2 c2, F2 (&e)[n]) {
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const float2 y = ((x[i] + minus_ref) * c2).get();
    e[i] = F2::of(ex2(y.x), ex2(y.y));
  }
}

// f(unit number, its elements as pairs, the largest of them) for a thread's units of a
// part, kBatch loads ahead; `raw` holds the first.
template <bool kWide, typename T, typename F>
__device__ __forceinline__ void for_units(const T* z, const Cut<T>& cut, uint4 (&raw)[kBatch], F f) {
  using U = Unit<T>;
  for (int32_t u0 = threadIdx.x; u0 < cut.units; u0 += kBatch * kThreads) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int32_t u = u0 + k * kThreads;
      if (u >= cut.units) break;
      const float most = U::max_of(raw[k]);
      F2 x[U::n / 2];
      U::widen(raw[k], x);
      if (u + kBatch * kThreads < cut.units) raw[k] = cut.template load<kWide>(z, u + kBatch * kThreads);
      f(u, x, most);
    }
  }
}

// A thread's first units of a part, asked for ahead of their use.
template <bool kWide, typename T>
__device__ __forceinline__ void load_first(const T* z, const Cut<T>& cut, uint4 (&raw)[kBatch]) {
#pragma unroll
  for (int k = 0; k < kBatch; ++k)
    if ((int)threadIdx.x + k * kThreads < cut.units)
      raw[k] = cut.template load<kWide>(z, threadIdx.x + k * kThreads);
}

// The gradient of a part of a row off the list: g 2^((z - ref) c).
template <bool kWide, typename T>
__device__ __forceinline__ void store_gradient(const T* z, T* dz, int32_t len, const Cut<T>& cut, uint4 (&raw)[kBatch],
                                               float c, float ref, float g) {
  using U = Unit<T>;
  const F2 g2 = F2::of(g, g), c2 = F2::of(c, c), minus_ref = F2::of(-ref, -ref);
  uint4* out = reinterpret_cast<uint4*>(dz + cut.head);
  for_units<kWide>(z, cut, raw, [&](int32_t u, const F2 (&x)[U::n / 2], float) {
    F2 e[U::n / 2];
    float2 w[U::n / 2];
    powers(x, minus_ref, c2, e);
#pragma unroll
    for (int i = 0; i < U::n / 2; ++i) w[i] = (e[i] * g2).get();
    out[u] = U::narrow(w);
  });
  for (int32_t o = threadIdx.x; o < len - cut.units * U::n; o += kThreads) {
    const int32_t e = cut.beside(o);
    dz[e] = Elem<T>::put(g * ex2((Elem<T>::get(z[e]) - ref) * c));
  }
}
template <typename T>
__device__ __forceinline__ void store_zeros(T* dz, int32_t len, const Cut<T>& cut) {
  for (int32_t u = threadIdx.x; u < cut.units; u += kThreads)
    reinterpret_cast<uint4*>(dz + cut.head)[u] = make_uint4(0, 0, 0, 0);
  for (int32_t o = threadIdx.x; o < len - cut.units * Unit<T>::n; o += kThreads) dz[cut.beside(o)] = Elem<T>::put(0.f);
}

// The listed tokens' gradient, stored over what store_gradient left there. Entries hold
// elements of the part (-1: another part's).
template <typename T>
__device__ __forceinline__ void store_listed(const DistillArgs& a, T* dz, const List& l, float scale, float M,
                                             float S) {
  for (int k = threadIdx.x; k < a.K; k += kThreads)
    if (l.id[k] >= 0 && is_first(l, k))
      dz[l.id[k]] = Elem<T>::put(scale * (ex2((l.z[k] - M) * a.c2) / S - q_of_token(l, k, a.K)));
}

// Marks the list's tokens of [r0, r0 + len) in a bitmap: element e at bit e + first.
__device__ __forceinline__ void mark_list(const DistillArgs& a, List& l, uint32_t* bitmap, int32_t r0, int32_t len,
                                          int32_t first) {
  for (int k = threadIdx.x; k < a.K; k += kThreads) {
    const int32_t e = l.id[k] - r0, p = e + first;
    if (l.id[k] < 0 || e < 0 || e >= len) continue;
    if (atomicOr(&bitmap[p >> 5], 1u << (p & 31)) >> (p & 31) & 1u) l.repeated = 1;
  }
}

// A cluster a row, `part_len` elements (a multiple of 64) a CTA.
template <typename T, bool kGrad, bool kWide>
__global__ void __launch_bounds__(kThreads, kRowBlocks) k_distill_rows(DistillArgs a, int32_t part_len, int log_ctas) {
  using U = Unit<T>;
  extern __shared__ __align__(16) uint32_t bitmap[];  // of the part; then the list
  __shared__ List l;
  __shared__ float scratch[64];
  __shared__ float4 parts[kMaxCluster];  // of every CTA: largest logit, reference off the list, sums off and on it
  cluster_arrive();  // shared memory of a CTA is written by others only once it runs
  const uint32_t ctas = 1u << log_ctas, rank = blockIdx.x & (ctas - 1);
  const int32_t n = blockIdx.x >> log_ctas;
  const int32_t r0 = min((int64_t)a.V, (int64_t)rank * part_len), len = min(a.V - r0, part_len);
  const T* z = static_cast<const T*>(a.z) + n * a.z_stride + r0;
  T* dz = kGrad ? static_cast<T*>(a.dz) + n * a.dz_stride + r0 : nullptr;
  pdl_wait();
  const Cut<T> cut(z, len);  // the order of the sums goes by the logits' alignment alone
  uint4 raw[kBatch];
  load_first<true>(z, cut, raw);
  const int32_t words = part_len / 32 + 1;  // units' bits start at bit 8: a byte or half of one each
  const int32_t first = 8 - cut.head;
  for (int32_t i = threadIdx.x; i < words; i += kThreads) bitmap[i] = 0;
  if (threadIdx.x == 0) {
    l.id = reinterpret_cast<int32_t*>(bitmap + words), l.q = reinterpret_cast<float*>(l.id + a.K), l.z = l.q + a.K;
    l.repeated = 0;
  }
  __syncthreads();
  // CTA 0 finds the loss: it needs the student's logit of every entry
  const int32_t lo = rank == 0 ? 0 : r0, hi = rank == 0 ? a.V : r0 + len;
  float L = 0.f, qsum = 0.f;
  const bool part =
      read_ids(a, n, l) &&
      read_list<T>(a, n, l, scratch, lo, hi, a.lse ? a.lse[n] : 0.f, a.lse != nullptr, &L, &qsum);
  if (!part) {  // the same for the whole cluster
    if (rank == 0 && threadIdx.x == 0) {
      a.loss[n] = 0.f;
      if (!kGrad) a.stats[n] = make_float4(0.f, 1.f, 0.f, L);
    }
    if (kGrad) store_zeros(dz, len, Cut<T>(dz, len));
    __syncwarp();
    cluster_wait();
    return;
  }
  mark_list(a, l, bitmap, r0, len, first);
  __syncthreads();
  // This thread's largest logit, and its sum off the list relative to a reference that is
  // raised when a value there exceeds it by a factor of 2^kSlack.
  constexpr float kSlack = 16.f;
  const float slack = kSlack / a.c2;
  float m = -INFINITY, ref = -3.402823466e38f;
  const F2 c2 = F2::of(a.c2, a.c2);
  F2 sum = F2::of(0.f, 0.f);
  auto raise = [&](float most) {
    if (most > ref + slack) {
      const float f = ex2((ref - most) * a.c2);
      sum = sum * F2::of(f, f);
      ref = most;
    }
  };
  const uint8_t* on_list = reinterpret_cast<const uint8_t*>(bitmap) + 1;
  for_units<true>(z, cut, raw, [&](int32_t u, F2 (&x)[U::n / 2], float most) {
    m = fmaxf(m, most);
    F2 e[U::n / 2];
    const uint32_t bits = U::n == 8 ? on_list[u] : on_list[u >> 1] >> (u & 1) * 4 & 15u;
    auto mask = [&] {
#pragma unroll
      for (int i = 0; i < U::n / 2; ++i) {
        const float2 y = x[i].get();
        x[i] = F2::of(bits >> 2 * i & 1u ? -INFINITY : y.x, bits >> 2 * i & 2u ? -INFINITY : y.y);
      }
    };
    if (most > ref + slack) {
      if (bits) {
        mask();
        most = -INFINITY;
#pragma unroll
        for (int i = 0; i < U::n / 2; ++i) most = fmaxf(most, fmaxf(x[i].get().x, x[i].get().y));
      }
      raise(most);
    }
    if (bits) mask();
    powers(x, F2::of(-ref, -ref), c2, e);
#pragma unroll
    for (int i = 0; i < U::n / 2; ++i) sum = sum + e[i];
  });
  for (int32_t o = threadIdx.x; o < len - cut.units * U::n; o += kThreads) {
    const int32_t e = cut.beside(o);
    const float x = Elem<T>::get(z[e]);
    m = fmaxf(m, x);
    if (bitmap[(e + first) >> 5] >> ((e + first) & 31) & 1u) continue;
    raise(x);
    sum = sum + F2::of(ex2((x - ref) * a.c2), 0.f);
  }
  const Cut<T> again(kGrad ? dz : z, len);
  if (kGrad) load_first<kWide>(z, again, raw);
  // the part's largest logit and reference, and its sums relative to them (with nothing but
  // -infinity there is none)
  float rest = sum.get().x + sum.get().y, top = 0.f, M = m, R = ref;
  block_both<true>(M, R, scratch);
  rest *= power_of(ref, R, a.c2);
  const float base = M == -INFINITY ? 0.f : M;
  for (int k = threadIdx.x; k < a.K; k += kThreads) {
    const int32_t e = l.id[k] - r0;
    if (l.id[k] >= 0 && e >= 0 && e < len && is_first(l, k)) top += ex2((l.z[k] - base) * a.c2);
  }
  block_both<false>(rest, top, scratch);
  __syncwarp();
  cluster_wait();
  if (threadIdx.x < ctas)
    cluster_store(cluster_map(smem_u32(&parts[rank]), threadIdx.x), make_float4(M, R, rest, top));
  __syncwarp();
  cluster_sync();
  // a lane a part, the same in every group of kMaxCluster lanes
  const uint32_t part_of = threadIdx.x % kMaxCluster;
  const float4 of_part = part_of < ctas ? parts[part_of] : make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
  M = of_part.x, R = of_part.y;
#pragma unroll
  for (int o = 1; o < kMaxCluster; o *= 2)
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o)), R = fmaxf(R, __shfl_xor_sync(0xffffffffu, R, o));
  float off = of_part.z * power_of(of_part.y, R, a.c2), S = of_part.w * power_of(of_part.x, M, a.c2);
#pragma unroll
  for (int o = 1; o < kMaxCluster; o *= 2)
    off += __shfl_xor_sync(0xffffffffu, off, o), S += __shfl_xor_sync(0xffffffffu, S, o);
  S += off * power_of(R, M, a.c2);
  float coef = 1.f;
  const float tail = a.lse ? tail_of(a, qsum, L, off, R, S, M, &coef) : 0.f;
  const float scale = (a.weight ? a.weight[n] : 1.f) * a.tau;
  if (kGrad) {
    float off_ref, g;
    off_list(a, coef, scale, M, S, &off_ref, &g);
    store_gradient<kWide>(z, dz, len, again, raw, a.c2, off_ref, g);
  }
  if (rank == 0) {
    const float loss = loss_of(a, n, l, scratch, M, S, L) + tail;
    if (threadIdx.x == 0) {
      a.loss[n] = a.tau * a.tau * loss;
      if (!kGrad) a.stats[n] = make_float4(M, S, coef, L);
    }
  }
  if (!kGrad) return;
  __syncthreads();
  for (int k = threadIdx.x; k < a.K; k += kThreads) {  // as elements of the part
    const int32_t e = l.id[k] - r0;
    l.id[k] = l.id[k] >= 0 && e >= 0 && e < len ? e : -1;
  }
  __syncthreads();
  store_listed(a, dz, l, scale, M, S);
}

// The gradient from the forward's sums: a block takes `piece` elements of a row.
template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads, kRowBlocks) k_distill_backward(DistillArgs a, int32_t pieces, int32_t piece) {
  extern __shared__ __align__(16) int32_t list[];
  __shared__ uint32_t bitmap[kPieceMost / 32];
  __shared__ List l;
  const int32_t n = blockIdx.x / (uint32_t)pieces, r0 = (blockIdx.x - (uint32_t)n * pieces) * piece;
  const int32_t len = min(a.V - r0, piece);
  const T* z = static_cast<const T*>(a.z) + n * a.z_stride + r0;
  T* dz = static_cast<T*>(a.dz) + n * a.dz_stride + r0;
  pdl_wait();
  pdl_trigger();
  const Cut<T> cut(dz, len);
  uint4 raw[kBatch];
  load_first<kWide>(z, cut, raw);
  const float4 st = a.stats[n];
  for (int i = threadIdx.x; i < piece / 32; i += kThreads) bitmap[i] = 0;
  if (threadIdx.x == 0)
    l.id = list, l.q = reinterpret_cast<float*>(list + a.K), l.z = l.q + a.K, l.repeated = 0;
  __syncthreads();
  const bool part = read_ids(a, n, l) && st.w != -INFINITY;
  for (int k = threadIdx.x; k < a.K; k += kThreads) {
    const int32_t e = l.id[k] - r0;
    if (l.id[k] < 0 || e < 0 || e >= len) {
      l.id[k] = -1;
      continue;
    }
    l.id[k] = e;
    l.q[k] = expf(teacher_logit(a, n, k) - st.w);
    l.z[k] = Elem<T>::get(z[e]);
    if (atomicOr(&bitmap[e >> 5], 1u << (e & 31)) >> (e & 31) & 1u) l.repeated = 1;
  }
  __syncthreads();  // in place, the listed logits are read before they are overwritten
  const float scale = (a.weight ? a.weight[n] : 1.f) * a.tau;
  if (!part) {
    store_zeros(dz, len, cut);
    return;
  }
  float ref, g;
  off_list(a, st.z, scale, st.x, st.y, &ref, &g);
  store_gradient<kWide>(z, dz, len, cut, raw, a.c2, ref, g);
  __syncthreads();
  store_listed(a, dz, l, scale, st.x, st.y);
}

// Do all rows of logits and gradient lie at the same places in 16 bytes? Then units that
// store 16 bytes load 16 bytes.
template <typename T>
bool wide_loads(const DistillArgs& a) {
  const uintptr_t z = reinterpret_cast<uintptr_t>(a.z), dz = reinterpret_cast<uintptr_t>(a.dz);
  return (z - dz) % 16 == 0 && (a.N == 1 || (a.z_stride - a.dz_stride) % Unit<T>::n == 0);
}

template <typename T>
cudaError_t launch_rows(int device, bool grad, DistillArgs& a, cudaStream_t s) {
  // Parts of at most 32768 elements (with a gradient: a part comes again, from L2 if it is
  // short enough) or 65536, as long as kMaxCluster of them hold the row, longer ones beyond;
  // smaller ones for few rows, while the GPU has not kRowBlocks CTAs an SM and parts stay
  // above kPartLeast.
  int log_ctas = 0;
  while ((1 << log_ctas) < kMaxCluster && (a.V >> log_ctas) > (grad ? 32768 : 65536)) ++log_ctas;
  while ((1 << log_ctas) < kMaxCluster && ((int64_t)a.N << log_ctas) < kRowBlocks * sm_count(device) &&
         (a.V >> log_ctas) > kPartLeast)
    ++log_ctas;
  int32_t part_len = ((a.V + (1 << log_ctas) - 1) >> log_ctas);
  part_len = (part_len + 63) / 64 * 64;
  const void* fn = !grad            ? reinterpret_cast<const void*>(&k_distill_rows<T, false, true>)
                   : wide_loads<T>(a) ? reinterpret_cast<const void*>(&k_distill_rows<T, true, true>)
                                      : reinterpret_cast<const void*>(&k_distill_rows<T, true, false>);
  void* args[] = {&a, &part_len, &log_ctas};
  return launch_clusters(fn, dim3((unsigned)a.N << log_ctas), dim3(kThreads), 1 << log_ctas,
                         (size_t)part_len / 8 + 4 + (size_t)a.K * 12, s, args, true);
}

template <typename T>
cudaError_t launch_mode(int device, int mode, DistillArgs& a, cudaStream_t s) {
  if (mode != kBackward) return launch_rows<T>(device, mode == kStep, a, s);
  // large pieces, so that the list is read by few blocks; smaller ones for few rows
  int32_t piece = kPieceMost;
  while (piece > kPieceLeast && (int64_t)a.N * ((a.V + piece - 1) / piece) < 2 * kRowBlocks * sm_count(device)) piece /= 2;
  int32_t pieces = (a.V + piece - 1) / piece;
  void* args[] = {&a, &pieces, &piece};
  const void* fn = wide_loads<T>(a) ? reinterpret_cast<const void*>(&k_distill_backward<T, true>)
                                    : reinterpret_cast<const void*>(&k_distill_backward<T, false>);
  return launch_kernel(fn, dim3((unsigned)a.N * pieces), dim3(kThreads), (size_t)a.K * 12, s, args, true);
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
  a.inv_tau = 1.f / a.tau;
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
