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
// Exponentials are base 2: p_v = 2^(z_v c - M c) / S with c = log2(e) / tau and M
// the row's largest logit. Sums are held in fp32.
#include <cmath>

#include "vocab.cuh"

namespace embbwd {
namespace {

constexpr int kMaxList = 1024;   // longest teacher list
constexpr int kRowThreads = 512;

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
  int32_t id[kMaxList];  // -1: no entry
  float q[kMaxList];
  float z[kMaxList];     // the student's logit there
  float scratch[36];
  int repeated;          // some id occurs more than once
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

// Reads the list; returns whether the row takes part. Sets l.q (given L, which is
// found first if the caller has none), *L and *qsum.
template <typename T>
__device__ bool read_list(const DistillArgs& a, int32_t n, List& l, float known_L, bool known, float* L, float* qsum) {
  const T* z = static_cast<const T*>(a.z) + n * a.z_stride;
  float big = -INFINITY, any = 0.f;
  for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
    const int64_t id = a.ids[n * a.t_stride + k];
    if (id < -1 || id >= a.V) report(a.status, kErrIndex);
    const bool ok = id >= 0 && id < a.V;
    l.id[k] = ok ? (int32_t)id : -1;
    const float t = ok ? __fdiv_rn(load_as_float(a.t, a.t_dtype, n * a.t_stride + k), a.tau) : -INFINITY;
    l.q[k] = t;
    l.z[k] = ok ? Elem<T>::get(z[id]) : 0.f;
    if (ok) any = 1.f;
    big = fmaxf(big, t);
  }
  *L = 0.f;
  if (block_all<false>(any, l.scratch) == 0.f) return false;
  *L = known_L;
  if (!known) {
    big = block_all<true>(big, l.scratch);
    float s = 0.f;
    for (int k = threadIdx.x; k < a.K; k += blockDim.x) s += expf(l.q[k] - (isinf(big) ? 0.f : big));
    s = block_all<false>(s, l.scratch);
    *L = -INFINITY;
    if (s == 0.f) return false;
    *L = (isinf(big) ? 0.f : big) + logf(s);
  }
  if (*L == -INFINITY) return false;
  float s = 0.f;
  for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
    const float q = l.id[k] >= 0 ? expf(l.q[k] - *L) : 0.f;
    l.q[k] = q;
    s += q;
  }
  *qsum = block_all<false>(s, l.scratch);
  return true;
}

// One block a row; the row is read once for its largest logit, once for its sums
// and once for its gradient. A bitmap of the vocabulary marks the list.
template <typename T, int kMode>
__global__ void __launch_bounds__(kRowThreads) k_distill_row(DistillArgs a) {
  extern __shared__ uint32_t on_list[];
  __shared__ List l;
  const int32_t n = blockIdx.x;
  const T* z = static_cast<const T*>(a.z) + n * a.z_stride;
  T* dz = static_cast<T*>(a.dz) + n * a.dz_stride;
  for (int i = threadIdx.x; i < (a.V + 31) / 32; i += kRowThreads) on_list[i] = 0;
  if (threadIdx.x == 0) l.repeated = 0;
  __syncthreads();
  float4 st = make_float4(0.f, 1.f, 0.f, 0.f);
  if (kMode == kBackward) st = a.stats[n];
  float L = 0.f, qsum = 0.f;
  const bool known = kMode == kBackward || a.lse != nullptr;
  const float known_L = kMode == kBackward ? st.w : (a.lse ? a.lse[n] : 0.f);
  if (!read_list<T>(a, n, l, known_L, known, &L, &qsum)) {
    if (threadIdx.x == 0) {
      if (kMode != kBackward) a.loss[n] = 0.f;
      if (kMode == kForward) a.stats[n] = make_float4(0.f, 1.f, 0.f, L);
    }
    if (kMode != kForward)
      for (int32_t v = threadIdx.x; v < a.V; v += kRowThreads) dz[v] = Elem<T>::put(0.f);
    return;
  }
  for (int k = threadIdx.x; k < a.K; k += kRowThreads)
    if (l.id[k] >= 0) {
      const uint32_t bit = 1u << (l.id[k] & 31);
      if (atomicOr(&on_list[l.id[k] >> 5], bit) & bit) l.repeated = 1;
    }
  __syncthreads();
  if (kMode != kBackward) {
    float m = -INFINITY;
    for (int32_t v = threadIdx.x; v < a.V; v += kRowThreads) m = fmaxf(m, Elem<T>::get(z[v]));
    m = block_all<true>(m, l.scratch);
    const float mc = m * a.c2;
    float rest = 0.f, top = 0.f;
    for (int32_t v = threadIdx.x; v < a.V; v += kRowThreads)
      if (!(on_list[v >> 5] >> (v & 31) & 1u)) rest += exp2f(fmaf(Elem<T>::get(z[v]), a.c2, -mc));
    rest = block_all<false>(rest, l.scratch);
    for (int k = threadIdx.x; k < a.K; k += kRowThreads)
      if (l.id[k] >= 0 && is_first(l, k)) top += exp2f(fmaf(l.z[k], a.c2, -mc));
    top = block_all<false>(top, l.scratch);
    const float S = rest + top, logS = logf(S);
    float ls = 0.f;
    for (int k = threadIdx.x; k < a.K; k += kRowThreads)
      if (l.q[k] > 0.f) {
        const float logp = fmaf(l.z[k], a.c2, -mc) * kLn2 - logS;
        ls += l.q[k] * ((__fdiv_rn(load_as_float(a.t, a.t_dtype, n * a.t_stride + k), a.tau) - L) - logp);
      } else if (!(l.q[k] == 0.f)) {
        ls = NAN;
      }
    ls = block_all<false>(ls, l.scratch);
    float coef = 1.f;
    if (a.lse) {
      const float r = fmaxf(0.f, 1.f - qsum), u = rest / S;
      if (r > 0.f) {
        ls += r * (logf(r) - logf(u));
        coef = 1.f - r / u;
      }
    }
    st = make_float4(m, S, coef, L);
    if (threadIdx.x == 0) {
      a.loss[n] = a.tau * a.tau * ls;
      if (kMode == kForward) a.stats[n] = st;
    }
  }
  if (kMode == kForward) return;
  const float mc = st.x * a.c2, scale = (a.weight ? a.weight[n] : 1.f) * a.tau / st.y;
  for (int32_t v = threadIdx.x; v < a.V; v += kRowThreads)
    if (!(on_list[v >> 5] >> (v & 31) & 1u))
      dz[v] = Elem<T>::put(scale * st.z * exp2f(fmaf(Elem<T>::get(z[v]), a.c2, -mc)));
  for (int k = threadIdx.x; k < a.K; k += kRowThreads)
    if (l.id[k] >= 0 && is_first(l, k))
      dz[l.id[k]] = Elem<T>::put(scale * (exp2f(fmaf(l.z[k], a.c2, -mc)) - q_of_token(l, k, a.K) * st.y));
}

template <typename T>
const void* row_kernel(int mode) {
  switch (mode) {
    case kForward: return reinterpret_cast<const void*>(&k_distill_row<T, kForward>);
    case kBackward: return reinterpret_cast<const void*>(&k_distill_row<T, kBackward>);
    default: return reinterpret_cast<const void*>(&k_distill_row<T, kStep>);
  }
}

const void* distill_kernel(int dtype, int mode) {
  switch (dtype) {
    case EMB_F32: return row_kernel<float>(mode);
    case EMB_F16: return row_kernel<__half>(mode);
    default: return row_kernel<__nv_bfloat16>(mode);
  }
}

emb_status distill(int device, int mode, int dtype, DistillArgs a, void* stream) {
  if (device < 0 || a.N < 0 || a.V < 1 || a.V > kMaxVocab || a.K < 0 || a.K > kMaxList) return EMB_ERR_INVALID_ARG;
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
  return on_device(device, [&] {
    void* args[] = {&a};
    const void* fn = distill_kernel(dtype, mode);
    const size_t smem = (size_t)((a.V + 31) / 32) * 4;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(fn, dim3(a.N), dim3(kRowThreads), smem, static_cast<cudaStream_t>(stream), args, false);
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
