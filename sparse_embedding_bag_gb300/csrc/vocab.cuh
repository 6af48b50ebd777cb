// Helpers shared by the vocabulary operators (logits.cu, distill.cu, micro.cu,
// micro_matmul.cu): element types, block reductions, and the host-side frame of
// an entry point that works without a plan.
#pragma once

#include "../../include/embbwd.h"
#include "internal.cuh"

namespace embbwd {

// Bits of the device status word of a vocabulary call (kErrIndex, kErrOffsets,
// kErrTimeout), added by the kernels when the caller passes one.
__device__ __forceinline__ void report(uint32_t* status, uint32_t bits) {
  if (status) atomicOr(status, bits);
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  __device__ __forceinline__ static float get(float x) { return x; }
  __device__ __forceinline__ static float put(float x) { return x; }
};
template <>
struct Elem<__half> {
  __device__ __forceinline__ static float get(__half x) { return __half2float(x); }
  __device__ __forceinline__ static __half put(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<__nv_bfloat16> {
  __device__ __forceinline__ static float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  __device__ __forceinline__ static __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

// Element i of an array of a type known at run time (short lists only).
__device__ __forceinline__ float load_as_float(const void* p, int dtype, int64_t i) {
  if (dtype == EMB_F32) return static_cast<const float*>(p)[i];
  if (dtype == EMB_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

constexpr int kGroup = 8;  // elements of a row that a thread takes together

// Eight consecutive elements, 16-byte aligned: the load and the widening apart.
template <typename T>
struct Raw8 {
  static constexpr int n = 16 / sizeof(T);
  uint4 u[kGroup / n];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kGroup / n; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void widen(float (&x)[kGroup]) const {
#pragma unroll
    for (int i = 0; i < kGroup / n; ++i) {
      const T* e = reinterpret_cast<const T*>(&u[i]);
#pragma unroll
      for (int k = 0; k < n; ++k) x[i * n + k] = Elem<T>::get(e[k]);
    }
  }
};
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[kGroup]) {
  constexpr int n = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < kGroup / n; ++i) {
    uint4 u;
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int k = 0; k < n; ++k) e[k] = Elem<T>::put(x[i * n + k]);
    reinterpret_cast<uint4*>(p)[i] = u;
  }
}

constexpr int32_t kMaxVocab = 1 << 20;  // widest row of logits

// Sums (maxima) over a block of up to 1024 threads, the same for every thread.
// `scratch` holds 33 floats. The order of additions is fixed. fmaxf drops NaN:
// a NaN among the values has to reach the result by another way (a sum).
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <bool kMax>
__device__ __forceinline__ float block_all(float v, float* scratch) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  v = kMax ? warp_max(v) : warp_sum(v);
  __syncthreads();  // scratch may still be read from the reduction before
  if (lane == 0) scratch[warp] = v;
  __syncthreads();
  v = lane < warps ? scratch[lane] : (kMax ? -INFINITY : 0.f);
  return kMax ? warp_max(v) : warp_sum(v);
}

// Both sums (maxima) over a block; `scratch` holds 64 floats.
template <bool kMax>
__device__ __forceinline__ void block_both(float& u, float& v, float* scratch) {
  constexpr float none = kMax ? -INFINITY : 0.f;
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  u = kMax ? warp_max(u) : warp_sum(u), v = kMax ? warp_max(v) : warp_sum(v);
  __syncthreads();
  if (lane == 0) scratch[warp] = u, scratch[32 + warp] = v;
  __syncthreads();
  u = lane < warps ? scratch[lane] : none, v = lane < warps ? scratch[32 + lane] : none;
  u = kMax ? warp_max(u) : warp_sum(u), v = kMax ? warp_max(v) : warp_sum(v);
}

// ---- host side

inline size_t dtype_size(int d) { return d == EMB_F32 ? 4 : 2; }
inline bool dtype_ok(int d) { return d >= EMB_F32 && d <= EMB_BF16; }
inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Runs `body` (a launch that returns a cudaError_t) with `device` current and
// puts the caller's device back.
template <typename F>
inline emb_status on_device(int device, F body) {
  int prev = -1;
  if (cudaGetDevice(&prev) != cudaSuccess) {
    prev = -1;
    cudaGetLastError();
  }
  if (prev != device && cudaSetDevice(device) != cudaSuccess) {
    cudaGetLastError();
    return EMB_ERR_CUDA;
  }
  const cudaError_t e = body();
  if (prev >= 0 && prev != device) cudaSetDevice(prev);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return EMB_ERR_CUDA;
  }
  return EMB_OK;
}

}  // namespace embbwd
