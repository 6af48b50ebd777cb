// Rows to microscaled 4-bit floating point, and back by row id.
#include <cmath>

#include "micro.cuh"

namespace embbwd {
namespace {

struct QuantArgs {
  const void* x;
  int64_t x_stride;
  int64_t R;
  int32_t K;
  float g;
  uint8_t* codes;
  uint8_t* scales;
};

// A thread takes one block of one row, in the padded range of the scale tiles.
template <typename T, int kFormat>
__global__ void __launch_bounds__(kThreads) k_micro_quantize(QuantArgs a) {
  constexpr int n = micro_block(kFormat);
  const int32_t tiles = micro_tiles(a.K, kFormat);
  const int64_t rows = (a.R + 127) / 128 * 128, total = rows * tiles * 4;
  const int64_t row_bytes = micro_row_bytes(a.K);
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    const int64_t r = i / (tiles * 4);
    const int32_t j = (int32_t)(i - r * (tiles * 4));
    uint32_t byte = 0;
    if (r < a.R && (int64_t)j * (n / 2) < row_bytes) {
      const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
      float v[n], amax = 0.f;
      bool nan = false;
#pragma unroll
      for (int e = 0; e < n; ++e) {
        const int32_t k = j * n + e;
        v[e] = k < a.K ? Elem<T>::get(x[k]) : 0.f;
        amax = fmaxf(amax, fabsf(v[e]));
        nan |= isnan(v[e]);
      }
      float f;
      byte = micro_scale<kFormat>(nan ? NAN : amax, a.g, &f);
      const bool bad = nan || isinf(amax);
#pragma unroll
      for (int e = 0; e < n; e += 2)
        a.codes[r * row_bytes + (j * n + e) / 2] = bad ? 0 : (uint8_t)e2m1x2(v[e] * f, v[e + 1] * f);
    }
    a.scales[micro_scale_at(r, j, tiles)] = (uint8_t)byte;
  }
}

struct LookupArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t R;
  int32_t K;
  float g;
  const int64_t* ids;
  int64_t n;
  void* out;
  int64_t out_stride;
  uint32_t* status;
};

template <typename T, int kFormat>
__global__ void __launch_bounds__(kThreads) k_micro_lookup(LookupArgs a) {
  constexpr int n = micro_block(kFormat);
  const int32_t tiles = micro_tiles(a.K, kFormat);
  const int64_t row_bytes = micro_row_bytes(a.K);
  const int32_t pairs = (a.K + 1) / 2;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < a.n * pairs; i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = i / pairs;
    const int32_t k = (int32_t)(i - row * pairs) * 2;
    const int64_t r = a.ids ? a.ids[row] : row;
    float2 v = make_float2(0.f, 0.f);
    if (r < 0 || r >= a.R) {
      report(a.status, kErrIndex);
    } else {
      v = e2m1x2_values(a.codes[r * row_bytes + k / 2]);
      const float s = micro_scale_value<kFormat>(a.scales[micro_scale_at(r, k / n, tiles)]);
      v.x = kFormat == kMicroMX ? v.x * s : __fmul_rn(v.x * s, a.g);
      v.y = kFormat == kMicroMX ? v.y * s : __fmul_rn(v.y * s, a.g);
    }
    T* out = static_cast<T*>(a.out) + row * a.out_stride + k;
    out[0] = Elem<T>::put(v.x);
    if (k + 1 < a.K) out[1] = Elem<T>::put(v.y);
  }
}

template <int kFormat>
const void* quantize_of(int dtype) {
  switch (dtype) {
    case EMB_F32: return reinterpret_cast<const void*>(&k_micro_quantize<float, kFormat>);
    case EMB_F16: return reinterpret_cast<const void*>(&k_micro_quantize<__half, kFormat>);
    default: return reinterpret_cast<const void*>(&k_micro_quantize<__nv_bfloat16, kFormat>);
  }
}

template <int kFormat>
const void* lookup_of(int dtype) {
  switch (dtype) {
    case EMB_F32: return reinterpret_cast<const void*>(&k_micro_lookup<float, kFormat>);
    case EMB_F16: return reinterpret_cast<const void*>(&k_micro_lookup<__half, kFormat>);
    default: return reinterpret_cast<const void*>(&k_micro_lookup<__nv_bfloat16, kFormat>);
  }
}

unsigned grid_for(int64_t items) {
  const int64_t blocks = (items + kThreads - 1) / kThreads;
  return (unsigned)(blocks < 152 * 8 ? blocks : 152 * 8);
}

}  // namespace
}  // namespace embbwd

using namespace embbwd;

extern "C" emb_status emb_micro_quantize(int device, const void* x, emb_dtype x_dtype, int64_t x_stride, int64_t R,
                                         int32_t K, emb_micro_format format, float tensor_scale, uint8_t* codes,
                                         uint8_t* scales, void* stream) {
  if (device < 0 || R < 0 || R > kMaxMicroRows || K < 1 || K > kMaxMicroCols) return EMB_ERR_INVALID_ARG;
  if (!dtype_ok(x_dtype) || !micro_format_ok(format)) return EMB_ERR_INVALID_ARG;
  if (!micro_tensor_scale_ok(format, tensor_scale)) return EMB_ERR_INVALID_ARG;
  if (R == 0) return EMB_OK;
  if (!x || !codes || !scales || !aligned(x, dtype_size(x_dtype)) || !aligned(codes, 16) || !aligned(scales, 16) ||
      (R > 1 && x_stride < K))
    return EMB_ERR_INVALID_ARG;
  QuantArgs a{x, x_stride, R, K, tensor_scale, codes, scales};
  return on_device(device, [&] {
    void* args[] = {&a};
    const void* fn = format == EMB_MICRO_MX ? quantize_of<kMicroMX>(x_dtype) : quantize_of<kMicroNV>(x_dtype);
    const int64_t items = (R + 127) / 128 * 128 * micro_tiles(K, format) * 4;
    return launch_kernel(fn, dim3(grid_for(items)), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), args, false);
  });
}

extern "C" emb_status emb_micro_lookup(int device, const uint8_t* codes, const uint8_t* scales, int64_t R, int32_t K,
                                       emb_micro_format format, float tensor_scale, const int64_t* ids, int64_t n,
                                       void* out, emb_dtype out_dtype, int64_t out_stride, uint32_t* device_status,
                                       void* stream) {
  if (device < 0 || R < 0 || R > kMaxMicroRows || K < 1 || K > kMaxMicroCols || n < 0 || n > kMaxMicroRows)
    return EMB_ERR_INVALID_ARG;
  if (!dtype_ok(out_dtype) || !micro_format_ok(format)) return EMB_ERR_INVALID_ARG;
  if (!micro_tensor_scale_ok(format, tensor_scale) || (!ids && n > R)) return EMB_ERR_INVALID_ARG;
  if (n == 0) return EMB_OK;
  if (!out || !aligned(out, dtype_size(out_dtype)) || (n > 1 && out_stride < K)) return EMB_ERR_INVALID_ARG;
  if (!codes || !scales || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(ids, 8) || !aligned(device_status, 4))
    return EMB_ERR_INVALID_ARG;
  LookupArgs a{codes, scales, R, K, tensor_scale, ids, n, out, out_stride, device_status};
  return on_device(device, [&] {
    void* args[] = {&a};
    const void* fn = format == EMB_MICRO_MX ? lookup_of<kMicroMX>(out_dtype) : lookup_of<kMicroNV>(out_dtype);
    return launch_kernel(fn, dim3(grid_for(n * ((K + 1) / 2))), dim3(kThreads), 0, static_cast<cudaStream_t>(stream),
                         args, false);
  });
}
