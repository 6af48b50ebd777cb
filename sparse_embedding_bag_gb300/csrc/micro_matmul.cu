// Product of two microscaled 4-bit matrices: out[m, n] = sum_k X[m, k] W[n, k].
// Products of two codes and two block scales are exact in fp32; sums are held in
// fp32 and rounded once to the output's type.
#include <cmath>

#include "micro.cuh"

namespace embbwd {
namespace {

constexpr int kTile = 64, kDepth = 32;

struct MatmulArgs {
  const uint8_t *x, *xs, *w, *ws;
  int32_t M, N, K;
  float alpha;
  void* out;
  int64_t out_stride;
};

// A block takes a 64 x 64 tile of the output, 4 x 4 values a thread; both operands
// are widened to fp32 in shared memory, 32 elements deep.
template <typename T, int kFormat>
__global__ void __launch_bounds__(256) k_micro_matmul(MatmulArgs a) {
  __shared__ float sx[kDepth][kTile + 1], sw[kDepth][kTile + 1];
  const int32_t m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile;
  const int64_t row_bytes = micro_row_bytes(a.K);
  const int32_t tiles = micro_tiles(a.K, kFormat);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int32_t k0 = 0; k0 < a.K; k0 += kDepth) {
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * kDepth / 2; i += 256) {
      const int r = i / (kDepth / 2), k = (i % (kDepth / 2)) * 2;
      float2 vx = make_float2(0.f, 0.f), vw = vx;
      const int32_t j = (k0 + k) / micro_block(kFormat);
      if (m0 + r < a.M) {
        vx = e2m1x2_values(a.x[(m0 + r) * row_bytes + (k0 + k) / 2]);
        const float s = micro_scale_value<kFormat>(a.xs[micro_scale_at(m0 + r, j, tiles)]);
        vx.x *= s, vx.y *= s;
      }
      if (n0 + r < a.N) {
        vw = e2m1x2_values(a.w[(n0 + r) * row_bytes + (k0 + k) / 2]);
        const float s = micro_scale_value<kFormat>(a.ws[micro_scale_at(n0 + r, j, tiles)]);
        vw.x *= s, vw.y *= s;
      }
      sx[k][r] = vx.x, sx[k + 1][r] = vx.y;
      sw[k][r] = vw.x, sw[k + 1][r] = vw.y;
    }
    __syncthreads();
#pragma unroll 4
    for (int k = 0; k < kDepth; ++k) {
      float u[4], v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = sx[k][ty * 4 + i], v[i] = sw[k][tx + 16 * i];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(u[i], v[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int32_t m = m0 + ty * 4 + i, n = n0 + tx + 16 * j;
      if (m < a.M && n < a.N) static_cast<T*>(a.out)[m * a.out_stride + n] = Elem<T>::put(acc[i][j] * a.alpha);
    }
}

template <int kFormat>
const void* matmul_of(int dtype) {
  switch (dtype) {
    case EMB_F32: return reinterpret_cast<const void*>(&k_micro_matmul<float, kFormat>);
    case EMB_F16: return reinterpret_cast<const void*>(&k_micro_matmul<__half, kFormat>);
    default: return reinterpret_cast<const void*>(&k_micro_matmul<__nv_bfloat16, kFormat>);
  }
}

}  // namespace
}  // namespace embbwd

using namespace embbwd;

extern "C" emb_status emb_micro_matmul(int device, const uint8_t* x_codes, const uint8_t* x_scales, float x_tensor_scale,
                                       int32_t M, const uint8_t* w_codes, const uint8_t* w_scales,
                                       float w_tensor_scale, int32_t N, int32_t K, emb_micro_format format, void* out,
                                       emb_dtype out_dtype, int64_t out_stride, uint32_t* device_status,
                                       void* stream) {
  if (device < 0 || M < 0 || N < 0 || M > kMaxMatmulRows || N > kMaxMatmulRows || K < 1 || K > kMaxMicroCols)
    return EMB_ERR_INVALID_ARG;
  if (!dtype_ok(out_dtype) || !micro_format_ok(format)) return EMB_ERR_INVALID_ARG;
  if (!micro_tensor_scale_ok(format, x_tensor_scale) || !micro_tensor_scale_ok(format, w_tensor_scale))
    return EMB_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return EMB_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales || !out || !aligned(x_codes, 16) || !aligned(x_scales, 16) ||
      !aligned(w_codes, 16) || !aligned(w_scales, 16) || !aligned(out, dtype_size(out_dtype)) ||
      !aligned(device_status, 4) || (M > 1 && out_stride < N))
    return EMB_ERR_INVALID_ARG;
  MatmulArgs a{x_codes, x_scales, w_codes, w_scales, M, N, K, x_tensor_scale * w_tensor_scale, out, out_stride};
  return on_device(device, [&] {
    void* args[] = {&a};
    const void* fn = format == EMB_MICRO_MX ? matmul_of<kMicroMX>(out_dtype) : matmul_of<kMicroNV>(out_dtype);
    return launch_kernel(fn, dim3((N + kTile - 1) / kTile, (M + kTile - 1) / kTile), dim3(256), 0,
                         static_cast<cudaStream_t>(stream), args, false);
  });
}
