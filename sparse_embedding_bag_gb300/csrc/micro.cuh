// Microscaled 4-bit floating point (E2M1 elements) as the library stores it.
//
//   format 0 (MX): 32 elements share a power of two, an E8M0 byte b = 2^(b - 127);
//                  255 stands for NaN. As the OCP Microscaling Formats specification
//                  (v1.0, section 6.3) puts it: exponent = floor(log2(amax)) - 2.
//   format 1 (NV): 16 elements share an E4M3 scale, and the tensor an fp32 scale g:
//                  scale = E4M3(amax / (6 g)).
//
// Codes: row r at codes + r * 16 * ceil(K / 32) bytes, element k in the low (k even)
// or high (k odd) half of byte k / 2; the row is padded with zeros to a multiple of
// 32 elements. Scales: tiles of 128 rows x 4 blocks of 512 bytes, one after the other
// along the row, then down the rows; block j of row r in tile (r / 128, j / 4) at byte
// (r % 32) * 16 + (r % 128 / 32) * 4 + j % 4. It is the order in which the tensor
// core's scale memory holds them, so that a tile is one copy. Padding is zero.
#pragma once

#include <cuda_fp8.h>

#include "vocab.cuh"

namespace embbwd {

constexpr int kMicroMX = 0, kMicroNV = 1;

constexpr int64_t kMaxMicroRows = (int64_t)1 << 31;
constexpr int32_t kMaxMicroCols = 1 << 20;
constexpr int32_t kMaxMatmulRows = 1 << 21;

inline bool micro_format_ok(int f) { return f == kMicroMX || f == kMicroNV; }
// MX has no tensor scale; NV takes one whose product with any block scale is normal.
inline bool micro_tensor_scale_ok(int f, float g) {
  return f == kMicroMX ? g == 1.f : (g >= 1e-15f && g <= 1e15f);
}
__host__ __device__ constexpr int micro_block(int format) { return format == kMicroMX ? 32 : 16; }
__host__ __device__ inline int64_t micro_row_bytes(int32_t K) { return (int64_t)((K + 31) / 32) * 16; }
// Scale tiles along a row.
__host__ __device__ inline int32_t micro_tiles(int32_t K, int format) {
  const int32_t blocks = (K + 31) / 32 * (32 / micro_block(format));
  return (blocks + 3) / 4;
}
__host__ __device__ inline int64_t micro_scale_at(int64_t r, int32_t j, int32_t tiles) {
  return ((r >> 7) * tiles + (j >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (j & 3);
}

// Two codes (bits 0-7) to their values.
__device__ __forceinline__ float2 e2m1x2_values(uint32_t codes) {
  uint32_t h;
  asm("{ .reg .b8 t; cvt.u8.u32 t, %1; cvt.rn.f16x2.e2m1x2 %0, t; }" : "=r"(h) : "r"(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// The value of a scale byte (without the tensor's scale).
template <int kFormat>
__device__ __forceinline__ float micro_scale_value(uint32_t byte) {
  if (kFormat == kMicroMX) {
    if (byte == 255) return NAN;
    return __uint_as_float(byte ? byte << 23 : 1u << 22);  // 2^-127 is subnormal
  }
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

// The scale of a block with largest magnitude amax: its byte, and the factor that
// takes the elements to code units (0 where no finite factor exists).
template <int kFormat>
__device__ __forceinline__ uint32_t micro_scale(float amax, float g, float* factor) {
  *factor = 0.f;
  if (kFormat == kMicroMX) {
    if (!(amax <= 3.402823466e38f)) return 255;  // infinities and NaN
    const int e = max((int)(__float_as_uint(amax) >> 23) - 129, -127);
    *factor = __uint_as_float((uint32_t)(127 - e) << 23);
    return (uint32_t)(e + 127);
  }
  if (!(amax <= 3.402823466e38f)) return 0x7f;
  const float t = __fdiv_rn(amax, __fmul_rn(6.f, g));
  const uint32_t byte = __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
  const float d = __fmul_rn(micro_scale_value<kFormat>(byte), g);
  if (d >= 1.175494351e-38f) *factor = __frcp_rn(d);
  return byte;
}

}  // namespace embbwd
