// Rows to microscaled 4-bit floating point, and back by row id.
//
// Both are bound by HBM traffic. A thread takes units of 8 elements, so that a warp's codes
// are whole 128-byte lines and its 16-bit values whole 512-byte ones; a team of lanes (a
// warp, or less for short rows) takes a piece of a row, kBatch loads of each lane in flight.
// Measured at 128256 x 4096 (HBM bytes over time): bf16 to MX 219 us, 6.1 TB/s, to NV 272 us,
// 4.9 TB/s (every lane of a block finds its scale: a division, two conversions and a
// reciprocal for 8 elements, where MX has a shift); fp32 to MX 326 us, 7.3 TB/s; MX or NV to
// bf16 208 us, 6.4 TB/s, to fp32 425 us, 5.6 TB/s. By id, to bf16: 1 row 2.2 us, 4096 random
// ones 9.8 us (NV 10.3), 65536 121 us. A row's scales lie 512 bytes apart, as the product wants
// them, so that 4096 random rows read 18.8 MB (MX) or 29.4 MB (NV) from HBM for 8.9 or 9.4 MB
// of codes and scales.
// 16-bit types are nearly bound by instructions (the conversions run at a quarter of the
// rate): checking every unit's place in its row took 10 % more.
#include <cmath>

#include "micro.cuh"
#include "sm103.cuh"

namespace embbwd {
namespace {

constexpr int kBatch = 4;  // units a thread of the quantisation has in flight

struct QuantArgs {
  const void* x;
  int64_t x_stride;
  int64_t R;
  int32_t K;
  float g;
  uint8_t* codes;
  uint8_t* scales;
};

// Eight floats to eight codes.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[kGroup]) {
  uint32_t r;
  asm("{ .reg .b8 a, b, c, d;\n"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      "mov.b32 %0, {a, b, c, d}; }"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// Rows and blocks are taken up to whole scale tiles, whose padding is zero. 16-bit rows that
// do not start at 16 bytes are read by words (128256 x 4096 bf16 to MX: 297 us against 219;
// element by element 454, shifting aligned 16-byte pieces 555), fp32 ones by elements.
template <typename T, int kFormat>
__global__ void __launch_bounds__(kThreads) k_micro_quantize(QuantArgs a, int log_team) {
  constexpr int n = micro_block(kFormat), lanes = n / kGroup;  // lanes of a block
  pdl_wait();
  pdl_trigger();
  const int32_t tiles = micro_tiles(a.K, kFormat), units = tiles * 4 * lanes;
  const int64_t row_bytes = micro_row_bytes(a.K);
  const int32_t team = 1 << log_team, lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * (kThreads >> log_team) + (threadIdx.x >> log_team);
  const int32_t u0 = (int32_t)blockIdx.y * kBatch * team + (threadIdx.x & (team - 1));
  const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
  const bool row = r < a.R, wide = row && reinterpret_cast<uintptr_t>(x) % 16 == 0;
  // Are all of this team's units whole and loaded 16 bytes at a time? Then nothing is checked.
  const bool plain = wide && ((int32_t)blockIdx.y + 1) * kBatch * team * kGroup <= a.K;
  // Units of 16-bit rows elsewhere come in the four or (rows at odd elements) five words that
  // cover them, where these lie in the row.
  const int32_t odd = sizeof(T) == 2 ? (int32_t)(reinterpret_cast<uintptr_t>(x) / 2 % 2) : 0;
  auto in_words = [&](int32_t k) { return sizeof(T) == 2 && row && !wide && k >= odd && k + kGroup + odd <= a.K; };
  Raw8<T> raw[kBatch];
  uint32_t fifth[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int32_t k = (u0 + b * team) * kGroup;
    if (plain || (wide && k + kGroup <= a.K)) {
      raw[b].load(x + k);
    } else if (in_words(k)) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(x + k - odd);
      raw[b].u[0] = make_uint4(w[0], w[1], w[2], w[3]);
      fifth[b] = odd ? w[4] : 0;
    }
  }
  uint8_t* codes = a.codes + r * row_bytes + u0 * 4;
  uint8_t* word_at = a.scales + micro_scale_at(r, u0 / lanes, tiles);
  const bool writes_word = lane % (4 * lanes) == 0 && r < (a.R + 127) / 128 * 128;
  auto unit = [&](int b, bool checked) {
    const int32_t u = u0 + b * team, k = u * kGroup;
    float v[kGroup];
    if (!checked || (wide && k + kGroup <= a.K)) {
      raw[b].widen(v);
    } else if (in_words(k)) {
      uint4& w = raw[b].u[0];
      if (odd)
        w = make_uint4(__funnelshift_r(w.x, w.y, 16), __funnelshift_r(w.y, w.z, 16), __funnelshift_r(w.z, w.w, 16),
                       __funnelshift_r(w.w, fifth[b], 16));
      raw[b].widen(v);
    } else {
#pragma unroll
      for (int i = 0; i < kGroup; ++i) v[i] = row && k + i < a.K ? Elem<T>::get(x[k + i]) : 0.f;
    }
    // the largest magnitude by its bits: infinity is above all numbers, NaN above infinity
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) most = max(most, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < lanes; o *= 2) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    float f;
    const uint32_t byte = micro_scale<kFormat>(__uint_as_float(most), a.g, &f);
    const F2 f2 = F2::of(f, f);
#pragma unroll
    for (int i = 0; i < kGroup; i += 2) {
      const float2 y = (F2::of(v[i], v[i + 1]) * f2).get();
      v[i] = y.x, v[i + 1] = y.y;
    }
    const uint32_t eight = most >= 0x7f800000u ? 0u : e2m1x8(v);
    if (!checked || (row && (int64_t)u * 4 < row_bytes)) *reinterpret_cast<uint32_t*>(codes + b * team * 4) = eight;
    // four blocks' bytes make one word of the scale tile
    uint32_t word = byte << ((lane / lanes & 3) * 8);
    word |= __shfl_xor_sync(0xffffffffu, word, lanes);
    word |= __shfl_xor_sync(0xffffffffu, word, 2 * lanes);
    if (writes_word && (!checked || u < units))
      *reinterpret_cast<uint32_t*>(word_at + b * team / (4 * lanes) * 512) = word;
  };
  if (__all_sync(0xffffffffu, plain)) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) unit(b, false);
  } else {
    for (int b = 0; b < kBatch; ++b) {
      if (b > 0 && ((int32_t)blockIdx.y * kBatch + b) * team >= units) break;  // the same for the whole block
      unit(b, true);
    }
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

template <int kFormat>
__device__ __forceinline__ float micro_value(float v, float s, float g) {
  return kFormat == kMicroMX ? v * s : __fmul_rn(v * s, g);
}

// Units a thread has in flight: what it loads is small, so that 16-bit outputs want many
// (128256 x 4096 MX to bf16, before the units were cheaper: 253 us with 8, 272 with 4, 321
// with 2); fp32 stores fill the queues by themselves (now 425 us with 1, 438 with 2, 460 with 4).
template <typename T>
struct LookupBatch {
  static constexpr int value = sizeof(T) == 2 ? 8 : 1;
};

// Units start at the row's first 16-byte boundary of the output: stores are whole, and the
// codes of a unit come from two words and two blocks where that is no multiple of 8.
template <typename T, int kFormat>
__global__ void __launch_bounds__(kThreads) k_micro_lookup(LookupArgs a, int log_team) {
  constexpr int n = micro_block(kFormat), out_n = 16 / sizeof(T), kBatch = LookupBatch<T>::value;
  pdl_wait();
  pdl_trigger();
  const int32_t team = 1 << log_team;
  const int64_t row = (int64_t)blockIdx.x * (kThreads >> log_team) + (threadIdx.x >> log_team);
  if (row >= a.n) return;
  const int64_t r = a.ids ? a.ids[row] : row;
  const bool ok = r >= 0 && r < a.R;
  const int32_t tiles = micro_tiles(a.K, kFormat), first = threadIdx.x & (team - 1);
  if (!ok && first == 0 && blockIdx.y == 0) report(a.status, kErrIndex);
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(a.codes + r * micro_row_bytes(a.K));
  const uint8_t* scales = a.scales + micro_scale_at(r, 0, tiles);
  auto scale_byte = [&](int32_t j) { return (uint32_t)__ldg(scales + (j >> 2) * 512 + (j & 3)); };
  T* out = static_cast<T*>(a.out) + row * a.out_stride;
  const int32_t head = min(a.K, (int32_t)(-(reinterpret_cast<uintptr_t>(out) / sizeof(T)) % out_n));
  const int32_t units = (a.K - head) / kGroup;
  const int32_t u0 = (int32_t)blockIdx.y * kBatch * team + first;
  uint32_t word[kBatch], next[kBatch], byte[kBatch], byte2[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int32_t u = u0 + b * team, k = head + u * kGroup;
    word[b] = next[b] = byte[b] = byte2[b] = 0;
    if (!ok || u >= units) continue;
    word[b] = __ldg(codes + k / 8);
    byte[b] = scale_byte(k / n);
    if (head) next[b] = __ldg(codes + (k + 7) / 8), byte2[b] = scale_byte((k + 7) / n);
  }
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int32_t u = u0 + b * team, k = head + u * kGroup;
    if (u >= units) break;
    const float s = micro_scale_value<kFormat>(byte[b]);
    float x[kGroup];
    if (head == 0) {
      const F2 s2 = F2::of(s, s), g2 = F2::of(a.g, a.g);
#pragma unroll
      for (int i = 0; i < kGroup; i += 2) {
        const float2 v = e2m1x2_values(word[b] >> 4 * i & 0xffu);
        F2 y = F2::of(v.x, v.y) * s2;
        if (kFormat == kMicroNV) y = y * g2;
        x[i] = y.get().x, x[i + 1] = y.get().y;
      }
    } else {
      const uint32_t w = __funnelshift_r(word[b], next[b], head * 4);
      const float s2 = micro_scale_value<kFormat>(byte2[b]);
      const int32_t same = n - k % n;  // elements of the unit in its first block
#pragma unroll
      for (int i = 0; i < kGroup; i += 2) {
        const float2 v = e2m1x2_values(w >> 4 * i & 0xffu);
        x[i] = micro_value<kFormat>(v.x, i < same ? s : s2, a.g);
        x[i + 1] = micro_value<kFormat>(v.y, i + 1 < same ? s : s2, a.g);
      }
    }
    store8(out + k, x);
  }
  if (blockIdx.y == 0)
    for (int32_t o = first; o < a.K - units * kGroup; o += team) {
      const int32_t k = o < head ? o : o + units * kGroup;
      float v = 0.f;
      if (ok) {
        const float2 pair = e2m1x2_values(codes[k / 8] >> (k & 6) * 4 & 0xffu);
        v = micro_value<kFormat>(k & 1 ? pair.y : pair.x, micro_scale_value<kFormat>(scale_byte(k / n)), a.g);
      }
      out[k] = Elem<T>::put(v);
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

// Teams of the smallest power of two that holds a row's units, up to a warp, and at least
// the lanes that make up a word of scales; blocks along y take pieces of a row.
cudaError_t launch_teams(const void* fn, int64_t rows, int32_t units, int log_least, int batch, cudaStream_t s,
                         void** args, int* log_team) {
  *log_team = log_least;
  while (*log_team < 5 && (1 << *log_team) < units) ++*log_team;
  const int64_t per_block = kThreads >> *log_team;
  const int32_t piece = batch << *log_team;
  return launch_kernel(fn, dim3((unsigned)((rows + per_block - 1) / per_block), (units + piece - 1) / piece),
                       dim3(kThreads), 0, s, args, true);
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
    int log_team;
    void* args[] = {&a, &log_team};
    const bool mx = format == EMB_MICRO_MX;
    return launch_teams(mx ? quantize_of<kMicroMX>(x_dtype) : quantize_of<kMicroNV>(x_dtype), (R + 127) / 128 * 128,
                        micro_tiles(K, format) * 4 * micro_block(format) / kGroup, mx ? 4 : 3, kBatch,
                        static_cast<cudaStream_t>(stream), args, &log_team);
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
    int log_team;
    void* args[] = {&a, &log_team};
    return launch_teams(format == EMB_MICRO_MX ? lookup_of<kMicroMX>(out_dtype) : lookup_of<kMicroNV>(out_dtype), n,
                        (K + kGroup - 1) / kGroup, 0, out_dtype == EMB_F32 ? LookupBatch<float>::value : LookupBatch<__half>::value,
                        static_cast<cudaStream_t>(stream), args, &log_team);
  });
}
