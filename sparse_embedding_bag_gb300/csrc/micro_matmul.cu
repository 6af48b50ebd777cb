// Product of two microscaled 4-bit matrices on the tensor cores:
// out[m, n] = sum_k X[m, k] W[n, k], X the rows of M tokens, W a table of N rows.
//
// The table is the MMA's A operand (128 rows a tile, the lanes of tensor memory) and the
// tokens its B operand (kTok columns), so that one token costs no more than a narrow
// tile. Codes reach shared memory by TMA in stages 256 elements deep (128 bytes a row,
// 128-byte swizzle), block scales as they are stored: their 512-byte tiles are what the
// MMA reads from tensor memory. Elements times block scales are multiplied and summed
// by the block-scaled MMA in fp32 in tensor memory; the tensor scales are applied
// to the sum, which is rounded once. Sums run over k in order: results do not depend on
// the launch.
//
// A persistent CTA an SM: warp 4 issues copies, warp 5 copies scales and issues MMAs,
// warps 0-3 move finished tiles from tensor memory to the output while the next is
// computed. Tensor memory holds two accumulators of kTok columns and one stage's
// scales in 512 columns. Where two accumulators do not fit beside the scales they
// overlap in some columns, which the epilogue empties first.
#include <cmath>

#include "micro.cuh"
#include "sm103.cuh"

namespace embbwd {
namespace {

constexpr int kRows = 128;       // table rows of a tile
constexpr int kDepth = 256;      // elements of a stage
constexpr int kStep = 64;        // elements of an MMA
constexpr uint32_t kTmemCols = 512;
constexpr int kMatmulThreads = 192;
constexpr uint32_t kSmemMost = 226 * 1024;

struct MatmulArgs {
  const uint8_t *xs, *ws;
  int32_t M, N, K;
  float alpha;
  void* out;
  int64_t out_stride;
  uint32_t* status;
};

template <int kFormat, int kTok>
struct Shape {
  static constexpr uint32_t kTiles = kDepth / (4 * micro_block(kFormat));  // scale tiles of a stage, along k
  static constexpr uint32_t kTokTiles = (kTok + 127) / 128;                // and across the tokens
  static constexpr uint32_t kA = kRows * 128, kB = kTok * 128;
  static constexpr uint32_t kSA = kTiles * 512, kSB = kTokTiles * kTiles * 512;
  static constexpr uint32_t kStage = kA + kB + kSA + kSB;
  static constexpr uint32_t kStageAligned = (kStage + 1023) / 1024 * 1024;  // the swizzle repeats every 1024 bytes
  static constexpr uint32_t kStages = (kSmemMost - 2048) / kStageAligned < 12 ? (kSmemMost - 2048) / kStageAligned : 12;
  static constexpr uint32_t kSmem = kStages * kStageAligned + 2048;
  static constexpr uint32_t kSfCols = kTiles * 4 * (1 + kTokTiles);
  static constexpr uint32_t kSf = kTmemCols - kSfCols;  // a stage's scales: the table's, then the tokens'
  // The second accumulator, and how many columns it shares with the first.
  static constexpr uint32_t kAcc1 = 2 * kTok <= kSf ? kTok : kSf - kTok;
  static constexpr uint32_t kShared = kTok - kAcc1;
  static_assert(kShared % 8 == 0 && kStages >= 2, "");
};

struct Control {
  uint64_t full[12], empty[12], acc_full[2], acc_empty[2], done;
  uint32_t tmem;
  int abort;
};

// The columns [c0, c1) of one accumulator to the output: this thread's row n of the
// table, one token a column.
template <typename T>
__device__ __forceinline__ void store_columns(const MatmulArgs& a, uint32_t tmem, int32_t n, int32_t m0, uint32_t c0,
                                              uint32_t c1) {
  for (uint32_t c = c0; c < c1 && m0 + (int32_t)c < a.M; c += 16) {
    float v[16];
    tmem_load16(tmem + c, v);
    tmem_load_wait();
    T* out = static_cast<T*>(a.out) + (int64_t)(m0 + c) * a.out_stride + n;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (c + i < c1 && m0 + (int32_t)c + i < a.M && n < a.N) out[i * a.out_stride] = Elem<T>::put(v[i] * a.alpha);
  }
}

template <typename T, int kFormat, int kTok>
__global__ void __launch_bounds__(kMatmulThreads, 1)
    k_micro_matmul(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, MatmulArgs a) {
  using S = Shape<kFormat, kTok>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Control ctl;
  const uint32_t stages = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int* abort = &ctl.abort;
  const int32_t w_tiles = (a.N + kRows - 1) / kRows, x_tiles = (a.M + kTok - 1) / kTok;
  const int64_t tiles = (int64_t)w_tiles * x_tiles;
  const int32_t k_stages = (a.K + kDepth - 1) / kDepth;
  const int32_t sf_tiles = micro_tiles(a.K, kFormat);

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S::kStages; ++s) mbar_init(smem_u32(&ctl.full[s]), 1), mbar_init(smem_u32(&ctl.empty[s]), 1);
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&ctl.acc_full[i]), 1), mbar_init(smem_u32(&ctl.acc_empty[i]), 4);
    mbar_init(smem_u32(&ctl.done), 1);
    ctl.abort = 0;
    mbar_init_fence();
  }
  if (warp == 5) tmem_alloc(smem_u32(&ctl.tmem), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem, 0);

  if (warp == 4 && lane == 0) {
    uint32_t s = 0, round = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const int32_t wt = (int32_t)(t / x_tiles), xt = (int32_t)(t - (int64_t)wt * x_tiles);
      const uint32_t tok_tiles = min((int32_t)S::kTokTiles, (a.M + 127) / 128 - xt * (int32_t)S::kTokTiles);
      for (int32_t k = 0; k < k_stages; ++k) {
        if (round && !mbar_wait(smem_u32(&ctl.empty[s]), (round - 1) & 1, abort)) {
          ok = false;
          break;
        }
        const uint32_t base = stages + s * S::kStageAligned, bar = smem_u32(&ctl.full[s]);
        const uint32_t sf = min((int32_t)S::kTiles, sf_tiles - k * (int32_t)S::kTiles) * 512;
        mbar_expect(bar, S::kA + S::kB + sf * (1 + tok_tiles));
        tensor_load(base, &wmap, k * 128, wt * kRows, bar);
        tensor_load(base + S::kA, &xmap, k * 128, xt * kTok, bar);
        const int64_t sf_at = (int64_t)k * S::kTiles;
        bulk_load(base + S::kA + S::kB, a.ws + ((int64_t)wt * sf_tiles + sf_at) * 512, sf, bar);
        for (uint32_t i = 0; i < tok_tiles; ++i)
          bulk_load(base + S::kA + S::kB + S::kSA + i * S::kTiles * 512,
                    a.xs + (((int64_t)xt * kTok / 128 + i) * sf_tiles + sf_at) * 512, sf, bar);
        if (++s == S::kStages) s = 0, ++round;
      }
    }
    // Copies of an abandoned tile are still in flight: wait for each issued stage.
    if (!ok) {
      for (uint32_t i = 0; i < S::kStages; ++i) {
        const uint32_t issued = round + (i < s);  // rounds issued into stage i
        const uint64_t t0 = global_ns();
        while (issued && !mbar_try(smem_u32(&ctl.full[i]), (issued - 1) & 1) && global_ns() - t0 < kWaitNs) {
        }
      }
    }
  } else if (warp == 5) {
    // A : table codes, B : token codes, both E2M1, fp32 sums (bits 7, 10); N / 8 (17); E8M0 scales (23); M / 128 (27)
    constexpr uint32_t idesc0 = 1u << 7 | 1u << 10 | (uint32_t)(kTok / 8) << 17 |
                                (kFormat == kMicroMX ? 1u << 23 : 0u) | (uint32_t)(kRows / 128) << 27;
    // The whole warp walks the stages, so that addresses and descriptors stay in uniform
    // registers; one lane issues. This warp paces the kernel: a stage is unrolled, with
    // constant offsets.
    const bool leader = elect_one();
    const uint32_t full0 = smem_u32(&ctl.full[0]), empty0 = smem_u32(&ctl.empty[0]);
    const uint32_t sfa = tmem + S::kSf, sfb = sfa + S::kTiles * 4;
    constexpr uint32_t kBlock = S::kStageAligned >> 4;  // of a stage, in a descriptor's units
    const uint64_t a_desc0 = operand_desc(stages), sf_desc0 = scales_desc(stages + S::kA + S::kB);
    uint32_t s = 0, parity = 0, j = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++j) {
      constexpr uint32_t lag = S::kShared ? 1 : 2;  // the tile whose columns this one takes over
      if (j >= lag && !mbar_wait(smem_u32(&ctl.acc_empty[(j - lag) & 1]), ((j - lag) >> 1) & 1, abort)) break;
      const uint32_t d = tmem + ((j & 1) ? S::kAcc1 : 0);
      for (int32_t k = 0; k < k_stages; ++k) {
        if (!mbar_wait(full0 + s * 8, parity, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t a_desc = a_desc0 + s * kBlock, b_desc = a_desc + (S::kA >> 4), sf_desc = sf_desc0 + s * kBlock;
        const int32_t used = sf_tiles - k * (int32_t)S::kTiles, steps = (a.K - k * kDepth + kStep - 1) / kStep;
        if (leader) {
#pragma unroll
          for (int i = 0; i < (int)S::kTiles; ++i) {
            if (i >= used) break;
            tc_copy_scales(sfa + i * 4, sf_desc + i * 32);
#pragma unroll
            for (uint32_t q = 0; q < S::kTokTiles; ++q)
              tc_copy_scales(sfb + (i * S::kTokTiles + q) * 4, sf_desc + (S::kSA >> 4) + (q * S::kTiles + i) * 32);
          }
#pragma unroll
          for (int e = 0; e < kDepth / kStep; ++e) {
            if (e >= steps) break;
            // MX: a scale tile serves two steps, its bytes 0-1 and 2-3; NV: a tile a step
            const uint32_t i = kFormat == kMicroMX ? e >> 1 : e;
            const uint32_t id = kFormat == kMicroMX ? (e & 1) * 2 : 0;
            tc_mma_f4<kFormat == kMicroMX>(d, a_desc + e * 2, b_desc + e * 2, idesc0 | id << 29 | id << 4, sfa + i * 4,
                                           sfb + i * S::kTokTiles * 4, e > 0 || k > 0);
          }
          tc_commit(empty0 + s * 8);
          if (k + 1 == k_stages) tc_commit(smem_u32(&ctl.acc_full[j & 1]));
        }
        __syncwarp();
        if (++s == S::kStages) s = 0, parity ^= 1;
      }
    }
    if (leader) tc_commit(smem_u32(&ctl.done));
  } else if (warp < 4) {
    uint32_t j = 0;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, ++j) {
      const int32_t wt = (int32_t)(t / x_tiles), xt = (int32_t)(t - (int64_t)wt * x_tiles);
      const bool ok = mbar_wait(smem_u32(&ctl.acc_full[j & 1]), (j >> 1) & 1, abort);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint32_t d = tmem + ((j & 1) ? S::kAcc1 : 0) + (warp * 32 << 16);
      const int32_t n = wt * kRows + warp * 32 + lane;
      const uint32_t first = (j & 1) ? 0 : kTok - S::kShared;  // the shared columns come first
      store_columns<T>(a, d, n, xt * kTok, first, first + S::kShared);
      if (S::kShared) {
        tc_fence_before();
        if (lane == 0) mbar_arrive(smem_u32(&ctl.acc_empty[j & 1]));
      }
      store_columns<T>(a, d, n, xt * kTok, (j & 1) ? S::kShared : 0, (j & 1) ? kTok : kTok - S::kShared);
      if (!S::kShared) {
        tc_fence_before();
        if (lane == 0) mbar_arrive(smem_u32(&ctl.acc_empty[j & 1]));
      }
    }
  }
  __syncwarp();
  // Nothing may be in flight when the tensor memory goes back.
  if (warp == 5 && lane == 0) {
    const uint64_t t0 = global_ns();
    while (!mbar_try(smem_u32(&ctl.done), 0) && global_ns() - t0 < kWaitNs) {
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && *abort) report(a.status, kErrTimeout);
  if (warp == 5) tmem_dealloc(tmem, kTmemCols);
}

template <typename T, int kFormat, int kTok>
cudaError_t launch(int device, const MatmulArgs& a, const uint8_t* x, const uint8_t* w, cudaStream_t s) {
  using S = Shape<kFormat, kTok>;
  const void* fn = reinterpret_cast<const void*>(&k_micro_matmul<T, kFormat, kTok>);
  static bool ready[64];
  cudaError_t e = allow_smem(fn, S::kSmem, device, ready);
  if (e != cudaSuccess) return e;
  CUtensorMap wmap, xmap;
  e = byte_matrix_map(&wmap, w, a.N, micro_row_bytes(a.K), kRows);
  if (e == cudaSuccess) e = byte_matrix_map(&xmap, x, a.M, micro_row_bytes(a.K), kTok);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)((a.N + kRows - 1) / kRows) * ((a.M + kTok - 1) / kTok);
  const unsigned grid = (unsigned)(tiles < sm_count(device) ? tiles : sm_count(device));
  MatmulArgs args_copy = a;
  void* args[] = {&wmap, &xmap, &args_copy};
  return launch_kernel(fn, dim3(grid), dim3(kMatmulThreads), S::kSmem, s, args, false);
}

template <typename T, int kFormat>
cudaError_t launch_tok(int device, const MatmulArgs& a, const uint8_t* x, const uint8_t* w, cudaStream_t s) {
  // the narrowest tile that holds the tokens
  if (a.M <= 16) return launch<T, kFormat, 16>(device, a, x, w, s);
  if (a.M <= 64) return launch<T, kFormat, 64>(device, a, x, w, s);
  if (a.M <= 128) return launch<T, kFormat, 128>(device, a, x, w, s);
  return launch<T, kFormat, 256>(device, a, x, w, s);
}

template <int kFormat>
cudaError_t launch_type(int device, int dtype, const MatmulArgs& a, const uint8_t* x, const uint8_t* w,
                        cudaStream_t s) {
  switch (dtype) {
    case EMB_F32: return launch_tok<float, kFormat>(device, a, x, w, s);
    case EMB_F16: return launch_tok<__half, kFormat>(device, a, x, w, s);
    default: return launch_tok<__nv_bfloat16, kFormat>(device, a, x, w, s);
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
  const MatmulArgs a{x_scales, w_scales, M, N, K, x_tensor_scale * w_tensor_scale, out, out_stride, device_status};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return on_device(device, [&] {
    return format == EMB_MICRO_MX ? launch_type<kMicroMX>(device, out_dtype, a, x_codes, w_codes, s)
                                  : launch_type<kMicroNV>(device, out_dtype, a, x_codes, w_codes, s);
  });
}
