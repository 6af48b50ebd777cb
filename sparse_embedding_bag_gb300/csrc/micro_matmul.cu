// Product of two microscaled 4-bit matrices on the tensor cores:
// out[m, n] = sum_k X[m, k] W[n, k], X the rows of M tokens, W a table of N rows.
//
// The table is the MMA's A operand (128 rows a CTA, the lanes of tensor memory) and the
// tokens its B operand (kTok columns), so that one token costs no more than a narrow
// tile. Codes reach shared memory by TMA in stages 256 elements deep (128 bytes a row,
// 128-byte swizzle), block scales as they are stored: their 512-byte tiles are what the
// MMA reads from tensor memory. Elements times block scales are multiplied and summed
// by the block-scaled MMA in fp32 in tensor memory; the tensor scales are applied
// to the sum, which is rounded once. Sums run over k in order: results do not depend on
// the launch.
//
// Persistent CTAs, one an SM: warp 4 issues copies, warp 5 copies scales and issues MMAs,
// warps 0-3 move finished tiles from tensor memory to the output while the next is
// computed. Tensor memory holds two accumulators of kTok columns and one stage's
// scales in 512 columns. Where two accumulators do not fit beside the scales they
// overlap in some columns, which the epilogue empties first.
//
// With more than a few tokens, two CTAs work as a pair (kPair): 256 rows of the table
// against kTok tokens, each CTA bringing its own rows and half of the tokens. What bounds
// a large product is the way from L2 to the SMs, not the MMA: at 2048 x 128256 x 4096 (NV)
// single CTAs of 128 x 256 moved 54 KB a stage and took 382 us, pairs 38 KB 375 us; both wait for L2 more than for the MMA (330 us
// with the stores left out). Fetching the table's next rows to L2 a tile ahead cost 25 us.
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
  int32_t M, N, K;
  float alpha;
  void* out;
  int64_t out_stride;
  uint32_t* status;
};

template <int kFormat, int kTok, bool kPair>
struct Shape {
  static constexpr uint32_t kCtas = kPair ? 2 : 1;
  static constexpr uint32_t kTiles = kDepth / (4 * micro_block(kFormat));  // scale tiles of a stage, along k
  static constexpr uint32_t kTokTiles = (kTok + 127) / 128;                // and across the tokens
  static constexpr uint32_t kA = kRows * 128, kB = kTok / kCtas * 128;     // of one CTA
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
  static_assert(kShared % 8 == 0 && kStages >= 2 && kB % 1024 == 0, "");
};

struct Control {
  uint64_t full[12], empty[12], acc_full[2], acc_empty[2], done;
  uint32_t tmem;
  int abort;
};

// The columns [c0, c1) of one accumulator (multiples of 8) to the output: this thread's
// row n of the table, one token a column, a warp's 32 values of a token side by side.
template <typename T>
__device__ __forceinline__ void store_columns(const MatmulArgs& a, uint32_t tmem, int32_t n, int32_t m0, int32_t c0,
                                              int32_t c1) {
  const int32_t end = min(c1, a.M - m0);
  T* out = static_cast<T*>(a.out) + (int64_t)(m0 + c0) * a.out_stride + n;
  const bool mine = n < a.N;
  for (int32_t c = c0; c < end; c += 16) {
    float v[16];
    tmem_load16(tmem + c, v);
    tmem_load_wait();
    if (!mine) continue;
    if (c + 16 <= end) {
#pragma unroll
      for (int i = 0; i < 16; ++i, out += a.out_stride) *out = Elem<T>::put(v[i] * a.alpha);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i, out += a.out_stride)
        if (c + i < end) *out = Elem<T>::put(v[i] * a.alpha);
    }
  }
}

// NaN in place of a tile that was given up.
template <typename T>
__device__ __forceinline__ void store_nan(const MatmulArgs& a, int32_t n, int32_t m0, int32_t cols) {
  if (n >= a.N) return;
  for (int32_t m = m0; m < min(a.M, m0 + cols); ++m)
    static_cast<T*>(a.out)[(int64_t)m * a.out_stride + n] = Elem<T>::put(NAN);
}

template <typename T, int kFormat, int kTok, bool kPair>
__global__ void __launch_bounds__(kMatmulThreads, 1)
    k_micro_matmul(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap wsmap,
                   const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap xsmap, MatmulArgs a) {
  using S = Shape<kFormat, kTok, kPair>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Control ctl;
  const uint32_t stages = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_rank() : 0;  // CTA 0 holds the barriers that both use
  volatile int* abort = &ctl.abort;
  const int32_t w_tiles = (a.N + kRows * S::kCtas - 1) / (kRows * S::kCtas), x_tiles = (a.M + kTok - 1) / kTok;
  const int64_t tiles = (int64_t)w_tiles * x_tiles;
  const int32_t k_stages = (a.K + kDepth - 1) / kDepth;
  const int32_t sf_tiles = micro_tiles(a.K, kFormat);
  const uint32_t first = blockIdx.x / S::kCtas, step = gridDim.x / S::kCtas;

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S::kStages; ++s) mbar_init(smem_u32(&ctl.full[s]), 1), mbar_init(smem_u32(&ctl.empty[s]), 1);
    for (int i = 0; i < 2; ++i)
      mbar_init(smem_u32(&ctl.acc_full[i]), 1), mbar_init(smem_u32(&ctl.acc_empty[i]), 4 * S::kCtas);
    mbar_init(smem_u32(&ctl.done), 1);
    ctl.abort = 0;
    mbar_init_fence();
  }
  if (kPair)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 5) tmem_alloc<kPair>(smem_u32(&ctl.tmem), kTmemCols);
  tc_fence_before();
  if (kPair)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem, 0);
  // The first rows of the table start towards L2 while the kernel before ends (it may write
  // them: what L2 holds is then written there). The kernel after is not let in early: its
  // waiting blocks beside these cost 2 us of 22 at 97 tokens x 50001 x 2056.
  if (warp == 4 && lane == 0 && x_tiles == 1 && first < tiles)
    for (int32_t k = 0; k < min(k_stages, (int32_t)S::kStages); ++k)
      tensor_prefetch(&wmap, k * 128, (int32_t)(first * S::kCtas + rank) * kRows);
  __syncwarp();
  pdl_wait();  // operands may come from the kernel before; it may still read the output's buffer

  if (warp == 4 && lane == 0) {
    uint32_t s = 0, round = 0;
    bool ok = true;
    for (int64_t t = first; t < tiles && ok; t += step) {
      const int32_t wt = (int32_t)(t / x_tiles), xt = (int32_t)(t - (int64_t)wt * x_tiles);
      const int32_t w_row = wt * kRows * (int32_t)S::kCtas + (int32_t)rank * kRows, x_row = xt * kTok;
      // tokens of this tile, a multiple of 16 a CTA; each CTA brings its half
      const int32_t toks = (min(kTok, a.M - x_row) + 16 * (int32_t)S::kCtas - 1) / (16 * (int32_t)S::kCtas) * 16;
      for (int32_t k = 0; k < k_stages; ++k) {
        if (round && !mbar_wait<kPair>(smem_u32(&ctl.empty[s]), (round - 1) & 1, abort)) {
          ok = false;
          break;
        }
        const uint32_t base = stages + s * S::kStageAligned;
        const uint32_t bar = kPair ? cluster_map(smem_u32(&ctl.full[s]), 0) : smem_u32(&ctl.full[s]);
        if (rank == 0) mbar_expect(smem_u32(&ctl.full[s]), S::kStage * S::kCtas);
        tensor_load<kPair>(base, &wmap, k * 128, w_row, bar);
        tensor_load<kPair>(base + S::kA, &xmap, k * 128, x_row + (int32_t)rank * toks, bar);
        tensor_load<kPair>(base + S::kA + S::kB, &wsmap, k * (int32_t)S::kTiles * 64, w_row / 128, bar);
        tensor_load<kPair>(base + S::kA + S::kB + S::kSA, &xsmap, k * (int32_t)S::kTiles * 64, x_row / 128, bar);
        if (++s == S::kStages) s = 0, ++round;
      }
    }
    // A CTA of a pair stays until its last stages are free: CTA 0's MMAs bring the news.
    for (uint32_t i = 0; kPair && i < S::kStages && ok; ++i) {
      if (round) ok = mbar_wait<kPair>(smem_u32(&ctl.empty[s]), (round - 1) & 1, abort);
      if (++s == S::kStages) s = 0, ++round;
    }
  } else if (warp == 5 && rank == 0) {
    // A: table codes, B: token codes, both E2M1, fp32 sums (bits 7, 10); tokens / 8 (17); E8M0 scales (23); rows / 128 (27)
    constexpr uint32_t idesc0 = 1u << 7 | 1u << 10 | (kFormat == kMicroMX ? 1u << 23 : 0u) | S::kCtas << 27;
    // The whole warp walks the stages, so that addresses and descriptors stay in uniform
    // registers; one lane issues. This warp paces the kernel: a stage is unrolled, with
    // constant offsets. (A single lane walking them took 1250 cycles a stage, 71 instead of
    // 44 us for one token against 128256 x 4096.)
    const bool leader = elect_one();
    const uint32_t full0 = smem_u32(&ctl.full[0]), empty0 = smem_u32(&ctl.empty[0]);
    const uint32_t sfa = tmem + S::kSf, sfb = sfa + S::kTiles * 4;
    constexpr uint32_t kBlock = S::kStageAligned >> 4;  // of a stage, in a descriptor's units
    const uint64_t a_desc0 = operand_desc(stages), sf_desc0 = scales_desc(stages + S::kA + S::kB);
    uint32_t s = 0, parity = 0, j = 0;
    bool ok = true;
    for (int64_t t = first; t < tiles && ok; t += step, ++j) {
      constexpr uint32_t lag = S::kShared ? 1 : 2;  // the tile whose columns this one takes over
      ok = j < lag || mbar_wait<kPair>(smem_u32(&ctl.acc_empty[(j - lag) & 1]), ((j - lag) >> 1) & 1, abort);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint32_t d = tmem + ((j & 1) ? S::kAcc1 : 0);
      const int32_t left = a.M - (int32_t)(t % x_tiles) * kTok;
      const uint32_t toks = (uint32_t)(min(kTok, left) + 16 * (int32_t)S::kCtas - 1) / (16 * S::kCtas) * (16 * S::kCtas);
      const uint32_t idesc = idesc0 | toks / 8 << 17;
      for (int32_t k = 0; k < k_stages; ++k) {
        ok = mbar_wait<kPair>(full0 + s * 8, parity, abort);
        tc_fence_after();
        const uint64_t a_desc = a_desc0 + s * kBlock, b_desc = a_desc + (S::kA >> 4), sf_desc = sf_desc0 + s * kBlock;
        const int32_t used = sf_tiles - k * (int32_t)S::kTiles, steps = (a.K - k * kDepth + kStep - 1) / kStep;
        if (leader && ok) {
#pragma unroll
          for (int i = 0; i < (int)S::kTiles; ++i) {
            if (i >= used) break;
            tc_copy_scales<kPair>(sfa + i * 4, sf_desc + i * 32);
#pragma unroll
            for (uint32_t q = 0; q < S::kTokTiles; ++q)
              tc_copy_scales<kPair>(sfb + (i * S::kTokTiles + q) * 4,
                                    sf_desc + (S::kSA >> 4) + (q * S::kTiles + i) * 32);
          }
#pragma unroll
          for (int e = 0; e < kDepth / kStep; ++e) {
            if (e >= steps) break;
            // MX: a scale tile serves two steps, its bytes 0-1 and 2-3; NV: a tile a step
            const uint32_t i = kFormat == kMicroMX ? e >> 1 : e;
            const uint32_t id = kFormat == kMicroMX ? (e & 1) * 2 : 0;
            tc_mma_f4<kPair, kFormat == kMicroMX>(d, a_desc + e * 2, b_desc + e * 2, idesc | id << 29 | id << 4,
                                                  sfa + i * 4, sfb + i * S::kTokTiles * 4, e > 0 || k > 0);
          }
          tc_commit<kPair>(empty0 + s * 8);
          if (k + 1 == k_stages) tc_commit<kPair>(smem_u32(&ctl.acc_full[j & 1]));
        }
        ok = __all_sync(0xffffffffu, ok);  // all lanes leave if one has given up
        if (!ok) break;
        if (++s == S::kStages) s = 0, parity ^= 1;
      }
    }
    if (leader) tc_commit<kPair, false>(smem_u32(&ctl.done));
  } else if (warp < 4) {
    uint32_t j = 0;
    auto emptied = [&] {
      tc_fence_before();
      if (lane != 0) return;
      if (kPair)
        mbar_arrive_cluster(cluster_map(smem_u32(&ctl.acc_empty[j & 1]), 0));
      else
        mbar_arrive(smem_u32(&ctl.acc_empty[j & 1]));
    };
    bool ok = true;
    for (int64_t t = first; t < tiles; t += step, ++j) {
      const int32_t wt = (int32_t)(t / x_tiles), xt = (int32_t)(t - (int64_t)wt * x_tiles);
      const int32_t n = wt * kRows * (int32_t)S::kCtas + (int32_t)(rank * kRows + warp * 32 + lane);
      ok = ok && __all_sync(0xffffffffu, mbar_wait<kPair>(smem_u32(&ctl.acc_full[j & 1]), (j >> 1) & 1, abort));
      if (!ok) {  // the tiles that will not come
        store_nan<T>(a, n, xt * kTok, kTok);
        continue;
      }
      tc_fence_after();
      const uint32_t d = tmem + ((j & 1) ? S::kAcc1 : 0) + (warp * 32 << 16);
      const uint32_t shared0 = (j & 1) ? 0 : kTok - S::kShared;  // the shared columns come first
      store_columns<T>(a, d, n, xt * kTok, shared0, shared0 + S::kShared);
      if (S::kShared) emptied();
      store_columns<T>(a, d, n, xt * kTok, (j & 1) ? S::kShared : 0, (j & 1) ? kTok : kTok - S::kShared);
      if (!S::kShared) emptied();
    }
  }
  __syncwarp();
  // Nothing may be in flight when the tensor memory goes back, nor when a CTA that holds
  // the pair's barriers or operands ends.
  if (warp == 5 && lane == 0 && rank == 0)
    for (Patience p; !mbar_try(smem_u32(&ctl.done), 0) && !p.over(kDrainNs);) {
    }
  __syncwarp();
  tc_fence_before();
  if (kPair)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  if (*abort) {
    // Copies of abandoned stages may be on their way to this CTA: none takes a millisecond.
    for (Patience p; !p.over(1000000);) {
    }
    if (threadIdx.x == 0) report(a.status, kErrTimeout);
  }
  if (warp == 5) tmem_dealloc<kPair>(tmem, kTmemCols);
}

struct Operands {
  const uint8_t *x, *xs, *w, *ws;
};

template <typename T, int kFormat, int kTok, bool kPair>
cudaError_t launch(int device, MatmulArgs a, const Operands& o, cudaStream_t s) {
  using S = Shape<kFormat, kTok, kPair>;
  const void* fn = reinterpret_cast<const void*>(&k_micro_matmul<T, kFormat, kTok, kPair>);
  static bool ready[64];
  cudaError_t e = allow_smem(fn, S::kSmem, device, ready);
  const int64_t row_bytes = micro_row_bytes(a.K), sf_tiles = micro_tiles(a.K, kFormat);
  CUtensorMap wmap, wsmap, xmap, xsmap;
  if (e == cudaSuccess) e = byte_matrix_map(&wmap, o.w, a.N, row_bytes, kRows);
  if (e == cudaSuccess) e = tile_matrix_map(&wsmap, o.ws, (a.N + 127) / 128, sf_tiles, 1, S::kTiles);
  if (e == cudaSuccess) e = byte_matrix_map(&xmap, o.x, a.M, row_bytes, kTok / S::kCtas);
  if (e == cudaSuccess) e = tile_matrix_map(&xsmap, o.xs, (a.M + 127) / 128, sf_tiles, S::kTokTiles, S::kTiles);
  if (e != cudaSuccess) return e;
  const int64_t rows = kRows * S::kCtas;
  const int64_t tiles = (a.N + rows - 1) / rows * ((a.M + kTok - 1) / kTok), most = sm_count(device) / S::kCtas;
  const unsigned grid = (unsigned)(tiles < most ? tiles : most) * S::kCtas;
  void* args[] = {&wmap, &wsmap, &xmap, &xsmap, &a};
  return kPair ? launch_clusters(fn, dim3(grid), dim3(kMatmulThreads), 2, S::kSmem, s, args, true)
               : launch_kernel(fn, dim3(grid), dim3(kMatmulThreads), S::kSmem, s, args, true);
}

template <typename T, int kFormat>
cudaError_t launch_tok(int device, const MatmulArgs& a, const Operands& o, cudaStream_t s) {
  // the narrowest tile that holds the tokens
  if (a.M <= 16) return launch<T, kFormat, 16, false>(device, a, o, s);
  if (a.M <= 64) return launch<T, kFormat, 64, true>(device, a, o, s);
  if (a.M <= 128) return launch<T, kFormat, 128, true>(device, a, o, s);
  return launch<T, kFormat, 256, true>(device, a, o, s);
}

template <int kFormat>
cudaError_t launch_type(int device, int dtype, const MatmulArgs& a, const Operands& o, cudaStream_t s) {
  switch (dtype) {
    case EMB_F32: return launch_tok<float, kFormat>(device, a, o, s);
    case EMB_F16: return launch_tok<__half, kFormat>(device, a, o, s);
    default: return launch_tok<__nv_bfloat16, kFormat>(device, a, o, s);
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
  const MatmulArgs a{M, N, K, x_tensor_scale * w_tensor_scale, out, out_stride, device_status};
  const Operands o{x_codes, x_scales, w_codes, w_scales};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return on_device(device, [&] {
    return format == EMB_MICRO_MX ? launch_type<kMicroMX>(device, out_dtype, a, o, s)
                                  : launch_type<kMicroNV>(device, out_dtype, a, o, s);
  });
}
