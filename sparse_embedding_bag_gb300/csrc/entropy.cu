// Softmax cross entropy of hidden states against a table of V tokens, without the N x V
// logits in memory: z = h W^T, loss = log sum exp z - z_target, and with
// G = weight (softmax(z) - onehot(target)) the gradients dh = G W and dW = G^T h.
//
// Rows that take part are packed first (k_entropy_rows), so that rows without a target cost
// nothing and whatever they hold reaches no sum. Forward: tiles of logits are computed
// on the tensor cores and reduced where they are to a reference and a sum of exponentials a
// row and tile (k_entropy_mm<Logits>), which k_entropy_loss joins. Backward: the vocabulary is
// taken in pieces; a piece's logits are computed again and leave as G in the operands' type
// (Logits with kGradient), then one launch multiplies G with both sides (k_entropy_mm<Grads>):
// the piece's rows of dW, whole sums over the tokens, and its part of dh, added to fp32 sums in
// the workspace. The order of all sums is fixed, and none stays in one accumulator for longer than
// most_summed() elements.
//
// G is rounded to the operands' type because the tensor cores take two operands of one type.
// bf16 keeps its range; fp16 is scaled by a power of two that brings the largest weight
// to 2^14..2^15, so that probabilities down to 2^-28 keep all bits in a row of that weight, and down to
// 2^(k - 28) in one whose weight is 2^-k of it (one scale for all rows: dW adds up rows). Gradients
// then carry two roundings, 0.0024 of the norm in bf16 and 0.00030 in fp16 where one makes 0.0017 and
// 0.00021. Up to 64 tokens G is two such
// numbers, its rounding and what that leaves, in rows n and n + 64 (up to 32 tokens n + 32) of a tile, which no token fills:
// with few tokens single roundings show in the gradients (5 % of the time at 128256 x 4096; two
// tiles of 128 tokens would cost 33 %; for all tokens both products of G, half of a step's time, would double).
//
// The products share one frame (k_entropy_mm): persistent CTAs, in pairs above 128 tokens
// (tiles of up to 256 x 256, each CTA half of both operands), stages 64 elements deep by TMA in the
// 128-byte swizzle, one warp that issues copies, one that issues MMAs, two groups of four
// warps that empty the two accumulators in tensor memory in turn. Measured (bf16): logits of 1024
// tokens against 128256 x 4096 in 565 us, 1.9 PFLOP/s, the tensor pipe 94 % busy; of one token
// 154 us, 6.8 TB/s; gradients of 4096 tokens 5.2 ms, 1.65 PFLOP/s, the tensor pipe 84 % busy where
// power does not limit it. Not kept: letting each kernel start while the one before ends (no
// difference from 16 tokens to 4096; only the losses of few tokens have work to do meanwhile).
#include <cmath>

#include "sm103.cuh"

namespace embbwd {
namespace {

constexpr int kDepth = 64;    // elements of a stage
constexpr int kMmThreads = 320;
constexpr uint32_t kSmemMost = 226 * 1024;
constexpr float kLog2e = 1.44269504f;
constexpr float kLn2 = 0.693147181f;

constexpr int64_t kMaxTokens = 1 << 20;
constexpr int32_t kMaxWidth = 1 << 15;
// Of G. Few large pieces: 4096 tokens, 128256 x 4096 bf16, loss and gradients, take 10.8 ms with
// 64 MB (G stays in L2), 10.3 with 128, 9.9 with 256, 9.8 with 512, 9.9 with the whole 1 GB;
// 1024 tokens, 50001 x 2056 fp16, gradients, 712, 567, 486, 455 us. A launch's first and
// last tiles cost more than G's way to HBM and back.
constexpr int64_t kPieceBytes = (int64_t)512 << 20;

// ---- packing the rows that take part

struct RowArgs {
  const void* hidden;
  int64_t stride;
  int32_t N, D, V;
  const int64_t* targets;
  const float* weight;  // NULL: 1
  const float* lse;     // NULL: par.x is not known yet
  uint16_t* rows;       // packed [cap, Dp]
  int32_t Dp;
  int32_t per_block;
  bool gradients;
  int32_t second;       // where rows are packed a second time, or 0
  bool scaled;          // choose a scale for fp16
  int32_t* count;
  int32_t* rank;        // [N]: packed row of a row, or -1
  const void* table;
  int64_t table_stride;
  int32_t* target;      // [cap]
  float* at_target;     // [cap]: the target's logit
  float2* par;          // [cap]: log2 of the sum of 2^(z log2 e), scaled weight
  float* scale;         // the scale of G and its reciprocal
  uint32_t* status;
};

// Elements k..k+7 of a row of D 16-bit elements, zeros after its end. Rows off 16-byte
// boundaries come in the words that cover them.
__device__ __forceinline__ uint4 load_eight(const uint16_t* src, int32_t k, int32_t D) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(src);
  const int32_t odd = (int32_t)(at / 2 % 2);
  if (at % 16 == 0 && k + 8 <= D) return *reinterpret_cast<const uint4*>(src + k);
  if (k >= odd && k + 8 + odd <= D) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(src + k - odd);
    if (!odd) return make_uint4(w[0], w[1], w[2], w[3]);
    return make_uint4(__funnelshift_r(w[0], w[1], 16), __funnelshift_r(w[1], w[2], 16), __funnelshift_r(w[2], w[3], 16),
                      __funnelshift_r(w[3], w[4], 16));
  }
  uint16_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = k + i < D ? src[k + i] : 0;
  return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}
template <typename T>
__device__ __forceinline__ float dot_eight(const uint4& x, const uint4& y, float sum) {
  float a[kGroup], b[kGroup];
  Raw8<T> u, v;
  u.u[0] = x, v.u[0] = y;
  u.widen(a), v.widen(b);
#pragma unroll
  for (int i = 0; i < kGroup; ++i) sum = fmaf(a[i], b[i], sum);
  return sum;
}

// Every block counts the rows that take part before its own (targets are few beside
// the rows that it copies), so that no launch has to come before. The logit of a row's
// target is summed here by fp32 FMAs: the tensor cores' sums lose their last bits (at
// D = 4096 some 3e-6 of a logit), which a loss that is the difference of two large numbers
// would show; it takes the place of the tiles' own. Bound by latency: 7 us for 301 rows, 32 for 4096 of
// 4096 elements (2.1 TB/s of rows read and written, as much again of the targets' rows).
constexpr int kPartSums = 8;
template <typename T>
__global__ void __launch_bounds__(kThreads) k_entropy_rows(RowArgs a) {
  __shared__ float f_scratch[kWarps], sums[kWarps][kPartSums];
  __shared__ int32_t before_w[kWarps], all_w[kWarps], list[kThreads], goal[kThreads], rank_w[kWarps];
  pdl_wait();
  const int32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t r0 = min(a.N, (int32_t)blockIdx.x * a.per_block), r1 = min(a.N, r0 + a.per_block);
  int32_t before = 0, all = 0;
  float most = 0.f;
  constexpr int kBatch = 8;  // targets asked for at once
  for (int32_t i0 = tid; i0 < a.N; i0 += kThreads * kBatch) {
    int64_t t[kBatch];
    float w[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int32_t i = i0 + b * kThreads;
      t[b] = i < a.N ? a.targets[i] : -1;
      w[b] = a.scaled && a.weight && i < a.N ? a.weight[i] : 1.f;
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const bool part = t[b] >= 0 && t[b] < a.V;
      all += part;
      before += part && i0 + b * kThreads < r0;
      if (part) most = fmaxf(most, fabsf(w[b]));
    }
  }
  before = __reduce_add_sync(0xffffffffu, before), all = __reduce_add_sync(0xffffffffu, all);
  most = warp_max(most);
  if (lane == 0) before_w[warp] = before, all_w[warp] = all, f_scratch[warp] = most;
  __syncthreads();
  before = all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) before += before_w[w], all += all_w[w], most = fmaxf(most, f_scratch[w]);
  // the largest weight to 2^14 .. 2^15; both factors normal
  float scale = 1.f;
  if (a.scaled && most > 0.f && most < INFINITY) {
    const int e = min(max(14 - ((int)(__float_as_uint(most) >> 23) - 127), -125), 125);
    scale = __uint_as_float((uint32_t)(127 + e) << 23);
  }
  if (blockIdx.x == 0 && tid == 0) *a.count = all, a.scale[0] = scale, a.scale[1] = 1.f / scale;

  for (int32_t base = r0; base < r1; base += kThreads) {
    const int32_t r = base + tid;
    const int64_t t = r < r1 ? a.targets[r] : -1;
    if (t >= a.V) report(a.status, kErrIndex);
    const bool part = t >= 0 && t < a.V;
    const uint32_t ballot = __ballot_sync(0xffffffffu, part);
    if (lane == 0) rank_w[warp] = __popc(ballot);
    __syncthreads();
    int32_t at = __popc(ballot & lanemask_lt()), here = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += rank_w[w];
      here += rank_w[w];
    }
    const int32_t n = before + at;
    if (r < r1) a.rank[r] = part ? n : -1;
    if (part) {
      list[at] = r, goal[at] = (int32_t)t;
      a.target[n] = (int32_t)t;
      a.par[n] = make_float2(a.lse ? a.lse[r] * kLog2e : 0.f, (a.weight ? a.weight[r] : 1.f) * scale);
    }
    __syncthreads();
    // a block's warps share out its rows: few rows, several warps each. However many take a row, its sum is that of
    // kPartSums, each of every eighth 256 elements: its bits do not depend on which of its neighbours take part
    const int32_t row_warps = here <= 1 ? 8 : here <= 2 ? 4 : here <= 4 ? 2 : 1;
    const int32_t together = kWarps / row_warps, lanes = row_warps * 32, l = tid & (lanes - 1);
    for (int32_t j = 0; j < here; j += together) {
      const int32_t i = j + tid / lanes;
      float part_of[kPartSums] = {};
      if (i < here) {
        const uint16_t* from = static_cast<const uint16_t*>(a.hidden) + (int64_t)list[i] * a.stride;
        const uint16_t* with = static_cast<const uint16_t*>(a.table) + (int64_t)goal[i] * a.table_stride;
        uint16_t* to = a.rows + (int64_t)(before + i) * a.Dp;
#pragma unroll 4
        for (int32_t k = l * 8; k < a.Dp; k += lanes * 8) {
          const uint4 u = load_eight(from, k, a.D);
          *reinterpret_cast<uint4*>(to + k) = u;
          if (a.second) *reinterpret_cast<uint4*>(to + (int64_t)a.second * a.Dp + k) = u;
          const float z = dot_eight<T>(u, load_eight(with, k, a.D), 0.f);
          const int32_t own = k / 256 % kPartSums;
#pragma unroll
          for (int s = 0; s < kPartSums; ++s) part_of[s] += s == own ? z : 0.f;
        }
      }
#pragma unroll
      for (int s = 0; s < kPartSums; ++s) part_of[s] = warp_sum(part_of[s]);
      if (row_warps > 1) {  // the others' parts are zeros here
        if (lane == 0) {
#pragma unroll
          for (int s = 0; s < kPartSums; ++s)
            if (s % row_warps == warp % row_warps) sums[warp / row_warps][s] = part_of[s];
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kPartSums; ++s) part_of[s] = sums[warp / row_warps][s];
        __syncthreads();
      }
      float z = 0.f;
#pragma unroll
      for (int s = 0; s < kPartSums; ++s) z += part_of[s];
      if (i < here && l == 0) a.at_target[before + i] = z;
    }
    before += here;
    __syncthreads();
  }
  // zeros up to a whole stage of the products that sum over the tokens
  const int32_t end = a.second ? a.second : a.gradients ? (all + kDepth - 1) / kDepth * kDepth : 0;
  for (int32_t n = all + (int32_t)blockIdx.x; n < end; n += gridDim.x)
    for (int32_t k = tid * 8; k < a.Dp; k += kThreads * 8) {
      uint16_t* to = a.rows + (int64_t)n * a.Dp + k;
      *reinterpret_cast<uint4*>(to) = make_uint4(0, 0, 0, 0);
      if (a.second) *reinterpret_cast<uint4*>(to + (int64_t)a.second * a.Dp) = make_uint4(0, 0, 0, 0);
    }
}

// Rows of G, of dh's parts: the packed ones, or with a second part whole tiles.
__host__ __device__ inline int32_t rows_of_g(int32_t count, int32_t second) { return second && count ? 2 * second : count; }

// A table whose rows TMA cannot read (off 16-byte boundaries, or ending between them), padded. Bound
// by HBM: 40 us for 50001 x 1031, 5.1 TB/s.
__global__ void __launch_bounds__(kThreads) k_entropy_pad(const uint16_t* table, int64_t stride, uint16_t* out, int32_t V,
                                                          int32_t D, int32_t Dp) {
  pdl_wait();
  const int64_t v = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (v >= V) return;
#pragma unroll 4
  for (int32_t k = (threadIdx.x & 31) * 8; k < Dp; k += 256)
    *reinterpret_cast<uint4*>(out + v * Dp + k) = load_eight(table + v * stride, k, D);
}

// ---- the frame of the products

// Tiles of up to kColumns columns; `kAsideBytes` of shared memory are for each warp of the epilogue.
template <bool kPair, int kColumns, uint32_t kAsideBytes>
struct Shape {
  static constexpr uint32_t kCtas = kPair ? 2 : 1;
  static constexpr int32_t kRows = 128 * kCtas;         // rows of a tile
  static constexpr int32_t kCols = kColumns;            // of an accumulator
  static constexpr int32_t kWidth = kCols / kCtas;      // columns that one CTA brings
  static constexpr uint32_t kA = 128 * 128, kB = kWidth * 128, kStage = kA + kB, kAside = kAsideBytes;
  static constexpr uint32_t kStages = (kSmemMost - 2048 - 8 * kAside) / kStage;
  static constexpr uint32_t kSmem = kStages * kStage + 8 * kAside + 2048;
};

struct Control {
  uint64_t full[8], empty[8], acc_full[2], acc_empty[2], done;
  uint32_t tmem;
  int abort;
};

struct Maps {
  CUtensorMap a, b, c;  // read in boxes
  CUtensorMap out;      // written in boxes of 32 rows x 64 columns of 16 bits
};

// fp32 sums (bit 4), operands' type (7, 10: 1 = bf16), columns / 8 (17), rows / 16 (24);
// bits 15, 16: A, B run along M, N
template <typename T>
__device__ __forceinline__ uint32_t idesc16(uint32_t rows, uint32_t cols) {
  constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
  return 1u << 4 | type << 7 | type << 10 | cols / 8 << 17 | rows / 16 << 24;
}

template <typename T>
__device__ __forceinline__ uint32_t two(float x, float y) {
  const T e[2] = {Elem<T>::put(x), Elem<T>::put(y)};
  uint32_t u;
  memcpy(&u, e, 4);
  return u;
}

// A warp's 32 rows x 64 columns, lane by lane a row, to its 4096 bytes of shared memory, in the
// 128-byte swizzle; and from there to the output. (Stored by each lane to its own row a tile of
// 128 x 256 took 2 us: every store touches 32 lines.)
template <typename T>
__device__ __forceinline__ void fill_box(uint8_t* aside, uint32_t lane, const float (&v)[2][32]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float* e = v[i / 4] + i % 4 * 8;
    *reinterpret_cast<uint4*>(aside + lane * 128 + ((i ^ (lane & 7)) * 16)) =
        make_uint4(two<T>(e[0], e[1]), two<T>(e[2], e[3]), two<T>(e[4], e[5]), two<T>(e[6], e[7]));
  }
}
template <typename T>
__device__ __forceinline__ void store_box(const CUtensorMap* out, int32_t x, int32_t y, uint8_t* aside, uint32_t lane,
                                          const float (&v)[2][32]) {
  if (lane == 0) bulk_wait_read();  // the box before has left
  __syncwarp();
  fill_box<T>(aside, lane, v);
  bulk_fence();
  __syncwarp();
  if (lane == 0) tensor_store(out, x, y, smem_u32(aside));
}
// The same to rows that bulk copies cannot write (off 16-byte boundaries, or not whole pieces of 16): 32 lanes write 32
// elements of a row side by side. `rows`, `cols`: how much of the box there is.
template <typename T>
__device__ __forceinline__ void store_box_plain(uint16_t* out, int64_t stride, int32_t rows, int32_t cols, uint8_t* aside,
                                                uint32_t lane, const float (&v)[2][32]) {
  __syncwarp();  // the box before has been read
  fill_box<T>(aside, lane, v);
  __syncwarp();
  const bool left = (int32_t)lane < cols, right = (int32_t)lane + 32 < cols;
  out += lane;
#pragma unroll 8
  for (int32_t r = 0; r < 32; ++r, out += stride) {
    const uint8_t* row = aside + r * 128 + lane % 8 * 2;
    const uint16_t x = *reinterpret_cast<const uint16_t*>(row + ((lane / 8 ^ (r & 7)) * 16));
    const uint16_t y = *reinterpret_cast<const uint16_t*>(row + ((lane / 8 + 4 ^ (r & 7)) * 16));
    if (r < rows && left) out[0] = x;
    if (r < rows && right) out[32] = y;
  }
}

// What a CTA group does for one tile after another. Policy:
//   Policy(args, group, groups)   after the kernel before has ended
//   bool next()                   the next tile with k_stages() > 0, or one to fill with zeros
//   load(maps, k, base, bar, rank), a_desc/b_desc(base), a_step, b_step, idesc
//   store(maps, tmem, warp (0..3), lane, rank, aside, ok, zero)   lane `lane` of the warp holds a row
// With kChunk an accumulator sums kChunk stages, and the epilogue's groups add these sums in registers,
// half of the columns each (zeros of a tile without stages):
//   finish(maps, sums, group, warp, lane, rank, aside, ok)
template <typename Policy, bool kPair>
__global__ void __launch_bounds__(kMmThreads, 1)
    k_entropy_mm(const __grid_constant__ Maps maps, const __grid_constant__ typename Policy::Args args) {
  using S = typename Policy::S;
  constexpr uint32_t kStages = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Control ctl;
  const uint32_t stages = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_rank() : 0;
  volatile int* abort = &ctl.abort;

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < kStages; ++s) mbar_init(smem_u32(&ctl.full[s]), 1), mbar_init(smem_u32(&ctl.empty[s]), 1);
    for (int i = 0; i < 2; ++i)
      mbar_init(smem_u32(&ctl.acc_full[i]), 1), mbar_init(smem_u32(&ctl.acc_empty[i]), (Policy::kChunk ? 8 : 4) * S::kCtas);
    mbar_init(smem_u32(&ctl.done), 1);
    ctl.abort = 0;
    mbar_init_fence();
  }
  if (kPair)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 9) tmem_alloc<kPair>(smem_u32(&ctl.tmem), 512);
  tc_fence_before();
  if (kPair)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem, 0);
  pdl_wait();
  Policy p(args, (int32_t)(blockIdx.x / S::kCtas), (int32_t)(gridDim.x / S::kCtas));

  if (warp == 8 && lane == 0) {
    uint32_t s = 0, round = 0;
    bool ok = true;
    while (ok && p.next()) {
      const int32_t n = p.k_stages();
      for (int32_t k = 0; k < n; ++k) {
        if (round && !mbar_wait<kPair>(smem_u32(&ctl.empty[s]), (round - 1) & 1, abort)) {
          ok = false;
          break;
        }
        const uint32_t bar = kPair ? cluster_map(smem_u32(&ctl.full[s]), 0) : smem_u32(&ctl.full[s]);
        if (rank == 0) mbar_expect(smem_u32(&ctl.full[s]), p.stage_bytes() * S::kCtas);
        p.load(maps, k, stages + s * S::kStage, bar, rank);
        if (++s == kStages) s = 0, ++round;
      }
    }
    // A CTA of a pair stays until its last stages are free: CTA 0's MMAs bring the news.
    for (uint32_t i = 0; kPair && i < kStages && ok; ++i) {
      if (round) ok = mbar_wait<kPair>(smem_u32(&ctl.empty[s]), (round - 1) & 1, abort);
      if (++s == kStages) s = 0, ++round;
    }
  } else if (warp == 9 && rank == 0) {
    // the whole warp walks the stages, one lane issues
    const bool leader = elect_one();
    const uint32_t full0 = smem_u32(&ctl.full[0]), empty0 = smem_u32(&ctl.empty[0]);
    uint32_t s = 0, parity = 0, j = 0;
    bool ok = true;
    while (ok && p.next()) {
      const int32_t n = p.k_stages();
      if (n == 0) continue;
      const uint32_t idesc = p.idesc(), a_step = p.a_step(), b_step = p.b_step();
      const uint64_t a0 = p.a_desc(stages), b0 = p.b_desc(stages + S::kA);
      const int32_t chunk = Policy::kChunk ? Policy::kChunk : n;  // stages that one accumulator sums
      for (int32_t k = 0, c = 0; k < n; ++k) {
        if (c == 0) {
          ok = j < 2 || mbar_wait<kPair>(smem_u32(&ctl.acc_empty[j & 1]), ((j - 2) >> 1) & 1, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t d = tmem + (j & 1) * S::kCols;
        const bool last = k + 1 == n || c + 1 == chunk;
        ok = mbar_wait<kPair>(full0 + s * 8, parity, abort);
        tc_fence_after();
        if (leader && ok) {
          const uint64_t a = a0 + s * (S::kStage >> 4), b = b0 + s * (S::kStage >> 4);
#pragma unroll
          for (uint32_t e = 0; e < kDepth / 16; ++e)
            tc_mma_16<kPair>(d, a + e * a_step, b + e * b_step, idesc, e > 0 || c > 0);
          tc_commit<kPair>(empty0 + s * 8);
          if (last) tc_commit<kPair>(smem_u32(&ctl.acc_full[j & 1]));
        }
        ok = __all_sync(0xffffffffu, ok);  // all lanes leave if one has given up
        if (!ok) break;
        if (++s == kStages) s = 0, parity ^= 1;
        c = last ? 0 : c + 1;
        j += last;
      }
    }
    if (leader) tc_commit<kPair, false>(smem_u32(&ctl.done));
  } else if (warp < 8) {
    uint32_t j = 0;
    bool ok = true;
    const uint32_t group = warp >> 2, lanes = (warp & 3) * 32 << 16;
    auto filled = [&](uint32_t i) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait<kPair>(smem_u32(&ctl.acc_full[i & 1]), (i >> 1) & 1, abort));
      tc_fence_after();
    };
    auto emptied = [&](uint32_t i) {
      tc_fence_before();
      __syncwarp();
      if (lane != 0 || !ok) return;
      if (kPair)
        mbar_arrive_cluster(cluster_map(smem_u32(&ctl.acc_empty[i & 1]), 0));
      else
        mbar_arrive(smem_u32(&ctl.acc_empty[i & 1]));
    };
    uint8_t* aside = smem_raw + (stages - smem_u32(smem_raw)) + kStages * S::kStage + warp * S::kAside;
    if constexpr (Policy::kChunk > 0) {
      constexpr int kHalf = S::kCols / 2;
      while (p.next()) {
        float v[kHalf];
        const int32_t n = p.k_stages();
        if (n == 0) {
#pragma unroll
          for (int i = 0; i < kHalf; ++i) v[i] = 0.f;
        }
        for (int32_t left = n; left > 0; left -= Policy::kChunk, ++j) {
          filled(j);
          const bool first = left == n;
#pragma unroll
          for (int q = 0; q < kHalf; q += 16) {
            if (!ok) break;
            float x[16];
            tmem_load16(tmem + (j & 1) * S::kCols + group * kHalf + q + lanes, x);
            tmem_load_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[q + i] = first ? x[i] : v[q + i] + x[i];
          }
          emptied(j);
        }
        p.finish(maps, v, group, warp & 3, lane, rank, aside, ok || n == 0);
      }
    } else {
      for (uint32_t i = 0; p.next(); ++i) {
        if (p.k_stages() == 0) {
          if ((i & 1) == group) p.store(maps, tmem, warp & 3, lane, rank, aside, false, true);
          continue;
        }
        const uint32_t mine = j++;
        if ((mine & 1) != group) continue;
        filled(mine);
        p.store(maps, tmem + group * S::kCols + lanes, warp & 3, lane, rank, aside, ok, false);
        emptied(mine);
      }
    }
    if (S::kAside && lane == 0) bulk_wait();
  }
  __syncwarp();
  // Nothing may be in flight when the tensor memory goes back, nor when a CTA that holds
  // the pair's barriers or operands ends.
  if (warp == 9 && lane == 0 && rank == 0)
    for (Patience w; !mbar_try(smem_u32(&ctl.done), 0) && !w.over(kDrainNs);) {
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
    for (Patience w; !w.over(1000000);) {
    }
    if (threadIdx.x == 0) report(args.status, kErrTimeout);
  }
  if (warp == 9) tmem_dealloc<kPair>(tmem, 512);
}

// ---- logits of a range of the vocabulary

struct LogitArgs {
  const int32_t* count;     // NULL: the rows are taken as they are, `N` of them
  int32_t N;
  const int64_t* targets;   // of rows taken as they are
  int32_t D, V0, V1;
  int32_t a_rows;  // rows of an A box
  int32_t second;  // gradient: rows from here on hold what G's rounding leaves, or 0
  int32_t cols;    // of a tile
  const int32_t* target;
  float2* partial;  // sums: [tiles, cap] (long ones: [2 tiles, cap], of each half) {reference, sum of 2^(z log2 e - reference) but for the target}
  int64_t cap;
  const float* at_target;  // [cap], the target's logit
  const float2* par;
  uint32_t* status;
};

constexpr int32_t kMostPlain = 8192;  // elements of fp16 rows whose gradients take logits of one sum

// Tiles run over the tokens first: the hidden states stay in L2, the table is read once.
enum LogitKind { kSums, kLongSums, kGradient, kLongGradient };
template <typename T, bool kPair, LogitKind kKind>
struct Logits {
  using Args = LogitArgs;
  static constexpr bool kOfGradient = kKind == kGradient || kKind == kLongGradient;
  using S = Shape<kPair, 256, kOfGradient ? 4096 : 0>;
  // The tensor cores cut what an accumulator cannot hold, towards zero, at every 16 elements: sums
  // over 4096 elements gave losses 0.9e-6 off, over 8192 2.7e-6. Wider rows (kLongSums) are
  // summed 2048 elements at a time. (Up to there each group of warps takes a whole tile: 271 tokens,
  // 50001 x 1031, 45 us instead of 58.) A logit of 15 that is not the target's is then off by 7e-5 at most.
  // fp16 gradients show such logits from 8192 elements on: up to there 0.00021 of the norm became 0.00023,
  // at 32768 0.00044 (kLongGradient: 0.00021). bf16 ones do not.
  static constexpr int kChunk = kKind == kLongSums || kKind == kLongGradient ? 32 : 0;
  const Args& a;
  uint32_t m_tiles, step, t, tiles;  // fewer than 2^29: divisions of 32 bits, between two tiles' MMAs
  int32_t count, m, n;
  __device__ Logits(const Args& args, int32_t group, int32_t groups) : a(args), step(groups) {
    if (!a.count) pdl_trigger();  // the losses' kernel has work that does not wait for the tiles
    count = a.count ? *a.count : a.N;
    m_tiles = ((kOfGradient ? rows_of_g(count, a.second) : count) + S::kRows - 1) / S::kRows;
    tiles = m_tiles * (uint32_t)((a.V1 - a.V0 + a.cols - 1) / a.cols);
    t = (uint32_t)(group - groups);
  }
  __device__ bool next() {
    t += step;
    if (t >= tiles) return false;
    n = (int32_t)(t / m_tiles), m = (int32_t)(t - n * m_tiles);
    return true;
  }
  __device__ int32_t k_stages() const { return (a.D + kDepth - 1) / kDepth; }
  __device__ uint32_t stage_bytes() const { return (uint32_t)a.a_rows * 128 + (uint32_t)(a.cols / S::kCtas) * 128; }
  __device__ void load(const Maps& maps, int32_t k, uint32_t base, uint32_t bar, uint32_t rank) const {
    tensor_load<kPair>(base, &maps.a, k * kDepth, m * S::kRows + (int32_t)rank * 128, bar);
    tensor_load<kPair>(base + S::kA, &maps.b, k * kDepth, a.V0 + n * a.cols + (int32_t)rank * (a.cols / (int32_t)S::kCtas), bar);
  }
  __device__ uint64_t a_desc(uint32_t at) const { return operand_desc(at); }
  __device__ uint64_t b_desc(uint32_t at) const { return operand_desc(at); }
  __device__ uint32_t a_step() const { return 2; }
  __device__ uint32_t b_step() const { return 2; }
  __device__ uint32_t idesc() const { return idesc16<T>(S::kRows, a.cols); }

  // Where the target of a row is in the tile, or -1.
  __device__ int32_t target_in_tile(int32_t row, int32_t v0, int32_t cols) const {
    if (row >= count) return -1;
    const int64_t at = (a.targets ? a.targets[row] : (int64_t)a.target[row]) - v0;
    return at >= 0 && at < cols ? (int32_t)at : -1;
  }
  // What a lane needs to know of its row of the tile to make it G.
  struct Row {
    int32_t row, cols, hit;
    bool left, part;
    float z_hit;
    float2 par;
  };
  __device__ Row row_of(uint32_t warp, uint32_t lane, uint32_t rank) const {
    Row r;
    r.row = m * S::kRows + (int32_t)(rank * 128 + warp * 32 + lane);
    r.left = a.second && r.row >= a.second;
    const int32_t token = r.left ? r.row - a.second : r.row, v0 = a.V0 + n * a.cols;
    r.part = token < count;
    r.cols = min(a.cols, a.V1 - v0), r.hit = target_in_tile(token, v0, r.cols);
    r.z_hit = r.part ? a.at_target[token] : 0.f;
    r.par = r.part ? a.par[token] : make_float2(0.f, 0.f);
    return r;
  }
  // Columns c..c+63 of the tile, as G.
  __device__ void leave(const Maps& maps, const Row& r, float (&v)[2][32], int32_t c, uint32_t lane, uint8_t* aside, bool ok) const {
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      float& x = v[i / 32][i % 32];
      const bool here = r.hit - c == i;
      float p = ex2(fmaf(here ? r.z_hit : x, kLog2e, -r.par.x));
      if (here) p -= 1.f;
      x = !r.part || c + i >= r.cols ? 0.f : ok ? p * r.par.y : NAN;
    }
    if (r.left) {  // all lanes of a warp, or none
#pragma unroll
      for (int i = 0; i < 64; ++i) v[i / 32][i % 32] -= Elem<T>::get(Elem<T>::put(v[i / 32][i % 32]));
    }
    store_box<T>(&maps.out, n * a.cols + c, r.row - (int32_t)lane, aside, lane, v);
  }
  // A thread holds a token's row of the tile.
  __device__ void store(const Maps& maps, uint32_t tmem, uint32_t warp, uint32_t lane, uint32_t rank, uint8_t* aside, bool ok,
                        bool) const {
    if constexpr (kOfGradient) {
      const Row r = row_of(warp, lane, rank);
#pragma unroll 1
      for (int32_t c = 0; c < a.cols; c += 64) {
        float v[2][32];
        __syncwarp();
        if (ok) {
          tmem_load32(tmem + c, v[0]);
          tmem_load32(tmem + c + 32, v[1]);
          tmem_load_wait();
        }
        leave(maps, r, v, c, lane, aside, ok);
      }
      return;
    }
    const int32_t row = m * S::kRows + (int32_t)(rank * 128 + warp * 32 + lane);
    const bool part = row < count;
    const int32_t v0 = a.V0 + n * a.cols, cols = min(a.cols, a.V1 - v0), hit = target_in_tile(row, v0, cols);
    float ref = -INFINITY, sum = 0.f;
#pragma unroll 1
    for (int32_t c = 0; c < cols && ok; c += 32) {
      float v[32];
      __syncwarp();
      tmem_load32(tmem + c, v);
      tmem_load_wait();
      if (c + 32 > cols || (hit >= c && hit < c + 32)) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c + i >= cols || c + i == hit) v[i] = -INFINITY;  // the target joins at the end, with all its bits
      }
      float most = v[0];
#pragma unroll
      for (int i = 1; i < 32; ++i) most = fmaxf(most, v[i]);
      const float next = fmaxf(ref, most * kLog2e), base = next == -INFINITY ? 0.f : next;
      float part4[4] = {sum * ex2(ref - base), 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 32; ++i) part4[i & 3] += ex2(fmaf(v[i], kLog2e, -base));
      sum = (part4[0] + part4[1]) + (part4[2] + part4[3]);
      ref = next;
    }
    if (part) a.partial[(int64_t)n * a.cap + row] = make_float2(ref, ok ? sum : NAN);
  }
  // Half of the tile's columns, from registers.
  __device__ void finish(const Maps& maps, float (&v)[128], uint32_t group, uint32_t warp, uint32_t lane, uint32_t rank,
                         uint8_t* aside, bool ok) const {
    if constexpr (kOfGradient) {
      const Row r = row_of(warp, lane, rank);
#pragma unroll
      for (int c = 0; c < 128; c += 64) {
        const int32_t at = (int32_t)group * 128 + c;
        if (at >= a.cols) continue;
        leave(maps, r, *reinterpret_cast<float (*)[2][32]>(v + c), at, lane, aside, ok);
      }
      return;
    }
    const int32_t row = m * S::kRows + (int32_t)(rank * 128 + warp * 32 + lane);
    const int32_t v0 = a.V0 + n * a.cols + (int32_t)group * 128;
    const int32_t cols = min(a.cols - (int32_t)group * 128, a.V1 - v0), hit = target_in_tile(row, v0, cols);
    float ref = -INFINITY, sum = 0.f;
    if (ok && cols > 0) {
      if (cols < 128 || hit >= 0) {
#pragma unroll
        for (int i = 0; i < 128; ++i)
          if (i >= cols || i == hit) v[i] = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < 128; ++i) ref = fmaxf(ref, v[i]);
      ref *= kLog2e;
      const float base = ref == -INFINITY ? 0.f : ref;
      float part4[4] = {};
#pragma unroll
      for (int i = 0; i < 128; ++i) part4[i & 3] += ex2(fmaf(v[i], kLog2e, -base));
      sum = (part4[0] + part4[1]) + (part4[2] + part4[3]);
    }
    if (row < count) a.partial[((int64_t)n * 2 + group) * a.cap + row] = make_float2(ref, ok ? sum : NAN);
  }
};

// ---- the tiles' sums joined

struct LossArgs {
  int32_t N, tiles, V, D;
  const int32_t* rank;       // NULL: rows are taken as they are, and their targets' logits found here
  const float2* partial;
  int64_t cap;
  const float* at_target;
  const void *hidden, *table;
  int64_t hidden_stride, table_stride;
  const int64_t* targets;
  float* loss;
  float* lse;   // may be NULL
  float2* par;  // may be NULL: takes the binary logarithm of the sum
  uint32_t* status;
};

constexpr int kLossWarps = 32;

// 32 rows a block; a warp finds a row's target's logit, then joins every 32nd tile of all rows. Bound by
// latency: 4 to 9 us.
template <typename T>
__global__ void __launch_bounds__(kLossWarps * 32) k_entropy_loss(LossArgs a) {
  __shared__ float2 parts[kLossWarps][33];
  __shared__ float hits[32];
  const int32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.x * 32 + lane;
  int32_t n = -1;
  if (a.rank) {
    pdl_wait();
    if (r < a.N) n = a.rank[r];
  } else {
    // The tiles' kernel lets this one in once the kernels before both have ended: the inputs
    // are there, the tiles' sums are not, nor has it ended that may still read the outputs' memory.
    const int64_t t = r < a.N ? a.targets[r] : -1;
    if (t >= 0 && t < a.V) n = r;
    if (t >= a.V && warp == 0) report(a.status, kErrIndex);
    const int64_t goal = __shfl_sync(0xffffffffu, t, warp);
    if (goal >= 0 && goal < a.V) {
      const uint16_t* h = static_cast<const uint16_t*>(a.hidden) + (int64_t)(blockIdx.x * 32 + warp) * a.hidden_stride;
      const uint16_t* w = static_cast<const uint16_t*>(a.table) + goal * a.table_stride;
      float z = 0.f;
#pragma unroll 4
      for (int32_t k = lane * 8; k < a.D; k += 256) z = dot_eight<T>(load_eight(h, k, a.D), load_eight(w, k, a.D), z);
      z = warp_sum(z);
      if (lane == 0) hits[warp] = z;
    }
    pdl_wait();
  }
  float ref = -INFINITY, sum = 0.f;
  auto join = [&](float2 q) {
    const float next = fmaxf(ref, q.x), base = next == -INFINITY ? 0.f : next;
    sum = sum * ex2(ref - base) + q.y * ex2(q.x - base);
    ref = next;
  };
  if (n >= 0) {
    constexpr int kBatch = 8;
    for (int32_t t = warp; t < a.tiles; t += kLossWarps * kBatch) {
      float2 q[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int32_t at = t + i * kLossWarps;
        q[i] = at < a.tiles ? a.partial[(int64_t)at * a.cap + n] : make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) join(q[i]);
    }
  }
  parts[warp][lane] = make_float2(ref, sum);
  __syncthreads();
  // warp w joins the 32 parts of row w
  const float2 q = parts[lane][warp];
  const float top = warp_max(q.x), base = top == -INFINITY ? 0.f : top;
  const float all = warp_sum(q.y * ex2(q.x - base));
  __syncthreads();
  if (lane == 0) parts[0][warp] = make_float2(top, all);
  __syncthreads();
  if (warp > 0 || r >= a.N) return;
  if (n < 0) {
    a.loss[r] = 0.f;
    if (a.lse) a.lse[r] = 0.f;
    return;
  }
  const float z = a.rank ? a.at_target[n] : hits[lane];
  ref = parts[0][lane].x, sum = parts[0][lane].y;
  const float next = fmaxf(ref, z * kLog2e), from = next == -INFINITY ? 0.f : next;
  sum = sum * ex2(ref - from) + ex2(fmaf(z, kLog2e, -from));
  const float log_sum = log2f(sum), loss = (fmaf(-z, kLog2e, next) + log_sum) * kLn2;
  a.loss[r] = loss < 0.f ? 0.f : loss;  // its last bits may fall below
  const float lse = (next + log_sum) * kLn2;
  if (a.lse) a.lse[r] = lse;
  if (a.par) a.par[n].x = lse * kLog2e;  // as a backward of its own has it
}

// ---- gradients of a piece of the vocabulary

// Elements that an accumulator of a gradient sums at most. At every 16 elements the tensor cores cut the sum and the
// products towards zero, by 2 to 4 times 2^-24 of the sum (measured; most where all products have one sign), so
// that a sum that grows evenly over n elements lacks up to n / 16 * 2^-23: 2^20 tokens in one accumulator lacked
// 2^-8. So many elements cost an eighth of the output's half step (2^-14 of the sum in fp16, 2^-11 in bf16).
__host__ __device__ constexpr int32_t most_summed(bool fp16) { return fp16 ? 1 << 13 : 1 << 16; }

// dh is summed over the vocabulary in `splits` parts; a part's fp32 sums lie at [part][packed
// row][Dp]. Beside dW, whose tiles fill up the launch: enough parts that every CTA group has
// one when there are few tokens. Alone: as many as leave the last round of the groups fullest (4096
// tokens, 32768 x 4096: 2 parts 3.4 rounds of 4, 95 % full; 1 part 84 %), in two rounds or of
// two parts at most. A part has four stages or more, for its way out and back costs as much (100
// tokens, 5000 x 304, dh alone: 25 us, 33 with single stages), and most_summed() elements or fewer.
struct SplitArgs {
  int32_t d_tiles, Dp;
  bool alone;
  int32_t most;       // parts of four stages in the first piece
  int32_t least;      // parts of most_summed() elements in it
};
template <bool kPair>
using GradShape = Shape<kPair, kPair ? 256 : 128, 4096>;
template <bool kPair>
__host__ __device__ inline int32_t splits_of(const SplitArgs& a, int32_t count, int32_t groups) {
  const int32_t tiles = (count + GradShape<kPair>::kRows - 1) / GradShape<kPair>::kRows * a.d_tiles;
  if (tiles == 0) return 1;
  int32_t best = (groups + 2 * tiles - 1) / (2 * tiles);
  if (a.alone) {  // the most parts of one round, of two, or one part and two
    const int32_t one = tiles < groups ? groups / tiles : 1, two = tiles < groups ? 2 * groups / tiles : 2;
    const int32_t one_rounds = (one * tiles + groups - 1) / groups, two_rounds = (two * tiles + groups - 1) / groups;
    best = two * one_rounds > one * two_rounds ? two : one;
  }
  if (best < a.least) best = a.least;
  return best < a.most ? best : a.most;
}

struct GradArgs {
  const int32_t* count;
  int32_t second;  // as in LogitArgs
  int32_t D, V0, V1;
  bool want_h, want_t, first, wide;
  SplitArgs split;
  float* acc;
  void* dtable;
  int64_t dtable_stride;
  const float* scale;
  uint32_t* status;
};

// The long sums (dh) come first, one or more a group; groups that have one fewer take
// as many more tiles of dW first as that sum is long, the rest goes round. kLong: dW alone, from sums over
// more than most_summed() tokens, added up in registers. (With dh's tiles among them, whose way out takes the
// registers that hold the sums: 70000 tokens of 8000 x 4096 bf16 18.5 ms, 6.3 apart.)
template <typename T, bool kPair, bool kLong>
struct Grads {
  static constexpr int kChunk = kLong ? most_summed(std::is_same<T, __half>::value) / kDepth : 0;
  using Args = GradArgs;
  using S = GradShape<kPair>;
  static constexpr int32_t kCols = S::kCols;
  const Args& a;
  int32_t count, group, groups;
  int32_t pad, splits, tiles_h, units_h, kh, kw;
  int32_t tiles_w, early, at, rest;
  // the current tile
  bool over_tokens;  // dW: the sum runs over the tokens
  int32_t row0, col0, k0, k1, part;
  int phase = 0;
  __device__ Grads(const Args& args, int32_t group_, int32_t groups_) : a(args), group(group_), groups(groups_) {
    count = rows_of_g(*a.count, a.second);
    pad = (count + S::kRows - 1) / S::kRows * S::kRows;
    splits = splits_of<kPair>(a.split, count, groups);
    tiles_h = !kLong && a.want_h ? pad / S::kRows * a.split.d_tiles : 0;
    units_h = tiles_h * splits;
    kh = (a.V1 - a.V0 + kDepth - 1) / kDepth, kw = (count + kDepth - 1) / kDepth;
    tiles_w = a.want_t ? (a.V1 - a.V0 + S::kRows - 1) / S::kRows * a.split.d_tiles : 0;
    rest = units_h % groups;
    const int64_t extra = rest ? (kh / splits) / (kw + 4) : 0;  // 4: a tile's own cost, in stages
    early = (int32_t)min(extra * (groups - rest), (int64_t)tiles_w);
    at = group - groups;
  }
  __device__ void to_tile(uint32_t t) {
    const uint32_t m = t / (uint32_t)a.split.d_tiles;
    row0 = (int32_t)m * S::kRows, col0 = (int32_t)(t - m * a.split.d_tiles) * kCols;
  }
  __device__ bool next() {
    while (phase == 0) {
      at += groups;
      if (at >= units_h) {
        phase = 1, at = (group < rest ? early : group - rest) - (groups - rest);
        break;
      }
      over_tokens = false;
      part = at / tiles_h;
      const int32_t t = at - part * tiles_h;
      to_tile(t);
      k0 = (uint32_t)kh * part / splits, k1 = (uint32_t)kh * (part + 1) / splits;  // 2^14 stages, 2^9 parts at most
      if (k0 < k1 || a.first) return true;  // else a part that a short last piece leaves empty
    }
    at += phase == 1 ? groups - rest : groups;
    if (phase == 1 && at >= early) phase = 2, at = early + group;
    if (at >= tiles_w) return false;
    over_tokens = true;
    to_tile(at);
    k0 = 0, k1 = kw;
    return true;
  }
  __device__ int32_t k_stages() const { return k1 - k0; }
  // The last tile of a row of D columns is as narrow as MMAs go: 32 columns a pair.
  __device__ int32_t width() const {
    constexpr int32_t unit = 16 * S::kCtas;
    return min(kCols, (a.D - col0 + unit - 1) / unit * unit);
  }
  __device__ int32_t boxes() const { return (width() / (int32_t)S::kCtas + 63) / 64; }  // of B, 64 columns each
  __device__ uint32_t stage_bytes() const { return S::kA + boxes() * 8192; }
  // maps: a = G, b = the packed hidden states, c = the table, all in boxes of 64 x 64
  __device__ void load(const Maps& maps, int32_t k, uint32_t base, uint32_t bar, uint32_t rank) const {
    const int32_t kk = (k0 + k) * kDepth, r = row0 + (int32_t)rank * 128, c = col0 + (int32_t)rank * (width() / (int32_t)S::kCtas);
    const int32_t n = boxes();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      tensor_load<kPair>(base + i * 8192, &maps.a, over_tokens ? r + i * 64 : kk, over_tokens ? kk : r + i * 64, bar);
#pragma unroll
    for (int i = 0; i < S::kWidth / 64; ++i)
      if (i < n)
        tensor_load<kPair>(base + S::kA + i * 8192, over_tokens ? &maps.b : &maps.c, c + i * 64, over_tokens ? kk : a.V0 + kk,
                           bar);
  }
  __device__ uint64_t a_desc(uint32_t at) const { return over_tokens ? across_desc(at, 8192) : operand_desc(at); }
  __device__ uint64_t b_desc(uint32_t at) const { return across_desc(at, 8192); }
  __device__ uint32_t a_step() const { return over_tokens ? 128 : 2; }  // 16 rows of 128 bytes, or 32 bytes
  __device__ uint32_t b_step() const { return 128; }
  __device__ uint32_t idesc() const { return idesc16<T>(S::kRows, width()) | (over_tokens ? 1u << 15 : 0u) | 1u << 16; }

  // A lane's row of the tile, in the output of that row, and columns of the tile that there are.
  __device__ int32_t row_of(uint32_t warp, uint32_t lane, uint32_t rank) const { return row0 + (int32_t)(rank * 128 + warp * 32 + lane); }
  __device__ int32_t cols() const { return min(kCols, (over_tokens ? a.D : a.split.Dp) - col0); }
  // Columns c..c+63 of the tile.
  __device__ void leave(const Maps& maps, float (&v)[2][32], int32_t row, int32_t c, uint32_t lane, uint8_t* aside) const {
    if (!kLong && !over_tokens) {  // Dp is a multiple of 64
      float* acc = a.acc + ((int64_t)part * pad + row) * a.split.Dp + col0 + c;
#pragma unroll
      for (int i = 0; i < 64; i += 4) {
        float4* at = reinterpret_cast<float4*>(acc + i);
        const float* e = &v[i / 32][i % 32];
        float4 x = make_float4(e[0], e[1], e[2], e[3]);
        if (!a.first) {
          const float4 y = *at;
          x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
        *at = x;
      }
      return;
    }
    const float back = a.scale[1];
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i / 32][i % 32] *= back;
    const int64_t first = a.V0 + row - (int32_t)lane;
    if (a.wide)
      store_box<T>(&maps.out, col0 + c, (int32_t)first, aside, lane, v);
    else
      store_box_plain<T>(static_cast<uint16_t*>(a.dtable) + first * a.dtable_stride + col0 + c, a.dtable_stride,
                         a.V1 - (int32_t)first, cols() - c, aside, lane, v);
  }
  __device__ void store(const Maps& maps, uint32_t tmem, uint32_t warp, uint32_t lane, uint32_t rank, uint8_t* aside, bool ok,
                        bool zero) const {
    const int32_t row = row_of(warp, lane, rank), there = cols();
#pragma unroll 1
    for (int32_t c = 0; c < there; c += 64) {
      float v[2][32];
      __syncwarp();
      if (ok) {
        tmem_load32(tmem + c, v[0]);
        tmem_load32(tmem + c + 32, v[1]);
        tmem_load_wait();
      } else {
#pragma unroll
        for (int i = 0; i < 64; ++i) v[i / 32][i % 32] = zero ? 0.f : NAN;
      }
      leave(maps, v, row, c, lane, aside);
    }
  }
  // Half of the tile's columns, from registers.
  __device__ void finish(const Maps& maps, float (&v)[kCols / 2], uint32_t group, uint32_t warp, uint32_t lane, uint32_t rank,
                         uint8_t* aside, bool ok) const {
    const int32_t row = row_of(warp, lane, rank), first = (int32_t)group * (kCols / 2), there = cols();
#pragma unroll
    for (int c = 0; c < kCols / 2; c += 64) {
      if (first + c >= there) continue;
      float (&x)[2][32] = *reinterpret_cast<float (*)[2][32]>(v + c);
      if (!ok) {
#pragma unroll
        for (int i = 0; i < 64; ++i) x[i / 32][i % 32] = NAN;
      }
      leave(maps, x, row, first + c, lane, aside);
    }
  }
};

struct FinishArgs {
  int32_t N, D;
  const int32_t* rank;
  const int32_t* count;
  int32_t second;
  SplitArgs split;
  int32_t groups;
  const float* acc;
  const float* scale;
  void* out;
  int64_t out_stride;
};

// dh of every row: the parts added in order, zero for rows that take no part. A block for 1024
// columns of a row: the parts of 64 tokens of 4096 take 7 us, and 16 with a block for 4096. A
// narrow row's parts are shared out among teams of lanes (16 tokens of 64: 4 us, 27 without).
template <typename T, bool kPair>
__global__ void __launch_bounds__(kThreads) k_entropy_finish(FinishArgs a) {
  pdl_wait();
  const int32_t r = blockIdx.x, n = a.rank[r], count = rows_of_g(*a.count, a.second);
  constexpr int32_t kRows = GradShape<kPair>::kRows;
  const int32_t pad = (count + kRows - 1) / kRows * kRows;
  const int32_t splits = splits_of<kPair>(a.split, count, a.groups), parts = a.second ? 2 * splits : splits;
  const int64_t stride = (int64_t)pad * a.split.Dp, second = (int64_t)a.second * a.split.Dp;
  const float back = a.scale[1];
  T* out = static_cast<T*>(a.out) + (int64_t)r * a.out_stride;
  const bool wide = reinterpret_cast<uintptr_t>(out) % 8 == 0;
  // a team of lanes has every teams-th part
  int32_t lanes = kThreads;
  while (lanes > 16 && lanes * 2 >= a.D) lanes /= 2;
  const int32_t team = (int32_t)threadIdx.x / lanes, teams = kThreads / lanes;
  const int32_t lane = (int32_t)threadIdx.x - team * lanes;
  __shared__ float4 of_team[kThreads];
  const int32_t d = ((int32_t)blockIdx.y * lanes + lane) * 4;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float4 y) { x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w); };
  if (n >= 0 && d < a.D) {
    const float* at = a.acc + (int64_t)n * a.split.Dp + d;
#pragma unroll 8
    for (int32_t s = team; s < parts; s += teams)
      add(*reinterpret_cast<const float4*>(at + (s < splits ? s * stride : (s - splits) * stride + second)));
  }
  if (teams > 1) {  // one block holds all of D then
    of_team[threadIdx.x] = x;
    __syncthreads();
    if (team > 0) return;
    for (int32_t t = 1; t < teams; ++t) add(of_team[t * lanes + lane]);
  }
  const float v[4] = {x.x * back, x.y * back, x.z * back, x.w * back};
  if (wide && d + 4 <= a.D) {
    *reinterpret_cast<uint2*>(out + d) = make_uint2(two<T>(v[0], v[1]), two<T>(v[2], v[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (d + i < a.D) out[d + i] = Elem<T>::put(v[i]);
  }
}

// ---- host side

struct Layout {
  int64_t cap, Dp, piece, count, scale, rank, target, par, rows, table, partial, at_target, g, acc, total;
  int32_t groups, d_tiles, v_tiles, cols, second;
  bool pair, padded;
};

// Whether TMA can read (or write) rows of D 16-bit elements. What lies beyond a row it leaves out
// by 16 bytes, not by elements.
bool readable(const void* rows, int64_t stride, int64_t n, int32_t D) {
  return D % 8 == 0 && aligned(rows, 16) && (n == 1 || stride % 8 == 0);
}

// Columns of a tile of logits, a multiple of `unit`: as few as still take no more rounds of the
// CTA groups than 256 would, so that the last round is nearly full.
int32_t tile_columns(int64_t N, int32_t V, bool pair, int32_t groups, int32_t unit) {
  const int64_t m = pair ? (N + 255) / 256 : 1, rounds = (m * ((V + 255) / 256) + groups - 1) / groups;
  const int64_t tiles = rounds * groups / m;  // at most
  const int64_t cols = ((V + tiles - 1) / tiles + unit - 1) / unit * unit;
  return cols < 256 ? (int32_t)cols : 256;
}

Layout layout(int device, int64_t N, int32_t V, int32_t D, const void* table, int64_t stride, int gradients, bool fp16) {
  Layout l{};
  l.cap = N > 0 ? (N + 255) / 256 * 256 : 256;
  l.Dp = (D + 63) / 64 * 64;  // whole lines: boxes of 128 bytes that straddle them cost twice
  // up to 64 tokens G has a second part, in the rows that they leave of a tile
  l.second = gradients && N <= 64 ? (N <= 32 ? 32 : 64) : 0;
  l.pair = N > 128;
  l.groups = sm_count(device) / (l.pair ? 2 : 1);
  if (l.groups < 1) l.groups = 1;
  const int32_t cols = l.pair ? GradShape<true>::kCols : GradShape<false>::kCols;
  l.d_tiles = (D + cols - 1) / cols;
  l.cols = tile_columns(N, V, l.pair, l.groups, l.pair ? 32 : 16);
  l.v_tiles = (V + l.cols - 1) / l.cols;
  l.padded = !readable(table, stride, V, D);
  // A piece's G, and (fp16, of whose sums there are more) half as much for the parts of dh, two at least.
  const int64_t rows = l.pair ? 256 : 128, m = N > 0 ? (N + rows - 1) / rows : 1, part = m * rows * l.Dp * 4;
  const int64_t whole = (int64_t)(V + 255) / 256, fit = kPieceBytes / 2 / part;
  int64_t most = kPieceBytes / (l.cap * 2 * 256);
  if (fp16 && most > (fit > 2 ? fit : 2) * (most_summed(true) / 256)) most = (fit > 2 ? fit : 2) * (most_summed(true) / 256);
  const int64_t pieces = most < 1 ? whole : (whole + most - 1) / most;
  l.piece = (whole + pieces - 1) / pieces * 256;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  l.count = take(4), l.scale = take(8);
  l.rank = take(N * 4), l.target = take(l.cap * 4), l.par = take(l.cap * 8);
  l.rows = take(l.cap * l.Dp * 2);
  l.table = l.padded ? take((int64_t)V * l.Dp * 2) : 0;
  l.partial = take((int64_t)l.v_tiles * 2 * l.cap * 8), l.at_target = take(l.cap * 4);
  if (gradients) {
    l.g = take(l.cap * l.piece * 2);
    // parts of dh: what splits_of() gives, for any number of packed rows
    const int64_t few = (2 * (int64_t)l.groups + l.d_tiles - 1) / l.d_tiles * (rows * l.Dp * 4);
    const int64_t first = V < l.piece ? V : l.piece, parts = (first + most_summed(fp16) - 1) / most_summed(fp16);
    const int64_t long_sums = (parts > 2 ? parts : 2) * part;
    l.acc = take(few > long_sums ? few : long_sums);
  }
  l.total = at;
  return l;
}

struct Call {
  int device;
  const void* hidden;
  emb_dtype dtype;
  int64_t hidden_stride, N;
  const void* table;
  int64_t table_stride;
  int32_t V, D;
  const int64_t* targets;
  const float *lse, *weight;
  float *loss, *lse_out;
  void* dhidden;
  int64_t dhidden_stride;
  void* dtable;
  int64_t dtable_stride;
  uint8_t* workspace;
  uint32_t* status;
  cudaStream_t s;
};

template <typename Policy, bool kPair>
cudaError_t launch_mm(int device, int32_t groups, const Maps& maps, const typename Policy::Args& args, cudaStream_t s) {
  constexpr uint32_t smem = Policy::S::kSmem;
  const void* fn = reinterpret_cast<const void*>(&k_entropy_mm<Policy, kPair>);
  static bool ready[64];
  const cudaError_t e = allow_smem(fn, smem, device, ready);
  if (e != cudaSuccess) return e;
  void* p[] = {const_cast<Maps*>(&maps), const_cast<typename Policy::Args*>(&args)};
  return kPair ? launch_clusters(fn, dim3(groups * 2), dim3(kMmThreads), 2, smem, s, p, true)
               : launch_kernel(fn, dim3(groups), dim3(kMmThreads), smem, s, p, true);
}

template <typename T, bool kPair>
cudaError_t run(const Call& c, const Layout& l) {
  uint8_t* w = c.workspace;
  const int32_t N = (int32_t)c.N, Dp = (int32_t)l.Dp;
  int32_t* count = reinterpret_cast<int32_t*>(w + l.count);
  float* scale = reinterpret_cast<float*>(w + l.scale);
  int32_t *rank = reinterpret_cast<int32_t*>(w + l.rank), *target = reinterpret_cast<int32_t*>(w + l.target);
  float2* par = reinterpret_cast<float2*>(w + l.par);
  float2* partial = reinterpret_cast<float2*>(w + l.partial);
  float* at_target = reinterpret_cast<float*>(w + l.at_target);
  const bool gradients = c.dhidden || c.dtable;
  cudaError_t e = cudaSuccess;

  // The losses of few tokens need no packing: a row that takes no part is one more row of the tile.
  const bool direct = !gradients && !kPair && readable(c.hidden, c.hidden_stride, N, c.D);
  // two blocks an SM and more, up to eight rows each; 1024 blocks at most, for each scans all targets
  const int32_t two = 2 * sm_count(c.device), per_block = N / 1024 > 8 ? N / 1024 : N < two ? 1 : N < 2 * two ? 2 : N < 4 * two ? 4 : 8;
  RowArgs rows{c.hidden, c.hidden_stride, N, c.D, c.V, c.targets, c.weight, c.lse,
               reinterpret_cast<uint16_t*>(w + l.rows), Dp, per_block, gradients, l.second,
               gradients && std::is_same<T, __half>::value, count, rank, c.table, c.table_stride, target, at_target, par, scale,
               c.status};
  void* rows_p[] = {&rows};
  int32_t blocks = (N + per_block - 1) / per_block;
  if (gradients && blocks < 64) blocks = 64;  // they share out the zeros
  if (!direct)
    e = launch_kernel(reinterpret_cast<const void*>(&k_entropy_rows<T>), dim3(blocks), dim3(kThreads), 0, c.s, rows_p, true);
  if (e != cudaSuccess) return e;
  const void* table = c.table;
  int64_t stride = c.V == 1 ? l.Dp : c.table_stride;  // one row: any stride
  if (l.padded) {
    const uint16_t* from = static_cast<const uint16_t*>(c.table);
    uint16_t* to = reinterpret_cast<uint16_t*>(w + l.table);
    int64_t from_stride = c.table_stride;
    int32_t V = c.V, D = c.D, pad = Dp;
    void* p[] = {&from, &from_stride, &to, &V, &D, &pad};
    e = launch_kernel(reinterpret_cast<const void*>(&k_entropy_pad), dim3((V + kWarps - 1) / kWarps), dim3(kThreads), 0, c.s,
                      p, true);
    if (e != cudaSuccess) return e;
    table = to, stride = l.Dp;
  }
  // Few tokens: only their rows are brought. What the tile's other rows hold stays in them.
  // (Rows beyond the end of a map are brought as zeros, but slowly: 232 us instead of 171 for
  // one token against 128256 x 4096.)
  const int32_t a_rows = l.second ? 2 * l.second : N < 128 ? N : 128;
  Maps logit_maps, grad_maps;
  e = direct ? half_matrix_map(&logit_maps.a, c.hidden, N, c.D, N == 1 ? l.Dp : c.hidden_stride, a_rows)
             : half_matrix_map(&logit_maps.a, w + l.rows, l.cap, l.Dp, l.Dp, a_rows);
  if (e == cudaSuccess) e = half_matrix_map(&logit_maps.b, table, c.V, l.padded ? l.Dp : c.D, stride, l.cols / (kPair ? 2 : 1));
  if (e != cudaSuccess) return e;
  logit_maps.c = logit_maps.out = logit_maps.b;
  LogitArgs la{direct ? nullptr : count, N, direct ? c.targets : nullptr, c.D, 0, c.V, a_rows, l.second, l.cols, target, partial, l.cap,
               at_target, par, c.status};
  if (c.loss) {
    const bool wide = c.D > kDepth * Logits<T, kPair, kLongSums>::kChunk;
    e = wide ? launch_mm<Logits<T, kPair, kLongSums>, kPair>(c.device, l.groups, logit_maps, la, c.s)
             : launch_mm<Logits<T, kPair, kSums>, kPair>(c.device, l.groups, logit_maps, la, c.s);
    if (e != cudaSuccess) return e;
    LossArgs loss{N, l.v_tiles * (wide ? 2 : 1), c.V, c.D, direct ? nullptr : rank, partial, l.cap, at_target, c.hidden, c.table,
                  c.hidden_stride, c.table_stride, c.targets, c.loss, c.lse_out, gradients ? par : nullptr, c.status};
    void* p[] = {&loss};
    e = launch_kernel(reinterpret_cast<const void*>(&k_entropy_loss<T>), dim3((N + 31) / 32), dim3(kLossWarps * 32), 0, c.s, p,
                      true);
    if (e != cudaSuccess) return e;
  }
  if (!gradients) return cudaSuccess;
  const bool wide = c.dtable && readable(c.dtable, c.dtable_stride, c.V, c.D);
  e = half_matrix_map(&logit_maps.out, w + l.g, l.cap, l.piece, l.piece, 32);
  if (e == cudaSuccess) e = half_matrix_map(&grad_maps.a, w + l.g, l.cap, l.piece, l.piece, 64);
  if (e == cudaSuccess) e = half_matrix_map(&grad_maps.b, w + l.rows, l.cap, l.Dp, l.Dp, 64);
  if (e == cudaSuccess) e = half_matrix_map(&grad_maps.c, table, c.V, l.padded ? l.Dp : c.D, stride, 64);
  grad_maps.out = grad_maps.c;
  if (e == cudaSuccess && wide)
    e = half_matrix_map(&grad_maps.out, c.dtable, c.V, c.D, c.V == 1 ? l.Dp : c.dtable_stride, 32);
  if (e != cudaSuccess) return e;
  const int64_t first = c.V < l.piece ? c.V : l.piece;
  constexpr bool kHalf = std::is_same<T, __half>::value;
  const bool apart = c.dtable && N > most_summed(kHalf);  // dW in a launch of its own
  const SplitArgs split{l.d_tiles, Dp, !c.dtable || apart, (int32_t)((first + 4 * kDepth - 1) / (4 * kDepth)),
                        (int32_t)((first + most_summed(kHalf) - 1) / most_summed(kHalf))};
  GradArgs ga{count, l.second, c.D, 0, 0, c.dhidden != nullptr, c.dtable != nullptr, true, wide, split,
              reinterpret_cast<float*>(w + l.acc), c.dtable, c.dtable_stride, scale, c.status};
  // G leaves in boxes of 64 columns
  la.cols = tile_columns(c.N, c.V < l.piece ? c.V : (int32_t)l.piece, kPair, l.groups, 64);
  e = half_matrix_map(&logit_maps.b, table, c.V, l.padded ? l.Dp : c.D, stride, la.cols / (kPair ? 2 : 1));
  if (e != cudaSuccess) return e;
  for (int64_t v = 0; v < c.V; v += l.piece) {
    la.V0 = ga.V0 = (int32_t)v;
    la.V1 = ga.V1 = (int32_t)(v + l.piece < c.V ? v + l.piece : c.V);
    ga.first = v == 0;
    if constexpr (kHalf)
      e = c.D > kMostPlain ? launch_mm<Logits<T, kPair, kLongGradient>, kPair>(c.device, l.groups, logit_maps, la, c.s)
                           : launch_mm<Logits<T, kPair, kGradient>, kPair>(c.device, l.groups, logit_maps, la, c.s);
    else
      e = launch_mm<Logits<T, kPair, kGradient>, kPair>(c.device, l.groups, logit_maps, la, c.s);
    if (e != cudaSuccess) return e;
    if constexpr (kPair) {
      if (apart) {
        e = launch_mm<Grads<T, true, true>, true>(c.device, l.groups, grad_maps, ga, c.s);
        if (e != cudaSuccess) return e;
        if (!c.dhidden) continue;
        ga.want_t = false;
      }
    }
    e = launch_mm<Grads<T, kPair, false>, kPair>(c.device, l.groups, grad_maps, ga, c.s);
    ga.want_t = c.dtable != nullptr;
    if (e != cudaSuccess) return e;
  }
  if (c.dhidden) {
    FinishArgs f{N, c.D, rank, count, l.second, split, l.groups, reinterpret_cast<const float*>(w + l.acc), scale, c.dhidden,
                 c.dhidden_stride};
    void* p[] = {&f};
    e = launch_kernel(reinterpret_cast<const void*>(&k_entropy_finish<T, kPair>), dim3(N, (c.D + 4 * kThreads - 1) / (4 * kThreads)),
                      dim3(kThreads), 0, c.s, p, true);
  }
  return e;
}

bool sizes_ok(int device, int64_t N, int32_t V, int32_t D) {
  return device >= 0 && N >= 0 && N <= kMaxTokens && V >= 1 && V <= kMaxVocab && D >= 1 && D <= kMaxWidth;
}

emb_status cross_entropy(Call c, int64_t workspace_bytes, bool gradients) {
  if (!sizes_ok(c.device, c.N, c.V, c.D) || (c.dtype != EMB_F16 && c.dtype != EMB_BF16)) return EMB_ERR_INVALID_ARG;
  if (!aligned(c.targets, 8) || !aligned(c.lse, 4) || !aligned(c.weight, 4) || !aligned(c.loss, 4) ||
      !aligned(c.lse_out, 4) || !aligned(c.status, 4) || !aligned(c.hidden, 2) || !aligned(c.table, 2) ||
      !aligned(c.dhidden, 2) || !aligned(c.dtable, 2) || !aligned(c.workspace, 256))
    return EMB_ERR_INVALID_ARG;
  // without tokens the table's gradient is still written: zeros
  if (c.N == 0 && !c.dtable) return EMB_OK;
  if ((c.N > 0 && (!c.hidden || !c.targets)) || !c.table || !c.workspace || (c.N > 1 && c.hidden_stride < c.D) ||
      (c.V > 1 && c.table_stride < c.D) || (c.N > 1 && c.dhidden && c.dhidden_stride < c.D) ||
      (c.V > 1 && c.dtable && c.dtable_stride < c.D))
    return EMB_ERR_INVALID_ARG;
  // the table is read until its gradient has been written, and the hidden states with it
  if ((c.dtable && (c.dtable == c.table || c.dtable == c.hidden || c.dtable == c.dhidden)) ||
      (c.dhidden && (c.dhidden == c.table || c.dhidden == c.hidden)))
    return EMB_ERR_INVALID_ARG;
  if (c.V == 1) c.table_stride = c.dtable_stride = c.D;
  const Layout l = layout(c.device, c.N, c.V, c.D, c.table, c.table_stride, gradients, c.dtype == EMB_F16);
  if (workspace_bytes < l.total) return EMB_ERR_INVALID_ARG;
  return on_device(c.device, [&] {
    if (c.N == 0)
      return cudaMemset2DAsync(c.dtable, c.dtable_stride * 2, 0, (size_t)c.D * 2, c.V, c.s);
    if (c.dtype == EMB_F16) return l.pair ? run<__half, true>(c, l) : run<__half, false>(c, l);
    return l.pair ? run<__nv_bfloat16, true>(c, l) : run<__nv_bfloat16, false>(c, l);
  });
}

}  // namespace
}  // namespace embbwd

using namespace embbwd;

extern "C" int64_t emb_cross_entropy_workspace(int device, int64_t N, int32_t V, int32_t D, const void* table,
                                               int64_t table_stride, int gradients) {
  if (!sizes_ok(device, N, V, D)) return -1;
  const int64_t fp16 = layout(device, N, V, D, table, table_stride, gradients, true).total;
  const int64_t bf16 = layout(device, N, V, D, table, table_stride, gradients, false).total;
  return fp16 > bf16 ? fp16 : bf16;
}

extern "C" emb_status emb_cross_entropy_forward(int device, const void* hidden, emb_dtype dtype, int64_t hidden_stride,
                                                int64_t N, const void* table, int64_t table_stride, int32_t V, int32_t D,
                                                const int64_t* targets, float* loss, float* lse, void* workspace,
                                                int64_t workspace_bytes, uint32_t* device_status, void* stream) {
  if (N > 0 && !loss) return EMB_ERR_INVALID_ARG;
  return cross_entropy({device, hidden, dtype, hidden_stride, N, table, table_stride, V, D, targets, nullptr, nullptr, loss,
                        lse, nullptr, 0, nullptr, 0, static_cast<uint8_t*>(workspace), device_status,
                        static_cast<cudaStream_t>(stream)},
                       workspace_bytes, false);
}

extern "C" emb_status emb_cross_entropy_backward(int device, const void* hidden, emb_dtype dtype, int64_t hidden_stride,
                                                 int64_t N, const void* table, int64_t table_stride, int32_t V, int32_t D,
                                                 const int64_t* targets, const float* lse, const float* row_weight,
                                                 void* grad_hidden, int64_t grad_hidden_stride, void* grad_table,
                                                 int64_t grad_table_stride, void* workspace, int64_t workspace_bytes,
                                                 uint32_t* device_status, void* stream) {
  if ((N > 0 && !lse) || (!grad_hidden && !grad_table)) return EMB_ERR_INVALID_ARG;
  return cross_entropy({device, hidden, dtype, hidden_stride, N, table, table_stride, V, D, targets, lse, row_weight, nullptr,
                        nullptr, grad_hidden, grad_hidden_stride, grad_table, grad_table_stride,
                        static_cast<uint8_t*>(workspace), device_status, static_cast<cudaStream_t>(stream)},
                       workspace_bytes, true);
}

extern "C" emb_status emb_cross_entropy_step(int device, const void* hidden, emb_dtype dtype, int64_t hidden_stride,
                                             int64_t N, const void* table, int64_t table_stride, int32_t V, int32_t D,
                                             const int64_t* targets, const float* row_weight, float* loss,
                                             void* grad_hidden, int64_t grad_hidden_stride, void* grad_table,
                                             int64_t grad_table_stride, void* workspace, int64_t workspace_bytes,
                                             uint32_t* device_status, void* stream) {
  if ((N > 0 && !loss) || (!grad_hidden && !grad_table)) return EMB_ERR_INVALID_ARG;
  return cross_entropy({device, hidden, dtype, hidden_stride, N, table, table_stride, V, D, targets, nullptr, row_weight, loss,
                        nullptr, grad_hidden, grad_hidden_stride, grad_table, grad_table_stride,
                        static_cast<uint8_t*>(workspace), device_status, static_cast<cudaStream_t>(stream)},
                       workspace_bytes, true);
}
