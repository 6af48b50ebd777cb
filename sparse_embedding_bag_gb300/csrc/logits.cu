// Logits before a token is chosen: penalties for repeated tokens, biases and a
// grammar mask, for a batch of requests with ragged histories.
//
// For token v of request b, with z the logit, c the times v is in the request's
// output and "seen" true if it is in its prompt or output:
//   y = seen ? (z > 0 ? z / rep_b : z * rep_b) : z
//   y = y - freq_b * c - pres_b * [c > 0] + (sum of the biases of v)
//   y = -inf where bit v % 32 of mask word v / 32 is clear
//
// A block takes a slice of one request's vocabulary. It counts the tokens of its slice in
// the request's history in shared memory (integer atomics, so that their order does not
// matter). Then it passes over its slice once, eight tokens a thread and step, whose first
// loads went out before the counting; last come the biased tokens, which the pass left
// alone.
//
// Bound: HBM traffic without lists (512 x 131071 bf16 to bf16: 42 us, 6400 GB/s). With
// histories of 4000 ids 70 us, bound by neither memory nor instructions (DRAM 44 %, issue slots
// 65 %, 24 of 64 warps an SM, most stalls on loads) but by latency: a block has the first
// 8192 tokens of its slice under way while it counts, and asks for the rest after; and every
// slice's block reads the whole history (4 slices a row). Measured and dropped: entries of 32
// bits throughout (half the slice: 85 us), the history shared out over a cluster that counts
// through distributed shared memory (157 us), a second kernel that rewrites only the listed
// tokens from a hash table (123 us: scattered reads and partial sectors from HBM), a list of
// the distinct tokens of a slice (115 us: atomics that return). Outputs beyond 16383 ids
// count in 32 bits and in pieces of half a slice: 64 x 128256 bf16 with 16000 output ids
// 21.6 us, with 20000 42.
#include <algorithm>
#include <cmath>

#include "sm103.cuh"

namespace embbwd {
namespace {

constexpr int kMinSlice = 2048, kMaxSlice = 36 * 1024;  // tokens of a block, a multiple of 1024
constexpr int kLogitThreads = 256, kLogitBlocks = 3;
constexpr int kBatch = 4;                            // steps whose loads are in flight together

struct LogitsArgs {
  const void* z;
  void* y;
  int64_t z_stride, y_stride;
  int32_t B, V;
  const int64_t *p_ids, *p_off, *o_ids, *o_off, *b_ids, *b_off;
  int64_t p_n, o_n, b_n;
  const float *rep, *freq, *pres, *b_val;
  const uint32_t* mask;
  int64_t mask_stride;
  uint32_t* status;
  int32_t slice;
};


// [start, end) of request b's list, empty (and reported) if the offsets are malformed or the
// list is longer than `most`.
__device__ __forceinline__ void list_of(const int64_t* off, int64_t n, int32_t b, uint32_t* status, int64_t* start,
                                        int64_t* end, int64_t most = INT32_MAX) {
  *start = off[b];
  *end = off[b + 1];
  if (*start < 0 || *end < *start || *end > n || *end - *start > most) {
    report(status, kErrOffsets);
    *start = *end = 0;
  }
}

// The request's penalties for a token seen `n` times in the output (0: only in the prompt).
// A division by `repetition` is a multiplication by its reciprocal (one more rounding in
// fp32), and nothing branches: a warp's 256 tokens are rarely all unseen, and a branch for
// each with a division behind it cost 20 us at 512 x 131071.
struct Penalty {
  float rep, inv, freq, pres;
  __device__ __forceinline__ float operator()(float z, bool seen, uint32_t n) const {
    const float y = seen ? z * (z > 0.f ? inv : rep) : z;
    return n ? fmaf(-freq, (float)n, y) - pres : y;
  }
};

// What the lists say of the tokens of a piece of the vocabulary, in shared memory: bits for
// "in the prompt" and "has a bias", and the times in the output. 16 bits a token where the
// output is short enough to be counted in 14 of them, else 32: pieces are twice as large
// with 16, and the history is read once a piece.
template <int kBits>
struct Counts {
  static constexpr uint32_t kPrompt = 1u << (kBits - 1), kBias = 1u << (kBits - 2), kTimes = kBias - 1;
  static constexpr int kWords = kGroup * kBits / 32;  // of a group
  uint32_t at;   // shared memory address of the entries
  uint32_t pad;  // entries before token 0, so that groups are 16-byte aligned
  __device__ __forceinline__ uint32_t address(uint32_t off) const {
    return at + (kBits == 16 ? (off + pad) / 2 : off + pad) * 4;
  }
  __device__ __forceinline__ uint32_t shift(uint32_t off) const { return kBits == 16 ? (off + pad) % 2 * 16 : 0; }
  // Adds to (or sets bits in) a token's entry if off < len. Predicated: a warp's 32 ids
  // rarely miss a piece all together, and a branch around every atomic costs more.
  __device__ __forceinline__ void add(uint32_t off, uint32_t len) const {
    asm volatile("{ .reg .pred p; setp.lt.u32 p, %0, %1; @p red.shared.add.u32 [%2], %3; }" ::"r"(off), "r"(len),
                 "r"(address(off)), "r"(1u << shift(off))
                 : "memory");
  }
  __device__ __forceinline__ void set(uint32_t off, uint32_t len, uint32_t bits) const {
    asm volatile("{ .reg .pred p; setp.lt.u32 p, %0, %1; @p red.shared.or.b32 [%2], %3; }" ::"r"(off), "r"(len),
                 "r"(address(off)), "r"(bits << shift(off))
                 : "memory");
  }
  __device__ __forceinline__ uint32_t word(uint32_t off) const {
    uint32_t w;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(address(off)) : "memory");
    return w;
  }
  __device__ __forceinline__ uint32_t get(uint32_t off) const {
    return kBits == 16 ? word(off) >> shift(off) & 0xffffu : word(off);
  }
  // A group's words; token k of them.
  __device__ __forceinline__ void group(uint32_t off, uint32_t (&w)[kWords]) const {
#pragma unroll
    for (int i = 0; i < kWords; i += 4)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "r"(address(off) + i * 4)
                   : "memory");
  }
  __device__ __forceinline__ static uint32_t of(const uint32_t (&w)[kWords], int k) {
    return kBits == 16 ? (k & 1 ? w[k / 2] >> 16 : w[k / 2] & 0xffffu) : w[k];
  }
};

// Counts the tokens [v0, v0 + len) among `pn` prompt and `on` output ids; returns whether
// an id is outside the vocabulary. An id is compared by its halves: the high one has to be
// 0. The loads of both lists' last pieces (most lists are no longer) go out together.
template <int kBits>
__device__ __forceinline__ bool count_ids(const int64_t* p_ids, int32_t pn, const int64_t* o_ids, int32_t on, uint32_t V,
                                          uint32_t v0, uint32_t len, const Counts<kBits>& counts) {
  constexpr int kAhead = 8;  // ids of a list in flight
  constexpr int32_t kRound = kLogitThreads * kAhead;
  uint32_t high = 0, most = 0;  // over all ids
  auto one = [&](uint2 id, bool output) {
    high |= id.y;
    most = max(most, id.x);
    const uint32_t off = id.y ? 0xffffffffu : id.x - v0;
    if (output)
      counts.add(off, len);
    else
      counts.set(off, len, Counts<kBits>::kPrompt);
  };
  const uint2* p = reinterpret_cast<const uint2*>(p_ids) + threadIdx.x;
  const uint2* o = reinterpret_cast<const uint2*>(o_ids) + threadIdx.x;
  uint2 id[kAhead];
  auto round = [&](const uint2* q, bool output) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) id[k] = __ldg(q + k * kLogitThreads);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) one(id[k], output);
  };
  for (; pn >= kRound; pn -= kRound, p += kRound) round(p, false);
  for (; on >= kRound; on -= kRound, o += kRound) round(o, true);
  uint2 id2[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if ((int)threadIdx.x + k * kLogitThreads < pn) id[k] = __ldg(p + k * kLogitThreads);
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if ((int)threadIdx.x + k * kLogitThreads < on) id2[k] = __ldg(o + k * kLogitThreads);
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if ((int)threadIdx.x + k * kLogitThreads < pn) one(id[k], false);
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if ((int)threadIdx.x + k * kLogitThreads < on) one(id2[k], true);
  return high != 0 || most >= V;
}

// A request's lists: [start, end) in each.
struct Lists {
  int64_t ps, pe, os, oe, bs, be;
};

// Groups of eight start `head` tokens into a piece, so that stores are 16-byte aligned, and
// loads too where input and output allow it together.
template <typename in_t, typename out_t>
__device__ __forceinline__ int32_t head_of(const in_t* z, const out_t* y, int32_t len, bool* wide_loads) {
  constexpr uint32_t in_n = 16 / sizeof(in_t), out_n = 16 / sizeof(out_t), both_n = in_n < out_n ? in_n : out_n;
  const uint32_t in_at = (uint32_t)(reinterpret_cast<uintptr_t>(z) / sizeof(in_t)) % in_n;
  const uint32_t out_at = (uint32_t)(reinterpret_cast<uintptr_t>(y) / sizeof(out_t)) % out_n;
  *wide_loads = in_at % both_n == out_at % both_n;
  return min(len, (int32_t)(*wide_loads && in_n > out_n ? -in_at % in_n : -out_at % out_n));
}

// The biased tokens of a piece where the list names one twice. A warp takes 512 of the piece's
// tokens at a time, a lane 16 of them, and goes over the list: every token's biases add in
// list order, and the work is (tokens of the piece / 4096) times the list's length.
template <typename in_t, typename out_t, int kBits>
__device__ __forceinline__ void add_biases(const LogitsArgs& a, int32_t b, int32_t v0, int32_t len, const Lists& l,
                                           const Penalty& penalty, const uint32_t* smem) {
  using C = Counts<kBits>;
  const in_t* z = static_cast<const in_t*>(a.z) + b * a.z_stride + v0;
  out_t* y = static_cast<out_t*>(a.y) + b * a.y_stride + v0;
  const uint32_t* mask = a.mask ? a.mask + b * a.mask_stride : nullptr;
  bool wide_loads;
  const C counts{smem_u32(smem), (uint32_t)(-head_of(z, y, len, &wide_loads) & 7)};
  constexpr int kOwn = 16, kAhead = 4;  // a lane's tokens, its entries in flight
  constexpr int32_t kWindow = kOwn * 32;
  const int32_t lane = threadIdx.x & 31;
  for (int32_t at = (threadIdx.x >> 5) * kWindow; at < len; at += kLogitThreads / 32 * kWindow) {
    float sum[kOwn];
    uint32_t mine = 0;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      const int32_t off = at + k * 32 + lane;
      const uint32_t c = off < len ? counts.get(off) : 0;
      sum[k] = 0.f;
      if (c & C::kBias) sum[k] = penalty(Elem<in_t>::get(z[off]), c & ~C::kBias, c & C::kTimes), mine |= 1u << k;
    }
    if (!__any_sync(0xffffffffu, mine)) continue;
    const int64_t first = (int64_t)v0 + at, count = min(kWindow, len - at);
    for (int64_t j0 = l.bs; j0 < l.be; j0 += 32 * kAhead) {
      int64_t token[kAhead];
      float bias[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t j = j0 + i * 32 + lane;
        token[i] = j < l.be ? a.b_ids[j] : -1;
        bias[i] = j < l.be ? a.b_val[j] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t o = token[i] - first;
        for (uint32_t here = __ballot_sync(0xffffffffu, o >= 0 && o < count); here; here &= here - 1) {
          const int from = __ffs(here) - 1;
          const int32_t off = __shfl_sync(0xffffffffu, (int32_t)o, from);
          const float x = __shfl_sync(0xffffffffu, bias[i], from);
          if (off % 32 != lane) continue;
#pragma unroll
          for (int k = 0; k < kOwn; ++k)
            if (off / 32 == k) sum[k] += x;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kOwn; ++k)
      if (mine >> k & 1u) {
        const int32_t off = at + k * 32 + lane;
        const uint32_t v = v0 + off;
        y[off] = Elem<out_t>::put(!mask || (mask[v >> 5] >> (v & 31) & 1u) ? sum[k] : -INFINITY);
      }
  }
}

// Tokens [v0, v0 + len) of request b. kBits 0: there are no lists.
template <typename in_t, typename out_t, int kBits>
__device__ __forceinline__ void process(const LogitsArgs& a, int32_t b, int32_t v0, int32_t len, const Lists& l,
                                        const Penalty& penalty, uint32_t* smem, int* repeated) {
  using C = Counts<kBits ? kBits : 32>;
  const in_t* z = static_cast<const in_t*>(a.z) + b * a.z_stride + v0;
  out_t* y = static_cast<out_t*>(a.y) + b * a.y_stride + v0;
  bool wide_loads;
  const int32_t head = head_of(z, y, len, &wide_loads);
  const int32_t groups = (len - head) / kGroup;
  const C counts{smem_u32(smem), (uint32_t)(-head & 7)};
  const uint32_t* mask = a.mask ? a.mask + b * a.mask_stride : nullptr;
  auto allowed = [&](uint32_t v) { return !mask || (mask[v >> 5] >> (v & 31) & 1u); };
  auto penalised = [&](float x, uint32_t c) { return penalty(x, c & ~C::kBias, c & C::kTimes); };
  // kBatch groups a thread are in flight; the first go out before the lists are read.
  const in_t* zg = z + head;
  out_t* yg = y + head;
  Raw8<in_t> raw[kBatch];
  uint2 words[kBatch];
  auto load = [&](int u, int32_t i) {
    if (i >= groups) return;
    if (wide_loads) raw[u].load(zg + i * kGroup);
    if (mask) {
      const int32_t v = v0 + head + i * kGroup;
      words[u].x = mask[v >> 5];
      words[u].y = mask[(v + kGroup - 1) >> 5];
    }
  };
#pragma unroll
  for (int u = 0; u < kBatch; ++u) load(u, threadIdx.x + u * kLogitThreads);
  // a thread's first bias: its token, logit and value, ahead of their use
  int64_t own_id = -1;
  float own_z = 0.f, own_bias = 0.f;
  if (kBits && l.bs + threadIdx.x < l.be) {
    own_id = a.b_ids[l.bs + threadIdx.x];
    own_bias = a.b_val[l.bs + threadIdx.x];
  }
  if (kBits) {
    uint4* c4 = reinterpret_cast<uint4*>(smem);
    for (int32_t i = threadIdx.x; i < (len + kGroup) * C::kWords / (4 * kGroup) + 1; i += kLogitThreads)
      c4[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) *repeated = 0;
    __syncthreads();
    bool bad = count_ids(a.p_ids + l.ps, (int32_t)(l.pe - l.ps), a.o_ids + l.os, (int32_t)(l.oe - l.os), a.V, v0, len,
                         counts);
    for (int64_t j = l.bs + threadIdx.x; j < l.be; j += kLogitThreads) {
      const int64_t v = j == l.bs + threadIdx.x ? own_id : a.b_ids[j];
      bad |= v < 0 || v >= a.V;
      if (v < v0 || v >= v0 + len) continue;
      const uint32_t off = (uint32_t)(v - v0), bit = C::kBias << counts.shift(off);
      uint32_t old;
      asm volatile("atom.shared.or.b32 %0, [%1], %2;" : "=r"(old) : "r"(counts.address(off)), "r"(bit) : "memory");
      if (old & bit) *repeated = 1;
    }
    if (bad) report(a.status, kErrIndex);
    if (own_id >= v0 && own_id < v0 + len) own_z = Elem<in_t>::get(z[own_id - v0]);
    __syncthreads();
  }
  for (int32_t i0 = threadIdx.x; i0 < groups; i0 += kBatch * kLogitThreads) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int32_t i = i0 + u * kLogitThreads;
      if (i >= groups) break;
      float x[kGroup];
      if (wide_loads) {
        raw[u].widen(x);
      } else {
#pragma unroll
        for (int k = 0; k < kGroup; ++k) x[k] = Elem<in_t>::get(zg[i * kGroup + k]);
      }
      const uint32_t keep = mask ? __funnelshift_r(words[u].x, words[u].y, v0 + head + i * kGroup) : ~0u;
      load(u, i + kBatch * kLogitThreads);
      uint32_t any = 0;
      if (kBits) {
        uint32_t w[C::kWords];
        counts.group(head + i * kGroup, w);
#pragma unroll
        for (int k = 0; k < C::kWords; ++k) any |= w[k];
        if (any) {
#pragma unroll
          for (int k = 0; k < kGroup; ++k) x[k] = penalised(x[k], C::of(w, k));
        }
      }
      if (mask) {
#pragma unroll
        for (int k = 0; k < kGroup; ++k)
          if (!(keep >> k & 1u)) x[k] = -INFINITY;
      }
      if (!(any & (kBits == 16 ? C::kBias * 0x10001u : C::kBias))) {
        store8(yg + i * kGroup, x);
      } else {
#pragma unroll
        for (int k = 0; k < kGroup; ++k)
          if (!(counts.get(head + i * kGroup + k) & C::kBias)) yg[i * kGroup + k] = Elem<out_t>::put(x[k]);
      }
    }
  }
  // the few tokens before the first group and after the last
  for (int32_t o = threadIdx.x; o < len - groups * kGroup; o += kLogitThreads) {
    const int32_t at = o < head ? o : o + groups * kGroup;
    const uint32_t c = kBits ? counts.get(at) : 0;
    if (!(c & C::kBias)) y[at] = Elem<out_t>::put(allowed(v0 + at) ? penalised(Elem<in_t>::get(z[at]), c) : -INFINITY);
  }
  if (!kBits || *repeated) return;
  // each biased token by the thread of its entry
  for (int64_t j = l.bs + threadIdx.x; j < l.be; j += kLogitThreads) {
    const bool first = j == l.bs + threadIdx.x;
    const int64_t v = first ? own_id : a.b_ids[j];
    if (v < v0 || v >= v0 + len) continue;
    const float x = penalised(first ? own_z : Elem<in_t>::get(z[v - v0]), counts.get((uint32_t)(v - v0)));
    y[v - v0] = Elem<out_t>::put(allowed((uint32_t)v) ? x + (first ? own_bias : a.b_val[j]) : -INFINITY);
  }
}

// Apart from the usual ones, so that they share no registers with these.
template <typename in_t, typename out_t>
__device__ __noinline__ void process_long(const LogitsArgs& a, int32_t b, int32_t v0, int32_t len, const Lists& l,
                                          const Penalty& penalty, uint32_t* smem, int* repeated) {
  process<in_t, out_t, 32>(a, b, v0, len, l, penalty, smem, repeated);
  if (*repeated) add_biases<in_t, out_t, 32>(a, b, v0, len, l, penalty, smem);
}

template <typename in_t, typename out_t, bool kLists>
__global__ void __launch_bounds__(kLogitThreads, kLogitBlocks) k_logits(LogitsArgs a) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ int repeated;  // a bias list names a token twice
  pdl_wait();
  pdl_trigger();
  const int32_t b = blockIdx.y;
  const int32_t v0 = (int32_t)blockIdx.x * a.slice, len = min(a.V - v0, a.slice);
  const float rep = a.rep ? a.rep[b] : 1.f;
  const Penalty penalty{rep, __frcp_rn(rep), a.freq ? a.freq[b] : 0.f, a.pres ? a.pres[b] : 0.f};
  Lists l{};
  if constexpr (!kLists) {
    process<in_t, out_t, 0>(a, b, v0, len, l, penalty, smem, &repeated);
    return;
  }
  if (a.p_ids) list_of(a.p_off, a.p_n, b, a.status, &l.ps, &l.pe);
  if (a.o_ids) list_of(a.o_off, a.o_n, b, a.status, &l.os, &l.oe, Counts<32>::kTimes);  // more are not counted
  if (a.b_ids) list_of(a.b_off, a.b_n, b, a.status, &l.bs, &l.be);
  if (l.oe - l.os <= (int64_t)Counts<16>::kTimes) {
    process<in_t, out_t, 16>(a, b, v0, len, l, penalty, smem, &repeated);
    if (repeated) add_biases<in_t, out_t, 16>(a, b, v0, len, l, penalty, smem);
    return;
  }
  const int32_t half = a.slice / 2;  // the room of a slice's 16-bit entries
  for (int32_t o = 0; o < len; o += half) {
    __syncthreads();  // the piece before is done with its counts
    process_long<in_t, out_t>(a, b, v0 + o, min(half, len - o), l, penalty, smem, &repeated);
  }
}

template <typename in_t, typename out_t>
cudaError_t launch(int device, LogitsArgs& a, cudaStream_t s) {
  void* args[] = {&a};
  // Slices as large as three blocks an SM have room to count, of a size that fills whole
  // waves of them: the fewest waves that such slices allow (64 x 128256 fp32: 26 us with
  // slices that took 1.1 waves, 20.5 with one).
  const int64_t slots = (int64_t)kLogitBlocks * sm_count(device);
  const int64_t least = (a.V + kMaxSlice - 1) / kMaxSlice, waves = (least * a.B + slots - 1) / slots;
  const int64_t a_row = waves * slots / a.B;  // slices of a row, at least `least`
  a.slice = std::max(kMinSlice, (int32_t)(((a.V + a_row - 1) / a_row + 1023) / 1024 * 1024));
  const dim3 grid((a.V + a.slice - 1) / a.slice, a.B);
  if (!a.p_ids && !a.o_ids && !a.b_ids)
    return launch_kernel(reinterpret_cast<const void*>(&k_logits<in_t, out_t, false>), grid, dim3(kLogitThreads), 0, s,
                         args, true);
  const void* fn = reinterpret_cast<const void*>(&k_logits<in_t, out_t, true>);
  static bool ready[64];
  const cudaError_t e = allow_smem(fn, kMaxSlice * 2 + 128, device, ready);
  if (e != cudaSuccess) return e;
  return launch_kernel(fn, grid, dim3(kLogitThreads), (size_t)a.slice * 2 + 128, s, args, true);
}

template <typename in_t>
cudaError_t launch_out(int device, int out, LogitsArgs& a, cudaStream_t s) {
  switch (out) {
    case EMB_F32: return launch<in_t, float>(device, a, s);
    case EMB_F16: return launch<in_t, __half>(device, a, s);
    default: return launch<in_t, __nv_bfloat16>(device, a, s);
  }
}

bool list_args_ok(const int64_t* ids, const int64_t* off, int64_t n) {
  if (n < 0 || n > INT32_MAX || !aligned(ids, 8) || !aligned(off, 8)) return false;
  return off || (!ids && n == 0);
}

}  // namespace
}  // namespace embbwd

using namespace embbwd;

extern "C" emb_status emb_logits_process(
    int device, const void* logits, emb_dtype logits_dtype, int64_t logits_stride, int32_t B, int32_t V,
    const int64_t* prompt_ids, const int64_t* prompt_offsets, int64_t prompt_n, const int64_t* output_ids,
    const int64_t* output_offsets, int64_t output_n, const float* repetition, const float* frequency,
    const float* presence, const int64_t* bias_ids, const int64_t* bias_offsets, const float* bias_values,
    int64_t bias_n, const uint32_t* mask, int64_t mask_stride, void* out, emb_dtype out_dtype, int64_t out_stride,
    uint32_t* device_status, void* stream) {
  if (device < 0 || B < 0 || B > 65535 || V < 1 || V > kMaxVocab) return EMB_ERR_INVALID_ARG;
  if (!dtype_ok(logits_dtype) || !dtype_ok(out_dtype)) return EMB_ERR_INVALID_ARG;
  if (!list_args_ok(prompt_ids, prompt_offsets, prompt_n) || !list_args_ok(output_ids, output_offsets, output_n) ||
      !list_args_ok(bias_ids, bias_offsets, bias_n) || (bias_ids && !bias_values))
    return EMB_ERR_INVALID_ARG;
  if (!aligned(repetition, 4) || !aligned(frequency, 4) || !aligned(presence, 4) || !aligned(bias_values, 4) ||
      !aligned(mask, 4) || !aligned(device_status, 4))
    return EMB_ERR_INVALID_ARG;
  if (B == 0) return EMB_OK;
  if (!logits || !out || !aligned(logits, dtype_size(logits_dtype)) || !aligned(out, dtype_size(out_dtype)))
    return EMB_ERR_INVALID_ARG;
  if (B > 1 && (logits_stride < V || out_stride < V)) return EMB_ERR_INVALID_ARG;
  if (mask && B > 1 && mask_stride < (V + 31) / 32) return EMB_ERR_INVALID_ARG;
  // in place means the same elements; another type there would be overwritten before it is read
  if (logits == out && (logits_dtype != out_dtype || (B > 1 && logits_stride != out_stride))) return EMB_ERR_INVALID_ARG;
  LogitsArgs a{logits,     out,        logits_stride, out_stride,    B,        V,        prompt_ids, prompt_offsets,
               output_ids, output_offsets, bias_ids,  bias_offsets,  prompt_n, output_n, bias_n,     repetition,
               frequency,  presence,   bias_values,   mask,          mask_stride, device_status, 0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return on_device(device, [&] {
    switch (logits_dtype) {
      case EMB_F32: return launch_out<float>(device, out_dtype, a, s);
      case EMB_F16: return launch_out<__half>(device, out_dtype, a, s);
      default: return launch_out<__nv_bfloat16>(device, out_dtype, a, s);
    }
  });
}
