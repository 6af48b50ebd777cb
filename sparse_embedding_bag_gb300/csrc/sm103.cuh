// sm_103a instructions used by the vocabulary operators, as inline PTX: mbarriers with
// bounded waits, bulk and tensor copies, tensor memory, block-scaled 4-bit MMA.
#pragma once

#include <cuda.h>

#include "vocab.cuh"

namespace embbwd {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// ---- arithmetic

// 2^x; the result is at most 2 ulp off, subnormal results are 0.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two floats in one register pair, two operations an instruction.
struct F2 {
  uint64_t u;
  __device__ __forceinline__ static F2 of(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.u) : "f"(a), "f"(b));
    return r;
  }
  __device__ __forceinline__ float2 get() const {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(u));
    return r;
  }
  __device__ __forceinline__ F2 operator+(F2 o) const {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(u), "l"(o.u));
    return r;
  }
  __device__ __forceinline__ F2 operator*(F2 o) const {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(u), "l"(o.u));
    return r;
  }
};

// ---- mbarriers

#ifndef EMB_WAIT_NS  // a test builds the library with waits that run out at once
#define EMB_WAIT_NS 2000000000ull
#endif
constexpr uint64_t kWaitNs = EMB_WAIT_NS;     // a wait gives up after two seconds
constexpr uint64_t kDrainNs = 2000000000ull;  // and one for work that is known to be under way

// The time that a wait has spent. What passes between two looks at the clock counts as ten
// milliseconds at most: a process that was suspended or lost its time slice for seconds has
// not waited for them.
struct Patience {
  uint64_t last = global_ns(), spent = 0;
  __device__ __forceinline__ bool over(uint64_t limit) {
    const uint64_t now = global_ns(), passed = now - last;
    spent += passed < 10000000 ? passed : 10000000;
    last = now;
    return spent > limit;
  }
};

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_init_fence() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_try_cluster(uint32_t bar, uint32_t parity) {  // sees the other CTAs' writes too
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// `bar` is a cluster address.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
template <bool kCluster>
__device__ __forceinline__ bool mbar_tries(uint32_t bar, uint32_t parity) {
  return kCluster ? mbar_try_cluster(bar, parity) : mbar_try(bar, parity);
}

// ---- clusters

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Writes of all threads of the cluster before it are seen by all after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same in two halves: arrive (early), and wait for the others' arrival.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The address of this CTA's shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ void cluster_store(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

// ---- bounded waits. `*abort` is a flag in shared memory, set by the first wait of a block (kPair:
// of a pair of CTAs, where both have it at the same address) that gives up; the others then
// do so too.

template <bool kPair>
__device__ __forceinline__ void give_up(volatile int* abort) {
  *abort = 1;
  if (kPair)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_map(smem_u32(const_cast<int*>(abort)), cluster_rank() ^ 1)),
                 "r"(1)
                 : "memory");
}
// Waits for the phase with that parity to complete; false if it does not. Lanes that wait
// together may differ in the answer.
template <bool kPair>
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (mbar_tries<kPair>(bar, parity)) return true;
  for (Patience p;;) {
    for (int i = 0; i < 8; ++i)
      if (mbar_tries<kPair>(bar, parity)) return true;
    if (*abort || p.over(kWaitNs)) {
      give_up<kPair>(abort);
      return false;
    }
  }
}

// ---- copies

// A box of a 2-D tensor map to this CTA's shared memory. With kPair the barrier (a cluster
// address) may be the other CTA's of the pair.
template <bool kPair>
__device__ __forceinline__ void tensor_load(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
  if (kPair)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
            "r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Brings a box to L2.
__device__ __forceinline__ void tensor_prefetch(const CUtensorMap* map, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}

// ---- tensor memory and block-scaled MMA, of one CTA or (kPair) of a cluster of two: then
// one lane of CTA 0 issues for both, an operand or scale address stands for the same
// address in both CTAs, and both allocate.

#define EMB_GROUP(text1, text2, ...)      \
  do {                                    \
    if (kPair)                            \
      asm volatile(text2 __VA_ARGS__);    \
    else                                  \
      asm volatile(text1 __VA_ARGS__);    \
  } while (0)

template <bool kPair>
__device__ __forceinline__ void tmem_alloc(uint32_t smem_result, uint32_t cols) {
  EMB_GROUP("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;",
            "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;", ::"r"(smem_result), "r"(cols)
            : "memory");
  EMB_GROUP("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;",
            "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;", );
}
template <bool kPair>
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
  EMB_GROUP("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;", "tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;",
            ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// All MMAs and copies issued so far by this thread arrive on the barrier when done; with
// kBoth on the barrier at that address in both CTAs of a pair.
template <bool kPair, bool kBoth = kPair>
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  if (kBoth)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
    EMB_GROUP("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];",
              "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];", ::"r"(bar)
              : "memory");
}
// 512 bytes of scales (32 rows of 16 bytes) to 4 columns, repeated for the four warps' lanes.
template <bool kPair>
__device__ __forceinline__ void tc_copy_scales(uint32_t tmem, uint64_t desc) {
  EMB_GROUP("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;", "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;",
            ::"r"(tmem), "l"(desc)
            : "memory");
}
#define EMB_MMA(group, kind)                                                                                  \
  "{ .reg .pred p; setp.ne.b32 p, %6, 0;\n"                                                                   \
  "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, [%4], [%5], p; }"
template <bool kPair, bool kE8M0>
__device__ __forceinline__ void tc_mma_f4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, bool accumulate) {
  if (kE8M0)
    EMB_GROUP(EMB_MMA("1", "mxf4.block_scale.scale_vec::2X"), EMB_MMA("2", "mxf4.block_scale.scale_vec::2X"), ::"r"(d),
              "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)accumulate)
              : "memory");
  else
    EMB_GROUP(EMB_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X"), EMB_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X"),
              ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)accumulate)
              : "memory");
}
#undef EMB_MMA
#undef EMB_GROUP
// 16 consecutive columns of this warp's 32 lanes: register i of lane l is column i of lane l.
__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&v)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptors. Operands: K-major, rows of 128 bytes in the
// 128-byte swizzle, groups of 8 rows 1024 bytes apart. Scales: no swizzle, groups of 8
// rows (16 bytes each) 128 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
__device__ __forceinline__ uint64_t scales_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

// ---- host side

// Launches fn with clusters of `cluster` CTAs along x (a divisor of grid.x); with pdl set, as a
// programmatic dependent of the kernel before it on the stream.
inline cudaError_t launch_clusters(const void* fn, dim3 grid, dim3 block, int cluster, size_t smem, cudaStream_t s,
                                   void** args, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}
// Raises fn's dynamic shared memory limit, once for each device (`ready`: 64 zeros).
inline cudaError_t allow_smem(const void* fn, size_t bytes, int device, bool* ready) {
  if (device < 64 && ready[device]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && device < 64) ready[device] = true;  // idempotent: a race sets the same limit twice
  return e;
}

// A 2-D map of `rows` rows of `row_bytes` bytes (a multiple of 16), read in boxes of
// box_rows x 128 bytes in the 128-byte swizzle; reads beyond the matrix give zeros.
cudaError_t byte_matrix_map(CUtensorMap* map, const void* base, int64_t rows, int64_t row_bytes, int box_rows);
// A 2-D map of `rows` rows of `tiles` 512-byte tiles, read in boxes of box_rows x box_tiles
// (at most 4); reads beyond it give zeros.
cudaError_t tile_matrix_map(CUtensorMap* map, const void* base, int64_t rows, int64_t tiles, int box_rows, int box_tiles);
// Streaming multiprocessors of the device (asked once).
int sm_count(int device);

}  // namespace embbwd
