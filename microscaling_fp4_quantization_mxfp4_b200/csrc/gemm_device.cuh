// Device-side building blocks shared by the tensor-core GEMM kernels of libfp4 (sm_100a only):
// mbarriers with bounded waits, TMA and bulk copies, tensor-memory loads, shared-memory
// descriptors, cluster helpers and the bf16 epilogue store.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include "copy_ring.h"

namespace fp4tc {

constexpr unsigned long long kWaitLimitNs = 4000000000ull;   // 4 s per wait
constexpr int kEpiStage = 4096;         // one 32-row x 64-column bf16 box, 128B-swizzled

// ------------------------------------------------------------ PTX wrappers --
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0u;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint64_t global_timer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Bounded wait: false when the time limit passes or another role raised abort.
// try_wait with a suspend-time hint: the warp sleeps in hardware until the
// phase completes or ~20 us pass, instead of spinning on issue slots.
__device__ __forceinline__ bool mbar_try_wait_sleep(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0u;
}
// Critical-path wait (producer, MMA issuer): spin on try_wait, checking the
// abort flag and the time limit every 1024 polls.
__device__ __forceinline__ bool wait_spin(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 1023u) == 0u) {
      if (*abort_flag != 0) return false;
      if (global_timer() - t0 > kWaitLimitNs) return false;
    }
  }
}
// Long waits (epilogue warps): sleep in hardware between polls.
static __device__ __noinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer();
  for (;;) {
    if (mbar_try_wait_sleep(bar, parity)) return true;
    if (*abort_flag != 0) return false;
    if (global_timer() - t0 > kWaitLimitNs) return false;
  }
}
__device__ __forceinline__ void raise_abort(volatile int* abort_flag, unsigned* error) {
  *abort_flag = 1;
  atomicOr(error, 1u);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_cp_sf(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Waits for this thread's tensor-memory loads into r[4][32].  The registers are in-out operands of
// the wait (and of an empty statement right after it), so the compiler cannot schedule any use of
// them ahead of the wait.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[4][32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0][0]), "+r"(r[0][1]), "+r"(r[0][2]), "+r"(r[0][3]), "+r"(r[0][4]), "+r"(r[0][5]), "+r"(r[0][6]), "+r"(r[0][7]), "+r"(r[0][8]), "+r"(r[0][9]), "+r"(r[0][10]), "+r"(r[0][11]), "+r"(r[0][12]), "+r"(r[0][13]), "+r"(r[0][14]), "+r"(r[0][15]), "+r"(r[0][16]), "+r"(r[0][17]), "+r"(r[0][18]), "+r"(r[0][19]), "+r"(r[0][20]), "+r"(r[0][21]), "+r"(r[0][22]), "+r"(r[0][23]), "+r"(r[0][24]), "+r"(r[0][25]), "+r"(r[0][26]), "+r"(r[0][27]), "+r"(r[0][28]), "+r"(r[0][29]), "+r"(r[0][30]), "+r"(r[0][31]),
                 "+r"(r[1][0]), "+r"(r[1][1]), "+r"(r[1][2]), "+r"(r[1][3]), "+r"(r[1][4]), "+r"(r[1][5]), "+r"(r[1][6]), "+r"(r[1][7]), "+r"(r[1][8]), "+r"(r[1][9]), "+r"(r[1][10]), "+r"(r[1][11]), "+r"(r[1][12]), "+r"(r[1][13]), "+r"(r[1][14]), "+r"(r[1][15]), "+r"(r[1][16]), "+r"(r[1][17]), "+r"(r[1][18]), "+r"(r[1][19]), "+r"(r[1][20]), "+r"(r[1][21]), "+r"(r[1][22]), "+r"(r[1][23]), "+r"(r[1][24]), "+r"(r[1][25]), "+r"(r[1][26]), "+r"(r[1][27]), "+r"(r[1][28]), "+r"(r[1][29]), "+r"(r[1][30]), "+r"(r[1][31])
               :
               : "memory");
  asm volatile(""
               : "+r"(r[2][0]), "+r"(r[2][1]), "+r"(r[2][2]), "+r"(r[2][3]), "+r"(r[2][4]), "+r"(r[2][5]), "+r"(r[2][6]), "+r"(r[2][7]), "+r"(r[2][8]), "+r"(r[2][9]), "+r"(r[2][10]), "+r"(r[2][11]), "+r"(r[2][12]), "+r"(r[2][13]), "+r"(r[2][14]), "+r"(r[2][15]), "+r"(r[2][16]), "+r"(r[2][17]), "+r"(r[2][18]), "+r"(r[2][19]), "+r"(r[2][20]), "+r"(r[2][21]), "+r"(r[2][22]), "+r"(r[2][23]), "+r"(r[2][24]), "+r"(r[2][25]), "+r"(r[2][26]), "+r"(r[2][27]), "+r"(r[2][28]), "+r"(r[2][29]), "+r"(r[2][30]), "+r"(r[2][31]),
                 "+r"(r[3][0]), "+r"(r[3][1]), "+r"(r[3][2]), "+r"(r[3][3]), "+r"(r[3][4]), "+r"(r[3][5]), "+r"(r[3][6]), "+r"(r[3][7]), "+r"(r[3][8]), "+r"(r[3][9]), "+r"(r[3][10]), "+r"(r[3][11]), "+r"(r[3][12]), "+r"(r[3][13]), "+r"(r[3][14]), "+r"(r[3][15]), "+r"(r[3][16]), "+r"(r[3][17]), "+r"(r[3][18]), "+r"(r[3][19]), "+r"(r[3][20]), "+r"(r[3][21]), "+r"(r[3][22]), "+r"(r[3][23]), "+r"(r[3][24]), "+r"(r[3][25]), "+r"(r[3][26]), "+r"(r[3][27]), "+r"(r[3][28]), "+r"(r[3][29]), "+r"(r[3][30]), "+r"(r[3][31]));
}

// TMA store of one box from shared memory, and bulk-group completion.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void bulk_commit_group() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read0() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all0() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// One epilogue warp's 32 rows x 128 accumulator columns (r[c][i] = column 32c + i of row
// y0 + lane) -> alpha * value in bf16 -> two 32 x 64 boxes through the warp's 4 KB staging
// buffer (1024-byte aligned, 128B-swizzled: 16-byte chunk j of row i at chunk j ^ (i & 7), the
// layout the tensor map's SWIZZLE_128B expects) -> TMA stores, which clip rows >= M and columns
// >= N.  The buffer is reused for the second box once the first store has read it.
__device__ __forceinline__ void epi_store_bf16_tma(const CUtensorMap* tmap_y, uint8_t* stg, const uint32_t (&r)[4][32],
                                                   float alpha, int x0, int y0, int M, int N, int lane) {
  const uint32_t base = smem_u32(stg) + (uint32_t)lane * 128u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (lane == 0) bulk_wait_read0();        // the previous box's store has read the buffer
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = __fmul_rn(__uint_as_float(r[2 * h + (j >> 2)][(j & 3) * 8 + 2 * i]), alpha);
        const float hi = __fmul_rn(__uint_as_float(r[2 * h + (j >> 2)][(j & 3) * 8 + 2 * i + 1]), alpha);
        w[i] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(lo)) |
               ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(hi)) << 16);
      }
      const uint32_t dst = base + (uint32_t)(((j ^ (lane & 7)) & 7) * 16);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                   : "memory");
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // generic writes -> async-proxy reads
    __syncwarp();
    if (lane == 0 && x0 + 64 * h < N && y0 < M) {       // boxes wholly past the edge are skipped
      tma_store_2d(tmap_y, smem_u32(stg), x0 + 64 * h, y0);
      bulk_commit_group();
    }
  }
}

// Shared-memory matrix descriptor: K-major operand, 128-byte rows, 128B
// swizzle, 8-row groups 1024 bytes apart (Blackwell descriptor version 1).
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)1u << 16) | ((uint64_t)(1024u >> 4) << 32) |
         ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}
// Descriptor of one 512-byte scale atom: 32 rows of 16 bytes, no swizzle,
// 8-row core matrices 128 bytes apart.
__device__ __forceinline__ uint64_t desc_sf(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)1u << 16) | ((uint64_t)(128u >> 4) << 32) |
         ((uint64_t)1u << 46);
}

// One 32-byte store (a whole L2 sector) of eight 32-bit words; dst 32-byte aligned.
__device__ __forceinline__ void st_global_v8(void* dst, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

__device__ __forceinline__ void tile_coords(int t, int num_m, int num_n, int& mt, int& nt) {
  constexpr int kGroup = 8;
  const int band = t / (kGroup * num_n);
  const int first = band * kGroup;
  const int gsize = min(kGroup, num_m - first);
  const int local = t - band * kGroup * num_n;
  mt = first + local % gsize;
  nt = local / gsize;
}


// ------------------------------------------------------- clusters and pairs --
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// shared::cluster address of the same shared-memory location in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(addr), "r"(rank));
  return d;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Bytes announced on a barrier of this CTA that no copy will bring.
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
__device__ __forceinline__ void tc_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
// commit of the pair's tensor-core work to a barrier of this CTA only
__device__ __forceinline__ void tc_commit_pair_local(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_cp_sf_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// How an SM pair ends: what its producers asked for, and whether a wait of the leader's ran out.
// The leader's words are written by both CTAs before a cluster barrier and read behind it.
struct PairEnd {
  uint32_t halted;
  uint32_t asked[2][2];            // [CTA][ring]: operands, scales
};
__device__ __forceinline__ void pair_end_init(PairEnd* e) {
  volatile uint32_t* w = reinterpret_cast<volatile uint32_t*>(e);
  for (int i = 0; i < 5; ++i) w[i] = 0u;
}
__device__ __forceinline__ void pair_end_asked(PairEnd* e, uint32_t rank, uint32_t operands, uint32_t scales) {
  const uint32_t at = map_rank(smem_u32(&e->asked[rank][0]), 0);
  st_cluster_u32(at, operands);
  st_cluster_u32(at + 4u, scales);
}
__device__ __forceinline__ void pair_end_halt(PairEnd* e) {
  for (uint32_t r = 0; r < 2; ++r) st_cluster_u32(map_rank(smem_u32(&e->halted), r), 1u);
}
__device__ __forceinline__ bool pair_halted(const PairEnd* e) { return *reinterpret_cast<const volatile uint32_t*>(&e->halted) != 0u; }

// One thread of the leader, behind the cluster barrier that both producers have reached: waits (each wait bounded) for
// the copies of ring `ring` that are still in flight.  `bytes`: one CTA's share of a copy.
static __device__ __noinline__ bool settle_pair_copies(uint64_t* bars, uint32_t slots, const PairEnd* end, int ring,
                                                       uint32_t bytes) {
  struct {
    uint32_t bar0, bytes;
    __device__ void announce_one(uint32_t slot) { mbar_expect_tx(bar0 + 8u * slot, bytes); }
    __device__ void forgo_one(uint32_t slot) { mbar_complete_tx(bar0 + 8u * slot, bytes); }
    __device__ bool wait(uint32_t slot, uint32_t parity) {
      volatile int never = 0;
      return wait_bounded(bar0 + 8u * slot, parity, &never);
    }
  } barriers{smem_u32(bars), bytes};
  const volatile uint32_t* asked = &end->asked[0][0];
  return fp4ring::settle_pair(asked[ring], asked[2 + ring], slots, barriers);
}

// One thread, behind the barrier that the producer has reached: waits (each wait bounded) for those of `asked` copies of
// a ring that are still in flight.
static __device__ __noinline__ bool settle_copies(uint64_t* bars, uint32_t slots, uint32_t asked) {
  volatile int never = 0;
  for (uint32_t n = fp4ring::first_open(asked, slots); n < asked; ++n)
    if (!wait_bounded(smem_u32(&bars[fp4ring::slot_of(n, slots)]), fp4ring::parity_of(n, slots), &never)) return false;
  return true;
}

// Called only between the two cluster barriers, which order it against the partials' stores.
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}


// ------------------------------------------------------------------- host --
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  return encode;
}

}  // namespace fp4tc
