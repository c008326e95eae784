// Block-scaled FP8 x FP8 product with fp32 accumulation on the sm_100a tensor cores (tcgen05), fed by TMA.
//
//   Y[M,N] = sum over 128-element blocks kb of 2^(ea[m,kb] + eb[n,kb]) * sum_{k in kb} a[m,k] * b[n,k]
//
// with A and B in E4M3 or E5M2 (each its own), both along K, and the E8M0 bytes of their 1 x 128 blocks
// (or 128 x 128 tiles, whose byte every row repeats) in the tensor-core scale layout.
//
// kind::mxf8f6f4 scales 32 elements of K by one byte of a row's 32-bit scale word, the byte chosen by
// the instruction.  The four K = 32 instructions of a 128-element block all name the same byte, so the
// layout holds one byte a block and one 512-byte atom (128 rows x 4 bytes) serves 512 elements of K: a
// quarter of the scale bytes, and of the copies into tensor memory, that 32-element blocks need.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "fp4_device.cuh"
#include "fp4_internal.h"
#include "fp8_internal.h"
#include "gemm_device.cuh"

namespace fp4lib {
using namespace fp4tc;
namespace {

constexpr int kBK = 128;                  // elements (= bytes) of K per stage: one scale block
constexpr uint32_t kCols = 512;           // tensor memory columns
constexpr uint32_t kScaleBufs = 4;        // scale buffers (512 elements of K each), shared memory and tensor memory
constexpr int kRing = 216 * 1024;

struct Fp8KernelArgs {
  const uint8_t* a_sf;
  const uint8_t* b_sf;
  void* y;
  long long ldy;
  int M, N, K;
  int num_m, num_n;
  int g4;                                 // 512-element scale atoms along K
  uint32_t a_type, b_type;                // 0 E4M3, 1 E5M2
  int vec_store;                          // output rows 16-byte aligned
  unsigned* error;
};

// One lane of a converged warp.  A loop that issues tcgen05 instructions behind `lane == 0` keeps their
// operands in vector registers and moves them to uniform ones before every instruction (170 cycles per
// M = 256, N = 256 MMA, measured); behind elect.sync the compiler keeps them uniform and the loop runs
// at the MMA's own 128.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0u;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// A: the 128 (or, over an SM pair, 256) rows of the accumulator; B: its n columns.  `id`: the byte of
// the scale words that this block's instructions use.
__device__ __forceinline__ uint32_t fp8_idesc(uint32_t m, uint32_t n, uint32_t a_type, uint32_t b_type, uint32_t id) {
  return (id << 4) | (a_type << 7) | (b_type << 10) | ((n >> 3) << 17) | (1u << 23) | ((m >> 7) << 27) | (id << 29);
}
__device__ __forceinline__ void fp8_mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}

// ------------------------------------------------- tiles of Y^T over clusters --
// Y^T = B . A^T in tiles of 128 rows of B by BNT rows of A (16 to 256), so that a product with few
// activation rows fills the MMA's 128 rows with weights and reads each of them once.  A tile's blocks
// of K are divided over a cluster of `split` CTAs; each CTA accumulates its share in tensor memory.
// A CTA on its own stores its tile from registers, 32 neighbours of a row of Y at a time (parking it first
// in shared memory to store 16 bytes a thread was slower: 48 x 11008 x 4096 12.4 -> 11.5 us, 32 x 32000 x
// 4096 27.9 -> 26.3).  In a cluster every CTA adds one slice of the tile, in rank order, and stores it.  Up
// to 64 rows of A each CTA writes its share of a slice into the memory of the CTA that adds it, behind the
// ring, and one cluster barrier later the sum reads its own memory.  More rows find no room there; their
// shares are parked in the idle ring and read by the others between two barriers (for up to 64 rows that
// took 7.0 against 6.6 us for 1 x 4096 x 4096, 8.7 against 7.9 for 64 x 4096 x 4096).  All barriers are
// reached on every path, errors included.
//
// warp 0 TMA producer, warp 1 MMA issuer (one thread each), warps 2-5 epilogue, warp 6 scale copies.
namespace tiles {

constexpr int kMaxSplit = 8;

template <int BNT>
struct Cfg {
  static constexpr int kThreads = 224;
  static constexpr int kWBytes = 128 * kBK;
  static constexpr int kXBytes = BNT * kBK;
  static constexpr int kXAtoms = (BNT + 127) / 128;
  static constexpr int kScaleBytes = (1 + kXAtoms) * 512;
  static constexpr int kStageBytes = kWBytes + kXBytes;
  static constexpr int kStages = std::min((kRing - (int)kScaleBufs * kScaleBytes) / kStageBytes, 12);
  // Up to 64 rows of A, clusters have room behind fewer stages for the peers' shares of a CTA's own columns:
  // [rank][row][slice_cols], where slice_cols * split is at most 144.
  static constexpr bool kPush = BNT <= 64;
  static constexpr int kRecvBytes = BNT * 144 * 4;
  static constexpr int kPushStages = std::min((kRing - kRecvBytes - (int)kScaleBufs * kScaleBytes) / kStageBytes, 12);
  static constexpr int kPStride = 128 + 4;                       // floats of a parked row
  static constexpr int kRingBytes =
      std::max(kStages * kStageBytes, kPush ? kPushStages * kStageBytes + kRecvBytes : BNT * kPStride * 4);
  static constexpr int kSmem = 1024 + kRingBytes + (int)kScaleBufs * kScaleBytes + 512;
  static constexpr uint32_t kScaleCol = 256;                     // scale buffers after the accumulator
  static constexpr uint32_t kScaleCols = 16;                     // B's 4 columns, then A's 4 or 8
};

// NV rows of Y from m0 on, in this lane's column n: a warp's lanes store 32 neighbours of each row.
template <int NV, bool BF16>
__device__ __forceinline__ void store_lane(const Fp8KernelArgs& p, const uint32_t (&r)[NV], int m0, int n) {
  if (n >= p.N) return;
  const long long o = (long long)m0 * p.ldy + n;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (m0 + i >= p.M) break;
    if (BF16) static_cast<__nv_bfloat16*>(p.y)[o + i * p.ldy] = __float2bfloat16_rn(__uint_as_float(r[i]));
    else static_cast<float*>(p.y)[o + i * p.ldy] = __uint_as_float(r[i]);
  }
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Columns of a CTA's slice of the tile, a multiple of 4.
__device__ __forceinline__ int slice_cols(int split) { return ((128 + split - 1) / split + 3) & ~3; }

// NV rows from m0 on, in this lane's column: into the memory of the CTA that adds that column.
template <int NV>
__device__ __forceinline__ void push_lane(uint32_t dst, const uint32_t (&r)[NV], int m0, int rows, int slice) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (m0 + i >= rows) break;
    st_cluster_u32(dst + (uint32_t)((m0 + i) * slice * 4), r[i]);
  }
}

// Four neighbours of a row of Y from column n0 on.
template <bool BF16>
__device__ __forceinline__ void store4(const Fp8KernelArgs& p, const float4& v, int m, int n0) {
  const float y4[4] = {v.x, v.y, v.z, v.w};
  const long long o = (long long)m * p.ldy + n0;
  if (BF16) {
    __nv_bfloat16* yr = static_cast<__nv_bfloat16*>(p.y) + o;
    if (p.vec_store && n0 + 4 <= p.N) {
      *reinterpret_cast<uint2*>(yr) =
          make_uint2((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(y4[0])) |
                         ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(y4[1])) << 16),
                     (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(y4[2])) |
                         ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(y4[3])) << 16));
    } else {
      for (int i = 0; i < 4; ++i)
        if (n0 + i < p.N) yr[i] = __float2bfloat16_rn(y4[i]);
    }
  } else {
    float* yr = static_cast<float*>(p.y) + o;
    if (p.vec_store && n0 + 4 <= p.N) {
      *reinterpret_cast<float4*>(yr) = v;
    } else {
      for (int i = 0; i < 4; ++i)
        if (n0 + i < p.N) yr[i] = y4[i];
    }
  }
}
__device__ __forceinline__ float4 add4(const float4& a, const float4& b) {
  return make_float4(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z), __fadd_rn(a.w, b.w));
}

template <int BNT, bool BF16, bool CLUSTER>
__global__ void __launch_bounds__(Cfg<BNT>::kThreads, 1)
    fp8_gemm_tile_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                         Fp8KernelArgs p, int cluster) {
  using C = Cfg<BNT>;
  constexpr bool PUSH = CLUSTER && C::kPush;
  constexpr int S = PUSH ? C::kPushStages : C::kStages;
  const int split = CLUSTER ? cluster : 1;
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sW = smem;
  uint8_t* sX = sW + S * C::kWBytes;
  float* part = reinterpret_cast<float*>(smem);                  // reuses the ring after the last MMA
  float* recv = reinterpret_cast<float*>(smem + C::kPushStages * C::kStageBytes);
  uint8_t* sScale = smem + C::kRingBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sScale + kScaleBufs * C::kScaleBytes);
  uint64_t* full = bars;
  uint64_t* empty = full + S;
  uint64_t* sload = empty + S;                                   // scale buffer in shared memory
  uint64_t* sfull = sload + kScaleBufs;                          // ... in tensor memory
  uint64_t* sempty = sfull + kScaleBufs;                         // ... read by its last MMA
  uint64_t* tfull = sempty + kScaleBufs;
  uint64_t* drain = tfull + 1;
  uint64_t* sdrain = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* asked = tmem_slot + 2;                      // copies of operands and of scales asked for

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CLUSTER ? cluster_rank() : 0u;
  const int tile = (int)(blockIdx.x / (uint32_t)split);
  const int nt = tile % p.num_n, mt = tile / p.num_n;
  const int nkb = (p.K + kBK - 1) / kBK;
  const int kb0 = (int)((int64_t)nkb * rank / split), kb1 = (int)((int64_t)nkb * (rank + 1) / split);

  if (threadIdx.x == 0) {
    prefetch_map(&tmap_w);
    prefetch_map(&tmap_x);
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (uint32_t b = 0; b < kScaleBufs; ++b) {
      mbar_init(smem_u32(&sload[b]), 1);
      mbar_init(smem_u32(&sfull[b]), 1);
      mbar_init(smem_u32(&sempty[b]), 1);
    }
    mbar_init(smem_u32(tfull), 1);
    mbar_init(smem_u32(drain), 1);
    mbar_init(smem_u32(sdrain), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (PUSH) cluster_arrive();               // this CTA runs: its peers may write to its memory
  pdl_wait();                               // the previous kernel's outputs (our operands) are complete

  if (warp == 0) {
    // ------------------------------------------------------------ producer --
    if (elect_one()) {
      const int x_atoms = min(C::kXAtoms, (p.M + 127) / 128 - mt * C::kXAtoms);
      int stage = 0;
      uint32_t lap = 0, ns = 0;                                  // rounds of the ring, scale copies asked for
      for (int kb = kb0; kb < kb1; ++kb) {
        if (kb == kb0 || (kb & 3) == 0) {                        // a new 512-element scale buffer
          const uint32_t b = ns % kScaleBufs, use = ns / kScaleBufs;
          if (!wait_spin(smem_u32(&sempty[b]), (use & 1u) ^ 1u, abort_flag)) {
            raise_abort(abort_flag, p.error);
            break;
          }
          const uint32_t lb = smem_u32(&sload[b]);
          uint8_t* dst = sScale + b * C::kScaleBytes;
          mbar_expect_tx(lb, (uint32_t)(512 * (1 + x_atoms)));
          bulk_load(smem_u32(dst), p.b_sf + ((size_t)nt * p.g4 + (kb >> 2)) * 512, 512u, lb);
          for (int i = 0; i < x_atoms; ++i)
            bulk_load(smem_u32(dst + 512 * (1 + i)),
                      p.a_sf + ((size_t)(mt * C::kXAtoms + i) * p.g4 + (kb >> 2)) * 512, 512u, lb);
          ++ns;
        }
        if (!wait_spin(smem_u32(&empty[stage]), (lap & 1u) ^ 1u, abort_flag)) {
          raise_abort(abort_flag, p.error);
          break;
        }
        const uint32_t fb = smem_u32(&full[stage]);
        mbar_expect_tx(fb, (uint32_t)C::kStageBytes);
        tma_load_2d(smem_u32(sW + stage * C::kWBytes), &tmap_w, kb * kBK, nt * 128, fb);
        tma_load_2d(smem_u32(sX + stage * C::kXBytes), &tmap_x, kb * kBK, mt * BNT, fb);
        if (++stage == S) {
          stage = 0;
          ++lap;
        }
      }
      asked[0] = lap * S + (uint32_t)stage;
      asked[1] = ns;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer --
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0, ns = 0;
      bool ok = true, any_mma = false;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (kb == kb0 || (kb & 3) == 0) {
          if (!wait_spin(smem_u32(&sfull[ns % kScaleBufs]), (ns / kScaleBufs) & 1u, abort_flag)) {
            raise_abort(abort_flag, p.error);
            ok = false;
            break;
          }
          ++ns;
        }
        if (!wait_spin(smem_u32(&full[stage]), phase, abort_flag)) {
          raise_abort(abort_flag, p.error);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t b = (ns - 1) % kScaleBufs;
        const uint32_t sw = tmem + C::kScaleCol + b * C::kScaleCols, sx = sw + 4u;
        const uint64_t wdesc = desc_sw128(smem_u32(sW + stage * C::kWBytes));
        const uint64_t xdesc = desc_sw128(smem_u32(sX + stage * C::kXBytes));
        const uint32_t idesc = fp8_idesc(128, BNT, p.b_type, p.a_type, (uint32_t)(kb & 3));
#pragma unroll
        for (int j = 0; j < 4; ++j)
          fp8_mma(tmem, wdesc + (uint64_t)(2 * j), xdesc + (uint64_t)(2 * j), idesc, sw, sx, (kb > kb0 || j > 0) ? 1u : 0u);
        any_mma = true;
        tc_commit(smem_u32(&empty[stage]));
        if ((kb & 3) == 3 || kb + 1 == kb1) tc_commit(smem_u32(&sempty[b]));
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok) {
        tc_commit(smem_u32(tfull));
      } else if (any_mma) {
        // the MMAs already issued end before tensor memory is released
        tc_commit(smem_u32(drain));
        volatile int never = 0;
        wait_bounded(smem_u32(drain), 0u, &never);
      }
    }
    __syncwarp();
  } else if (warp == 6) {
    // -------------------------------------------------------- scale copies --
    if (elect_one()) {
      uint32_t ns = 0;
      bool ok = true, any_cp = false;
      for (int kb = kb0; kb < kb1; kb = (kb & ~3) + 4, ++ns) {
        const uint32_t b = ns % kScaleBufs;
        if (!wait_spin(smem_u32(&sload[b]), (ns / kScaleBufs) & 1u, abort_flag)) {
          raise_abort(abort_flag, p.error);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sw = tmem + C::kScaleCol + b * C::kScaleCols;
        uint8_t* src = sScale + b * C::kScaleBytes;
#pragma unroll
        for (int i = 0; i <= C::kXAtoms; ++i) tc_cp_sf(sw + 4u * i, desc_sf(smem_u32(src + 512 * i)));
        tc_commit(smem_u32(&sfull[b]));
        any_cp = true;
      }
      if (!ok && any_cp) {
        tc_commit(smem_u32(sdrain));
        volatile int never = 0;
        wait_bounded(smem_u32(sdrain), 0u, &never);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------- this CTA's share, one row per row of A --
    // warp w reads tensor-memory lanes 32 * (w % 4) .. + 31 (rows of B) and all BNT columns
    const int q = warp & 3;
    int ok = 1;
    if (lane == 0) ok = wait_bounded(smem_u32(tfull), 0u, abort_flag) ? 1 : 0;
    ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    if (PUSH) cluster_wait();               // the peers run
    if (!ok) {
      if (lane == 0) raise_abort(abort_flag, p.error);
    } else {
      tc_fence_after();
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // ring bytes last touched by the async proxy
      float* col = part + q * 32 + lane;
      const int n = q * 32 + lane, rows = p.M - mt * BNT, slice = slice_cols(split), owner = n / slice;
      uint32_t dst = 0;
      if (PUSH)
        dst = map_rank(smem_u32(recv) + (uint32_t)(((int)rank * BNT * slice + n - owner * slice) * 4), (uint32_t)owner);
      if (BNT == 16) {
        uint32_t r[16];
        tmem_ld16(tbase, r);
        asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]),
                     "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                     "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
        if (!CLUSTER) {
          store_lane<16, BF16>(p, r, mt * BNT, nt * 128 + n);
        } else if (PUSH) {
          push_lane<16>(dst, r, 0, rows, slice);
        } else {
#pragma unroll
          for (int m = 0; m < 16; ++m) col[m * C::kPStride] = __uint_as_float(r[m]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < BNT / 32; ++c) {
          uint32_t r[32];
          tmem_ld32(tbase + (uint32_t)(32 * c), r);
          asm volatile("tcgen05.wait::ld.sync.aligned;"
                       : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                         "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                         "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                         "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                         "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
          if (!CLUSTER) {
            store_lane<32, BF16>(p, r, mt * BNT + 32 * c, nt * 128 + n);
          } else if (PUSH) {
            push_lane<32>(dst, r, 32 * c, rows, slice);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) col[(32 * c + i) * C::kPStride] = __uint_as_float(r[i]);
          }
        }
      }
    }
  }
  // ------------------------------------------- add one slice over the cluster --
  tc_fence_before();
  if (PUSH) {
    __syncwarp();
    if (warp < 2 || warp == 6) cluster_wait();
    cluster_sync_all();                     // every share of this CTA's columns is in its memory
    const int slice = slice_cols(split), c0 = (int)rank * slice, rows = min(BNT, p.M - mt * BNT);
    const int c4n = (min(min(128, p.N - nt * 128), c0 + slice) - c0 + 3) / 4;
    const int across = slice / 4, c4 = (int)threadIdx.x % across, down = C::kThreads / across;
    if (c4 < c4n && (int)threadIdx.x < down * across)
      for (int r = (int)threadIdx.x / across; r < rows; r += down) {
        const float* src = recv + r * slice + 4 * c4;
        float4 acc = *reinterpret_cast<const float4*>(src);
        for (int s = 1; s < split; ++s) acc = add4(acc, *reinterpret_cast<const float4*>(src + s * BNT * slice));
        store4<BF16>(p, acc, mt * BNT + r, nt * 128 + c0 + 4 * c4);
      }
  } else if (CLUSTER) {
    __syncthreads();
    cluster_sync_all();                     // every CTA's share is in its shared memory
    const int rows = min(BNT, p.M - mt * BNT), nvalid = min(128, p.N - nt * 128);
    const int c4n = (nvalid + 3) / 4;                              // groups of four columns of Y
    const int items = rows * c4n;
    const int i0 = (int)((int64_t)items * rank / split), i1 = (int)((int64_t)items * (rank + 1) / split);
    const uint32_t part_base = smem_u32(part);
    for (int it = i0 + (int)threadIdx.x; it < i1; it += (int)blockDim.x) {
      const int r = it / c4n, c4 = it - r * c4n;
      const uint32_t addr = part_base + (uint32_t)((r * C::kPStride + 4 * c4) * 4);
      float4 v[kMaxSplit];                                         // all remote loads in flight at once
#pragma unroll
      for (int s = 0; s < kMaxSplit; ++s)
        if (s < split) v[s] = ld_cluster_f4(map_rank(addr, (uint32_t)s));
      float4 acc = v[0];
#pragma unroll
      for (int s = 1; s < kMaxSplit; ++s)
        if (s < split) acc = add4(acc, v[s]);
      store4<BF16>(p, acc, mt * BNT + r, nt * 128 + 4 * c4);
    }
    cluster_sync_all();                     // no CTA leaves while a peer may still read its share
  }
  tc_fence_after();
  __syncthreads();
  // where a wait ran out, its own or another warp's, the producer's copies still land before the CTA goes
  if (__builtin_expect(*abort_flag != 0, 0) && threadIdx.x == 0 && settle_copies(full, S, asked[0]))
    settle_copies(sload, kScaleBufs, asked[1]);
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
  }
}

}  // namespace tiles

// ------------------------------------------------------ 256 x TN over SM pairs --
// A cluster of two CTAs on neighbouring SMs computes 256 x TN of Y with M = 256, N = TN MMAs issued by the
// even CTA.  Each CTA stages its 128 rows of A, half of B's TN rows and the scales of its A rows and of all B
// rows; both CTAs' loads signal the even CTA's barriers, whose MMA commits reach both.  Persistent: one cluster
// an SM pair walks the tiles.
//
// TN = 256: shared memory delivers 128 bytes a clock and SM; a block's operands, (128 + TN / 2) * 128 bytes, are
// written to it once and read once, in the 2 TN cycles of its MMAs: all of it at 256, which wider tiles would
// relieve and narrower ones overrun.  One accumulator (two would leave no columns for the scales); it is free
// for the next tile as soon as its columns are in the epilogue warps' registers.
// TN = 192: two accumulators, so that a tile is drained and stored while the next one is computed.  The 2700
// cycles from a 256-column tile's last MMA to the next tile's first are as long as five blocks of K, and more
// than the narrower tile's operands cost while K is short.
//
// warp 0 TMA producer, warp 1 MMA issuer, warps 2-9 epilogue, warp 10 scale copies.
namespace pairs {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 96 + 32 * kEpiWarps;
constexpr int kScaleWarp = 2 + kEpiWarps;
constexpr int kScaleBytes = 3 * 512;                   // A's atom, B's two
constexpr uint32_t kCols = 512, kScaleCols = 16;       // tensor memory columns, of them a scale buffer's
constexpr int kStageRows = 2048;                       // bytes an epilogue warp passes its rows through

template <int TN>
struct Cfg {
  static constexpr int kAccs = TN == 256 ? 1 : 2;
  static constexpr int kA = 128 * kBK, kB = TN / 2 * kBK;        // bytes of A, and of B, a CTA stages per block
  static constexpr int kStageBytes = kA + kB;
  static constexpr int kFixed = (int)kScaleBufs * kScaleBytes + kEpiWarps * kStageRows + 512;
  static constexpr int kStages = (226 * 1024 - 1024 - kFixed) / kStageBytes;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kFixed;
  static constexpr uint32_t kScaleCol = kAccs * TN;              // scale buffers behind the accumulators
  static_assert((TN == 256 || TN == 192) && kScaleCol + kScaleBufs * kScaleCols <= kCols, "tile width");
};

__device__ __forceinline__ void fp8_mma_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}

// 64 bytes' worth of columns of 32 rows of a tile from (m0, n0), lane = row: through 2 KB of shared memory (16-byte
// piece j of row r at j ^ (r / 2 mod 4): no bank conflicts either way), so that four lanes store 64 contiguous
// bytes of a row.  Measured against it: 16 bytes a lane straight from the registers (32 lines an instruction;
// 50432 x 2304 x 768 136 against 93 us), 32 bytes a lane (96 us), TMA stores (92 us, but 2048 x 2048 x 512 8.0
// against 7.6).  The columns are r[COL] on.
template <bool BF16, int COL>
__device__ __forceinline__ void store_rows(const Fp8KernelArgs& p, uint32_t stage, const uint32_t (&r)[32], int m0, int n0,
                                           int lane) {
  constexpr int kEl = BF16 ? 2 : 4, kPer = 16 / kEl;                // bytes of an element, elements of a piece
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4 v;
    if (BF16) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(r[8 * j + 2 * i]))) |
               ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(r[8 * j + 2 * i + 1]))) << 16);
      v = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      v = make_uint4(r[COL + 4 * j], r[COL + 4 * j + 1], r[COL + 4 * j + 2], r[COL + 4 * j + 3]);
    }
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)), "r"(v.x),
                 "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
  }
  __syncwarp();
  const int piece = lane & 3, n = n0 + piece * kPer, row0 = lane >> 2;
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                 : "r"(stage + (row0 + 8 * i) * 64 + ((piece ^ ((row0 >> 1) & 3)) << 4))
                 : "memory");
  __syncwarp();
  uint8_t* y = static_cast<uint8_t*>(p.y) + ((long long)(m0 + row0) * p.ldy + n) * kEl;
  if (p.vec_store && n + kPer <= p.N) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (m0 + row0 + 8 * i < p.M) *reinterpret_cast<uint4*>(y + 8 * i * p.ldy * kEl) = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (n + e < p.N && m0 + row0 + 8 * i < p.M) {
          if (BF16) reinterpret_cast<uint16_t*>(y + 8 * i * p.ldy * kEl)[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
          else reinterpret_cast<uint32_t*>(y + 8 * i * p.ldy * kEl)[e] = w[e];
        }
    }
  }
}

template <int TN, bool BF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fp8_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                         const __grid_constant__ CUtensorMap tmap_sa, const __grid_constant__ CUtensorMap tmap_sb,
                         Fp8KernelArgs p) {
  using C = Cfg<TN>;
  constexpr int S = C::kStages;
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + S * C::kA;
  uint8_t* sOut = sB + S * C::kB;
  uint8_t* sScale = sOut + kEpiWarps * kStageRows;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sScale + kScaleBufs * kScaleBytes);
  uint64_t* full = bars;
  uint64_t* empty = full + S;
  uint64_t* sload = empty + S;                          // scale buffer in both CTAs' shared memory
  uint64_t* sfull = sload + kScaleBufs;                 // ... in tensor memory
  uint64_t* sempty = sfull + kScaleBufs;                // ... read by its last MMA
  uint64_t* tfull = sempty + kScaleBufs;
  uint64_t* tempty = tfull + C::kAccs;
  uint64_t* drain = tempty + C::kAccs;
  uint64_t* sdrain = drain + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sdrain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  PairEnd* end = reinterpret_cast<PairEnd*>(tmem_slot + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    prefetch_map(&tmap_a);
    prefetch_map(&tmap_b);
    prefetch_map(&tmap_sa);
    prefetch_map(&tmap_sb);
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (uint32_t b = 0; b < kScaleBufs; ++b) {
      mbar_init(smem_u32(&sload[b]), 1);
      mbar_init(smem_u32(&sfull[b]), 1);
      mbar_init(smem_u32(&sempty[b]), 1);
    }
    for (int a = 0; a < C::kAccs; ++a) {
      mbar_init(smem_u32(&tfull[a]), 1);
      mbar_init(smem_u32(&tempty[a]), 2 * kEpiWarps);
    }
    mbar_init(smem_u32(drain), 1);
    mbar_init(smem_u32(sdrain), 1);
    *abort_flag = 0;
    pair_end_init(end);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_sync_all();                  // barriers of both CTAs initialised before any remote signal
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();                          // the previous kernel's outputs (our operands) are complete

  const int num_tiles = p.num_m * p.num_n;
  const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
  const int nkb = (p.K + kBK - 1) / kBK;

  if (warp == 0) {
    // ------------------------------------------------------------ producer --
    if (elect_one()) {
      int stage = 0;
      uint32_t lap = 0, ns = 0;                                // rounds of the ring, scale copies asked for
      bool ok = true;
      for (int t = cluster; t < num_tiles && ok; t += nclusters) {
        int mt, nt;
        tile_coords(t, p.num_m, p.num_n, mt, nt);
        for (int kb = 0; kb < nkb; ++kb) {
          if ((kb & 3) == 0) {                                 // a new 512-element scale buffer
            const uint32_t b = ns % kScaleBufs, use = ns / kScaleBufs;
            if (!wait_spin(smem_u32(&sempty[b]), (use & 1u) ^ 1u, abort_flag)) {
              raise_abort(abort_flag, p.error);
              ok = false;
              break;
            }
            const uint32_t lb = map_rank(smem_u32(&sload[b]), 0);
            const uint32_t dst = smem_u32(sScale + b * kScaleBytes);
            if (leader) mbar_expect_tx(smem_u32(&sload[b]), 2u * (uint32_t)kScaleBytes);
            tma_load_2d_pair(dst, &tmap_sa, 0, (mt * 2 + (int)rank) * p.g4 + (kb >> 2), lb);
            const int atom = nt * TN / 128;                    // B's first atom (192: its rows may start in the middle)
            tma_load_2d_pair(dst + 512, &tmap_sb, 0, atom * p.g4 + (kb >> 2), lb);
            tma_load_2d_pair(dst + 1024, &tmap_sb, 0, (atom + 1) * p.g4 + (kb >> 2), lb);
            ++ns;
          }
          if (!wait_spin(smem_u32(&empty[stage]), (lap & 1u) ^ 1u, abort_flag)) {
            raise_abort(abort_flag, p.error);
            ok = false;
            break;
          }
          const uint32_t fb = map_rank(smem_u32(&full[stage]), 0);
          if (leader) mbar_expect_tx(smem_u32(&full[stage]), 2u * (uint32_t)C::kStageBytes);
          tma_load_2d_pair(smem_u32(sA + stage * C::kA), &tmap_a, kb * kBK, mt * 256 + (int)rank * 128, fb);
          tma_load_2d_pair(smem_u32(sB + stage * C::kB), &tmap_b, kb * kBK, nt * TN + (int)rank * (TN / 2), fb);
          if (++stage == S) {
            stage = 0;
            ++lap;
          }
        }
      }
      pair_end_asked(end, rank, lap * S + (uint32_t)stage, ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------- MMA issuer (leader) --
    if (leader && elect_one()) {
      int stage = 0;
      uint32_t phase = 0, ns = 0, local = 0;
      bool ok = true, any_mma = false;
      for (int t = cluster; t < num_tiles && ok; t += nclusters, ++local) {
        const uint32_t acc = local % C::kAccs;
        if (!wait_spin(smem_u32(&tempty[acc]), ((local / C::kAccs) & 1u) ^ 1u, abort_flag)) {
          raise_abort(abort_flag, p.error);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + acc * TN;
        int mt, nt;
        tile_coords(t, p.num_m, p.num_n, mt, nt);
        const uint32_t sb_off = 4u + (((uint32_t)(nt * TN) >> 5) & 3u);       // B's first row in its atom, 32 a column
        for (int kb = 0; kb < nkb; ++kb) {
          if ((kb & 3) == 0) {
            if (!wait_spin(smem_u32(&sfull[ns % kScaleBufs]), (ns / kScaleBufs) & 1u, abort_flag)) {
              raise_abort(abort_flag, p.error);
              ok = false;
              break;
            }
            ++ns;
          }
          if (!wait_spin(smem_u32(&full[stage]), phase, abort_flag)) {
            raise_abort(abort_flag, p.error);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t b = (ns - 1) % kScaleBufs;
          const uint32_t sa = tmem + C::kScaleCol + b * kScaleCols, sb = sa + sb_off;
          const uint64_t adesc = desc_sw128(smem_u32(sA + stage * C::kA));
          const uint64_t bdesc = desc_sw128(smem_u32(sB + stage * C::kB));
          const uint32_t idesc = fp8_idesc(256, TN, p.a_type, p.b_type, (uint32_t)(kb & 3));
#pragma unroll
          for (int j = 0; j < 4; ++j)
            fp8_mma_pair(d, adesc + (uint64_t)(2 * j), bdesc + (uint64_t)(2 * j), idesc, sa, sb,
                         (kb > 0 || j > 0) ? 1u : 0u);
          any_mma = true;
          tc_commit_pair(smem_u32(&empty[stage]));
          if ((kb & 3) == 3 || kb + 1 == nkb) tc_commit_pair(smem_u32(&sempty[b]));
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit_pair(smem_u32(&tfull[acc]));
      }
      if (!ok && any_mma) {
        // the MMAs already issued end before tensor memory is released
        tc_commit_pair_local(smem_u32(drain));
        volatile int never = 0;
        wait_bounded(smem_u32(drain), 0u, &never);
      }
    }
    __syncwarp();
  } else if (warp == kScaleWarp) {
    // ------------------------------------------------ scale copies (leader) --
    // cta_group::2 copies fill the same columns of both CTAs' tensor memory, each from its own shared memory
    if (leader && elect_one()) {
      uint32_t ns = 0;
      bool ok = true, any_cp = false;
      for (int t = cluster; t < num_tiles && ok; t += nclusters) {
        for (int kb = 0; kb < nkb; kb += 4, ++ns) {
          const uint32_t b = ns % kScaleBufs;
          if (!wait_spin(smem_u32(&sload[b]), (ns / kScaleBufs) & 1u, abort_flag)) {
            raise_abort(abort_flag, p.error);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = tmem + C::kScaleCol + b * kScaleCols;
#pragma unroll
          for (int i = 0; i < 3; ++i)
            tc_cp_sf_pair(sa + 4u * i, desc_sf(smem_u32(sScale + b * kScaleBytes + 512 * i)));
          tc_commit_pair_local(smem_u32(&sfull[b]));
          any_cp = true;
        }
      }
      if (!ok && any_cp) {
        tc_commit_pair_local(smem_u32(sdrain));
        volatile int never = 0;
        wait_bounded(smem_u32(sdrain), 0u, &never);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue --
    // warp w: tensor-memory lanes 32 * (w % 4) .. + 31 and half of the tile's columns
    const int q = warp & 3;
    const int col0 = ((warp - 2) / 4) * (TN / 2);
    const uint32_t stage = smem_u32(sOut + (warp - 2) * kStageRows);
    const uint32_t tempty_leader = map_rank(smem_u32(tempty), 0);
    uint32_t local = 0;
    for (int t = cluster; t < num_tiles; t += nclusters, ++local) {
      int mt, nt;
      tile_coords(t, p.num_m, p.num_n, mt, nt);
      const uint32_t acc = local % C::kAccs;
      int ok = 1;
      if (lane == 0) ok = wait_bounded(smem_u32(&tfull[acc]), (local / C::kAccs) & 1u, abort_flag) ? 1 : 0;
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (!ok) {
        if (lane == 0) raise_abort(abort_flag, p.error);
        break;
      }
      tc_fence_after();
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + acc * TN + (uint32_t)col0;
      uint32_t r[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c < TN / 64) {
          tmem_ld32(tbase + (uint32_t)(32 * c), r[c]);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) r[c][i] = 0u;
        }
      }
      tmem_ld_wait(r);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(tempty_leader + 8u * acc);
      const int m0 = mt * 256 + (int)rank * 128 + q * 32, n0 = nt * TN + col0;
#pragma unroll
      for (int c = 0; c < TN / 64; ++c) {
        store_rows<BF16, 0>(p, stage, r[c], m0, n0 + 32 * c, lane);
        if (!BF16) store_rows<BF16, 16>(p, stage, r[c], m0, n0 + 32 * c + 16, lane);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // an MMA warp that ends its tiles has seen every copy land; where a wait of the leader's ran out, those in
  // flight are waited for
  if (leader && threadIdx.x == 0 && *abort_flag != 0) pair_end_halt(end);
  __syncwarp();
  cluster_sync_all();                  // neither CTA frees tensor memory or exits while the pair is busy
  if (__builtin_expect(pair_halted(end), 0)) {
    if (leader && threadIdx.x == 0 && settle_pair_copies(full, S, end, 0, C::kStageBytes))
      settle_pair_copies(sload, kScaleBufs, end, 1, kScaleBytes);
    __syncwarp();
    cluster_sync_all();
  }
  tc_fence_after();
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
  }
}

}  // namespace pairs

// ------------------------------------------------------------------ host ---
// [rows, k] bytes with row pitch ld: boxes of 128 bytes x box_rows, 128B swizzle.  The map ends at k, so
// the elements of the last block that lie past it read as zero whatever the row's padding holds.
bool code_map(CUtensorMap* map, const uint8_t* base, int64_t rows, int64_t k, int64_t ld, int box_rows) {
  auto enc = encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld};
  cuuint32_t box[2] = {(cuuint32_t)kBK, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

Fp8KernelArgs kernel_args(const Fp8GemmParams& q) {
  Fp8KernelArgs p;
  p.a_sf = q.a_sf;
  p.b_sf = q.b_sf;
  p.y = q.y;
  p.ldy = q.ldy;
  p.M = (int)q.M;
  p.N = (int)q.N;
  p.K = (int)q.K;
  p.num_m = p.num_n = 0;
  p.g4 = (int)((fp8_groups(q.K) + 3) / 4);
  p.a_type = (uint32_t)q.a_fmt;
  p.b_type = (uint32_t)q.b_fmt;
  const int64_t esz = q.y_bf16 ? 2 : 4;
  p.vec_store = (q.ldy * esz) % 16 == 0 && (reinterpret_cast<uintptr_t>(q.y) & 15u) == 0;
  p.error = q.error;
  return p;
}

// Clusters of `split` CTAs of this kernel that the device holds at once (0 if unknown).
template <int BNT, bool BF16>
int max_clusters(int split) {
  using C = tiles::Cfg<BNT>;
  static std::mutex mu;
  static int cache[tiles::kMaxSplit + 1] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (cache[split] == 0) {
    auto kernel = tiles::fp8_gemm_tile_kernel<BNT, BF16, true>;
    int n = 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split);
    cfg.blockDim = dim3((unsigned)C::kThreads);
    cfg.dynamicSmemBytes = (size_t)C::kSmem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)split;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) n = -1;
    cache[split] = n;
  }
  return cache[split] > 0 ? cache[split] : 0;
}

template <int BNT, bool BF16>
cudaError_t run_tiles(const Fp8GemmParams& q, int num_sms, cudaStream_t st) {
  using C = tiles::Cfg<BNT>;
  static_assert((C::kPush ? C::kPushStages : C::kStages) >= 2 && C::kSmem <= 227 * 1024, "shared memory");
  auto alone = tiles::fp8_gemm_tile_kernel<BNT, BF16, false>, together = tiles::fp8_gemm_tile_kernel<BNT, BF16, true>;
  static SmemLimit limit[2];
  cudaError_t attr = limit[0].raise(alone, C::kSmem);
  if (attr == cudaSuccess) attr = limit[1].raise(together, C::kSmem);
  if (attr != cudaSuccess) return attr;
  CUtensorMap tw, tx;
  if (!code_map(&tw, q.b, q.N, q.K, q.ldb, 128)) return cudaErrorNotSupported;
  if (!code_map(&tx, q.a, q.M, q.K, q.lda, BNT)) return cudaErrorNotSupported;
  Fp8KernelArgs p = kernel_args(q);
  p.num_m = (int)((q.M + BNT - 1) / BNT);
  p.num_n = (int)((q.N + 127) / 128);
  const int64_t n = (int64_t)p.num_m * p.num_n, nkb = fp8_groups(q.K);
  // as many CTAs a tile as leave at most one CTA a SM, none without a block of K, and every cluster
  // resident at once
  int64_t split = std::max<int64_t>(1, std::min<int64_t>({num_sms / n, (int64_t)tiles::kMaxSplit, nkb}));
  while (split > 1 && n > max_clusters<BNT, BF16>((int)split)) --split;
  return launch_kernel(split > 1 ? together : alone, dim3((unsigned)(n * split)), dim3(C::kThreads), C::kSmem, st, false,
                       (unsigned)split, tw, tx, p, (int)split);
}

// Scales in the tensor-core layout as rows of 512 bytes (one 128 x 4 atom), one atom a box.
bool scale_map(CUtensorMap* map, const uint8_t* base, int64_t atoms) {
  auto enc = encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {128, (cuuint64_t)atoms};
  cuuint64_t strides[1] = {512};
  cuuint32_t box[2] = {128, 1};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int TN, bool BF16>
cudaError_t run_pairs(const Fp8GemmParams& q, int num_sms, cudaStream_t st) {
  using C = pairs::Cfg<TN>;
  static_assert(C::kStages >= 2 && C::kSmem <= 227 * 1024, "shared memory");
  auto kernel = pairs::fp8_gemm_pair_kernel<TN, BF16>;
  static SmemLimit limit;
  const cudaError_t attr = limit.raise(kernel, C::kSmem);
  if (attr != cudaSuccess) return attr;
  Fp8KernelArgs p = kernel_args(q);
  CUtensorMap ta, tb, tsa, tsb;
  if (!code_map(&ta, q.a, q.M, q.K, q.lda, 128)) return cudaErrorNotSupported;
  if (!code_map(&tb, q.b, q.N, q.K, q.ldb, TN / 2)) return cudaErrorNotSupported;
  if (!scale_map(&tsa, q.a_sf, (q.M + 127) / 128 * p.g4)) return cudaErrorNotSupported;
  if (!scale_map(&tsb, q.b_sf, (q.N + 127) / 128 * p.g4)) return cudaErrorNotSupported;
  p.num_m = (int)((q.M + 255) / 256);
  p.num_n = (int)((q.N + TN - 1) / TN);
  const int clusters = std::min(num_sms / 2, p.num_m * p.num_n);
  return launch_kernel(kernel, dim3(2 * clusters), dim3(pairs::kThreads), C::kSmem, st, false, 1u, ta, tb, tsa, tsb, p);
}

template <bool BF16>
cudaError_t dispatch(const Fp8GemmParams& q, int num_sms, cudaStream_t st) {
  // Up to 128 rows of A: tiles of Y^T stream B over every SM (128 x 4096 x 4096: 10.1 against 12.8 us in SM pairs;
  // 128 x 11008 x 4096: 13.8 against 14.6; 128 x 32000 x 4096: 31.1 against 31.6).
  if (q.M > 128) {
    const int64_t num_m = (q.M + 255) / 256, narrow = num_m * ((q.N + 191) / 192), wide = num_m * ((q.N + 255) / 256);
    const int64_t pairs = num_sms / 2, narrow_waves = (narrow + pairs - 1) / pairs, wide_waves = (wide + pairs - 1) / pairs;
    // Few tiles and a long K: K divided over clusters (256 x 1024 x 8192, 6 tiles: 12.7 against 19.1 us; 512 x 1024 x
    // 4096, 12 tiles: 11.7 against 12.0; 256 x 4096 x 4096, 22 tiles: 13.8 against 13.0).
    if (8 * narrow <= num_sms && q.K >= 4096) return run_tiles<256, BF16>(q, num_sms, st);
    // A wave of 192 columns takes 0.70 to 0.78 of one of 256 from K = 1536 on and 0.80 to 0.84 at 768 (8192 x 11008 x
    // 4096: 26 waves in 257 us against 19 in 260; 4096 x 4096 x 2048: 5 in 27.9 against 4 in 30.4; 50432 x 2304 x 768:
    // 32 in 99.7 against 24 in 93.4).  Rows that start between 32-byte sectors cost a load a fifth sector, and narrow
    // tiles load more (4096 x 4096 x 8201 in rows of 8208 bytes: 5 waves in 151 us against 4 in 142).
    const bool sectors = q.lda % 32 == 0 && q.ldb % 32 == 0;
    if ((q.K >= 1536 && sectors ? 75 : 82) * narrow_waves <= 100 * wide_waves) return run_pairs<192, BF16>(q, num_sms, st);
    return run_pairs<256, BF16>(q, num_sms, st);
  }
  if (q.M <= 16) return run_tiles<16, BF16>(q, num_sms, st);
  if (q.M <= 32) return run_tiles<32, BF16>(q, num_sms, st);
  if (q.M <= 64) return run_tiles<64, BF16>(q, num_sms, st);
  return run_tiles<128, BF16>(q, num_sms, st);
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8GemmParams& q, int num_sms, cudaStream_t st) {
  return q.y_bf16 ? dispatch<true>(q, num_sms, st) : dispatch<false>(q, num_sms, st);
}

}  // namespace fp4lib
