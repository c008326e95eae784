// The end of an SM pair that stopped early, without the tensor cores: two CTAs ask for different numbers of copies
// (byte counts stand in for them), which land while the leader waits.  Every wait is bounded.
#include <cuda_runtime.h>

#include "gemm_device.cuh"

using namespace fp4tc;

namespace {

constexpr uint32_t kShare = 64;

__device__ void land(uint64_t* bar, uint32_t rank) {
  if (rank == 0) mbar_complete_tx(smem_u32(bar), kShare);
  else
    asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(map_rank(smem_u32(bar), 0)),
                 "r"(kShare)
                 : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(64)
    pair_settle_kernel(uint32_t slots, uint32_t done, uint32_t mine, uint32_t peers, uint32_t delay_ns, int* out) {
  __shared__ uint64_t bars[8];
  __shared__ PairEnd end;
  const uint32_t rank = cluster_rank();
  const uint32_t asked = rank == 0 ? mine : peers;
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < slots; ++s) mbar_init(smem_u32(&bars[s]), 1);
    pair_end_init(&end);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  cluster_sync_all();
  for (uint32_t n = 0; n < done; ++n) {                    // copies of both, landed and read
    if (threadIdx.x == 0) {
      if (rank == 0) mbar_expect_tx(smem_u32(&bars[n % slots]), 2 * kShare);
      land(&bars[n % slots], rank);
    }
    __syncwarp();
    cluster_sync_all();
  }
  if (threadIdx.x == 0) {
    if (rank == 0)
      for (uint32_t n = done; n < mine; ++n) mbar_expect_tx(smem_u32(&bars[n % slots]), 2 * kShare);
    pair_end_asked(&end, rank, asked, 0);
  }
  __syncwarp();
  cluster_sync_all();
  if (threadIdx.x == 32) {                                 // the shares land
    const uint64_t t0 = global_timer();
    while (global_timer() - t0 < delay_ns && delay_ns < 1000000u) {
    }
    for (uint32_t n = done; n < asked; ++n) land(&bars[n % slots], rank);
  }
  if (rank == 0 && threadIdx.x == 0) {
    int ok = settle_pair_copies(bars, slots, &end, 0, kShare) ? 1 : 0;
    const uint32_t most = mine > peers ? mine : peers;
    for (uint32_t n = fp4ring::first_open(most, slots); n < most; ++n)     // every phase is over, and no further one
      if (!mbar_try_wait(smem_u32(&bars[n % slots]), fp4ring::parity_of(n, slots))) ok = 0;
    out[0] = ok;
  }
  __syncwarp();
  cluster_sync_all();
}

}  // namespace

extern "C" int pair_settle(uint32_t slots, uint32_t done, uint32_t mine, uint32_t peers, uint32_t delay_ns, int* out) {
  if (slots < 1 || slots > 8 || mine < done || peers < done || mine > done + slots || peers > done + slots) return -1;
  pair_settle_kernel<<<2, 64>>>(slots, done, mine, peers, delay_ns, out);
  return (int)cudaGetLastError();
}
