// RMS norm with the residual's addition and 8-bit block-scaled output, and its backward pass.
//
//   h = bf16(x + residual)            (h = x without a residual; the stream is a bf16 tensor and the
//                                      norm is the norm of what the stream holds)
//   rstd = 1 / sqrt(mean(h^2) + eps)
//   y = (h * rstd) * weight           quantized along the row, 128 elements a block (fp8_device.cuh)
//
//   g = dy * weight, xh = h * rstd, c = mean(g * xh)
//   dx = rstd * (g - xh * c) + dresidual,  dweight = sum over rows of dy * xh
//
// Sums and statistics are fp32 or wider, y is fp32.  The squares, their sum and its root are fp64, where no finite row
// overflows or vanishes.  Against eight squares at a time in fp32, which made rows past 2^62.5 zero and rows near 1e-23
// NaN: 16384 x 4096 with a residual 75.3 -> 72.1 us, without one 45.7 -> 49.1; 4096 x 11008 60.2 -> 54.0; 50432 x 768
// 47.6 -> 48.0; 300 x 4096 6.7 -> 7.1 (inputs past L2).  Squares of values moved to fp64 by integer arithmetic, in place of the
// conversion, took longer (53.5 without a residual).
// The only roundings to fewer bits are the outputs' own.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "copy_ring.h"
#include "fp4_device.cuh"
#include "fp4_internal.h"
#include "fp8_device.cuh"
#include "fp8_internal.h"

namespace fp4lib {
namespace {

using namespace fp8dev;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(a)) |
         ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(b)) << 16);
}
__device__ __forceinline__ void load_weight8(const void* w, int f32, uint32_t chunk, float (&v)[8]) {
  if (f32) {
    const float4 a = reinterpret_cast<const float4*>(w)[2 * chunk], b = reinterpret_cast<const float4*>(w)[2 * chunk + 1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    fp4dev::unpack8(reinterpret_cast<const uint4*>(w)[chunk], v);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}
// Sum over the `warps` warps of a row (every thread of the block takes part; `part` holds one value per warp of
// the block).  Within the warp, then over the row's warps, in a fixed order.  WARP: the row is one warp's.
template <bool WARP>
__device__ __forceinline__ double row_sum64(double v, double* part, uint32_t first_warp, uint32_t warps) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = __dadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  if (!WARP) {
    const uint32_t lane = threadIdx.x & 31u;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? part[first_warp + lane] : 0.0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = __dadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  }
  return v;
}

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;
  const void* weight;
  long long rows, ldx, ldr, ldc;
  double eps, inv_cols;
  uint8_t* codes;
  uint8_t* scales;
  uint16_t* residual_out;
  uint16_t* norm_out;
  float* rstd;
  uint32_t cols, chunks, groups, main_ctas;
  uint32_t tpr, slots;          // threads of a row (a multiple of 32), rows of a block
  int weight_f32, sf_mma;
};

// tpr threads a row, CPT 8-element chunks a thread: the row stays in registers between the sum of
// squares and the quantization, so x and the residual are read once.  Bound by HBM (7 bytes an element
// with a residual; 16384 x 4096: 72 us, the copy rate); one row of few: by the latency of load -> sum ->
// store (2.6 us).  Two chunks a thread took 91 us, eight 122: a row's fixed work (some 150 instructions a thread) is
// spread over more elements, until the registers leave too few rows in flight.  Rows of up to 1024 elements are one
// warp's, eight a block, and nothing waits for another warp.  MOST, BLOCKS: threads of a block, blocks an SM;
// three blocks of up to 384 threads (56 registers) against two took 4096 x 11008 from 70.7 to 59.9 us (54.0 now).
constexpr int kShortThreads = 256;
template <int FMT, int CPT, int MOST, int BLOCKS>
__global__ void __launch_bounds__(MOST, BLOCKS) rmsnorm_fp8_kernel(NormArgs p) {
  constexpr bool WARP = MOST == kShortThreads;
  __shared__ double part[32];
  pdl_trigger();
  const uint32_t TPR = WARP ? 32u : p.tpr;
  const uint32_t slot = WARP ? threadIdx.x >> 5 : threadIdx.x / TPR, t = threadIdx.x - slot * TPR;
  pdl_wait();
  if (blockIdx.x >= p.main_ctas) {
    zero_pad_rows(p.scales, p.rows, p.groups);
    return;
  }
  const long long row = (long long)blockIdx.x * p.slots + slot;
  const bool live = row < p.rows;
  bool on[CPT];
  uint4 h[CPT];
  const uint16_t* x = p.x + row * p.ldx + t * 8;
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    on[k] = live && t + k * TPR < p.chunks;
    h[k] = make_uint4(0, 0, 0, 0);
    if (on[k]) h[k] = *reinterpret_cast<const uint4*>(x + k * TPR * 8);
  }
  if (p.residual != nullptr) {
    uint4 r[CPT];
    const uint16_t* res = p.residual + row * p.ldr + t * 8;
    uint16_t* out = p.residual_out + row * p.cols + t * 8;
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      r[k] = make_uint4(0, 0, 0, 0);
      if (on[k]) r[k] = *reinterpret_cast<const uint4*>(res + k * TPR * 8);
    }
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      float2 a[4], b[4];
      unpack2(h[k], a);
      unpack2(r[k], b);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = fp4dev::add2(a[i], b[i]);
      h[k] = make_uint4(pack_bf16(a[0].x, a[0].y), pack_bf16(a[1].x, a[1].y), pack_bf16(a[2].x, a[2].y),
                        pack_bf16(a[3].x, a[3].y));
      if (on[k]) *reinterpret_cast<uint4*>(out + k * TPR * 8) = h[k];
    }
  }
  // squares of bf16 are exact in fp64 and neither overflow nor vanish there
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    float2 a[4];
    unpack2(h[k], a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum = __fma_rn((double)a[i].x, (double)a[i].x, sum);
      sum = __fma_rn((double)a[i].y, (double)a[i].y, sum);
    }
  }
  const double ss = row_sum64<WARP>(sum, part, slot * (TPR / 32), TPR / 32);
  const float rstd = (float)rsqrt(__fma_rn(ss, p.inv_cols, p.eps));
  if (live && t == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
  const float2 r2 = make_float2(rstd, rstd);
  float2 y[CPT][4];
  uint32_t m[CPT];
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    unpack2(h[k], y[k]);
    float am = 0.0f;
    if (on[k]) {
      float w[8];
      load_weight8(p.weight, p.weight_f32, t + k * TPR, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[k][i] = __fmul2_rn(__fmul2_rn(y[k][i], r2), make_float2(w[2 * i], w[2 * i + 1]));
        am = max_abs3(am, y[k][i].x, y[k][i].y);
      }
    }
    m[k] = __float_as_uint(am) & 0x7FFFFFFFu;
  }
  float inv[CPT];
  int own;
  bool stores;
  const uint32_t byte = block_scales<FMT>(m, inv, own, stores);
  uint8_t* codes = p.codes + row * p.ldc + t * 8;
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    if (on[k]) {
      *reinterpret_cast<uint2*>(codes + k * TPR * 8) = codes8<FMT>(y[k], inv[k]);
      if (p.norm_out != nullptr)
        *reinterpret_cast<uint4*>(p.norm_out + row * p.cols + (t + k * TPR) * 8) =
            make_uint4(pack_bf16(y[k][0].x, y[k][0].y), pack_bf16(y[k][1].x, y[k][1].y),
                       pack_bf16(y[k][2].x, y[k][2].y), pack_bf16(y[k][3].x, y[k][3].y));
    }
  }
  const uint32_t g = (t + own * TPR) >> 4;
  if (stores && live && own < CPT && g < p.groups) {
    uint8_t* out = p.scales + sf_offset(p.sf_mma, row, g, p.groups);
    *out = (uint8_t)byte;
    if (p.sf_mma && g + 1 == p.groups)                              // groups that pad the layout to 4
      for (uint32_t k = 1; (g + k) & 3u; ++k) out[k] = 0;
  }
}

struct NormBwdArgs {
  const uint16_t* dy;
  const uint16_t* h;
  const void* weight;
  const float* rstd;
  const uint16_t* dres;
  uint16_t* dx;
  float* partials;
  long long rows, lddy, ldh, lddr;
  float inv_cols;
  uint32_t cols, chunks, tpr, slots;
  int weight_f32;
};

// Writes the block's row of `partials`: eight columns of each chunk.
template <int CPT>
__device__ __forceinline__ void store_partials(const NormBwdArgs& p, const float2 (&acc)[CPT][4], uint32_t t, uint32_t tpr) {
#pragma unroll
  for (int k = 0; k < CPT; ++k)
    if (t + k * tpr < p.chunks) {
      float* o = p.partials + (long long)blockIdx.x * p.cols + (t + k * tpr) * 8;
      reinterpret_cast<float4*>(o)[0] = make_float4(acc[k][0].x, acc[k][0].y, acc[k][1].x, acc[k][1].y);
      reinterpret_cast<float4*>(o)[1] = make_float4(acc[k][2].x, acc[k][2].y, acc[k][3].x, acc[k][3].y);
    }
}

// Rows of up to 1024 elements: a warp a row, eight rows a block.  A warp walks its rows with the next one's
// loads issued before this one's sum and keeps its columns' sums of dy * xh in registers.  Bound by HBM (50432 x 768
// with a residual: 58 us, 0.83 of the copy rate; rows over 64 threads with a barrier each took 125).
template <int CPT>
__global__ void __launch_bounds__(256, 2) rmsnorm_backward_short_kernel(NormBwdArgs p) {
  extern __shared__ float2 slot_sums[];             // [7][4][chunks]
  pdl_trigger();
  const uint32_t slot = threadIdx.x >> 5, t = threadIdx.x & 31u;
  const long long step = (long long)gridDim.x * p.slots;
  float2 acc[CPT][4];
#pragma unroll
  for (int k = 0; k < CPT; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[k][i] = make_float2(0.0f, 0.0f);
  pdl_wait();
  uint4 nd[CPT], nh[CPT];
  float nrstd = 0.0f;
  auto load = [&](long long row) {
    const bool live = row < p.rows;
    nrstd = live ? p.rstd[row] : 0.0f;
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const uint32_t c = t + k * 32;
      nd[k] = nh[k] = make_uint4(0, 0, 0, 0);
      if (live && c < p.chunks) {
        nd[k] = *reinterpret_cast<const uint4*>(p.dy + row * p.lddy + c * 8);
        nh[k] = *reinterpret_cast<const uint4*>(p.h + row * p.ldh + c * 8);
      }
    }
  };
  long long row = (long long)blockIdx.x * p.slots + slot;
  load(row);
  for (; row < p.rows; row += step) {
    const float2 r2 = make_float2(nrstd, nrstd);
    uint4 d[CPT], h[CPT], r4[CPT];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const uint32_t c = t + k * 32;
      d[k] = nd[k];
      h[k] = nh[k];
      r4[k] = make_uint4(0, 0, 0, 0);
      if (p.dres != nullptr && c < p.chunks) r4[k] = *reinterpret_cast<const uint4*>(p.dres + row * p.lddr + c * 8);
    }
    load(row + step);
    float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const uint32_t c = t + k * 32;
      if (c < p.chunks) {
        float2 a[4], b[4];
        float w[8];
        unpack2(d[k], a);
        unpack2(h[k], b);
        load_weight8(p.weight, p.weight_f32, c, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 xh = __fmul2_rn(b[i], r2);
          s2 = __ffma2_rn(__fmul2_rn(a[i], make_float2(w[2 * i], w[2 * i + 1])), xh, s2);
          acc[k][i] = __ffma2_rn(a[i], xh, acc[k][i]);
        }
      }
    }
    const float sum = warp_sum(__fadd_rn(s2.x, s2.y));
    // dx = g * rstd + (xh * (-rstd * c) + dresidual)
    const float kf = __fmul_rn(-r2.x, __fmul_rn(sum, p.inv_cols));
    const float2 k2 = make_float2(kf, kf);
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const uint32_t c = t + k * 32;
      if (c < p.chunks) {
        float2 a[4], b[4], e[4];
        float w[8];
        unpack2(d[k], a);
        unpack2(h[k], b);
        unpack2(r4[k], e);
        load_weight8(p.weight, p.weight_f32, c, w);
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = __ffma2_rn(__fmul2_rn(a[i], make_float2(w[2 * i], w[2 * i + 1])), r2,
                                      __ffma2_rn(__fmul2_rn(b[i], r2), k2, e[i]));
          o[i] = pack_bf16(v.x, v.y);
        }
        *reinterpret_cast<uint4*>(p.dx + row * p.cols + c * 8) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  // the eight warps' sums, in order
#pragma unroll
  for (int k = 0; k < CPT; ++k)
    if (slot > 0 && t + k * 32 < p.chunks)
#pragma unroll
      for (int i = 0; i < 4; ++i) slot_sums[((slot - 1) * 4 + i) * p.chunks + t + k * 32] = acc[k][i];
  __syncthreads();
  if (slot > 0) return;
#pragma unroll
  for (int k = 0; k < CPT; ++k)
    if (t + k * 32 < p.chunks)
      for (uint32_t j = 0; j + 1 < p.slots; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[k][i] = fp4dev::add2(acc[k][i], slot_sums[(j * 4 + i) * p.chunks + t + k * 32]);
  store_partials<CPT>(p, acc, t, 32);
}

// Longer rows: a block takes R rows at a time, CPT = 2 chunks a thread.  Rows arrive in a ring of shared-memory
// slots by bulk copies (one an array), so that what is in flight takes no registers, and are read from there
// twice, for the sum and for dx.  The sums of R rows share one barrier; behind it every thread has read the
// previous R rows, and their slots are filled again.  What a row costs a thread besides its elements (waits,
// shuffles, addresses: some 60 instructions) is why a thread takes 16 elements of it and not 8, and the
// arithmetic runs on packed pairs.  Bound by HBM (16384 x 4096 with a residual: 93 us, 0.90 of the copy rate; a block
// a row with everything in registers took 106, eight elements a thread 155).
template <int R>
__global__ void __launch_bounds__(1024) rmsnorm_backward_long_kernel(NormBwdArgs p, int ring_rows, unsigned* error) {
  constexpr int CPT = 2;
  extern __shared__ __align__(128) uint8_t ring[];              // [ring_rows][arrays][cols] bf16, then the barriers
  __shared__ float part[2][R][32];
  pdl_trigger();
  const uint32_t t = threadIdx.x, TPR = p.tpr, warp = t >> 5, lane = t & 31u, warps = TPR / 32;
  const uint32_t row_bytes = p.cols * 2, arrays = p.dres != nullptr ? 3 : 2, slot_bytes = row_bytes * arrays;
  const uint32_t ring0 = fp4dev::smem_addr(ring), bar0 = ring0 + (uint32_t)ring_rows * slot_bytes;
  if (t == 0) {
    for (int s = 0; s < ring_rows; ++s) fp4dev::mbar_init(bar0 + 8 * s, 1);
    fp4dev::mbar_init_fence();
  }
  float2 acc[CPT][4], w[CPT][4];
#pragma unroll
  for (int k = 0; k < CPT; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[k][i] = w[k][i] = make_float2(0.0f, 0.0f);
  pdl_wait();
  __syncthreads();
  const int count = (int)((p.rows - blockIdx.x + gridDim.x - 1) / gridDim.x);      // rows blockIdx + n * gridDim
  int fetched = 0, fetch_slot = 0;                             // thread 0: rows asked for, the next one's slot
  long long fetch_row = blockIdx.x;
  auto fetch = [&] {
    const uint32_t bar = bar0 + 8 * fetch_slot, dst = ring0 + (uint32_t)fetch_slot * slot_bytes;
    fp4dev::mbar_expect_tx(bar, slot_bytes);
    fp4dev::bulk_g2s(dst, p.dy + fetch_row * p.lddy, row_bytes, bar);
    fp4dev::bulk_g2s(dst + row_bytes, p.h + fetch_row * p.ldh, row_bytes, bar);
    if (arrays == 3) fp4dev::bulk_g2s(dst + 2 * row_bytes, p.dres + fetch_row * p.lddr, row_bytes, bar);
    ++fetched;
    fetch_row += gridDim.x;
    if (++fetch_slot == ring_rows) fetch_slot = 0;
  };
  if (t == 0)
    while (fetched < ring_rows && fp4ring::may_ask(false, fetched, count)) fetch();
#pragma unroll
  for (int k = 0; k < CPT; ++k)
    if (t + k * TPR < p.chunks) {
      float v[8];
      load_weight8(p.weight, p.weight_f32, t + k * TPR, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[k][i] = make_float2(v[2 * i], v[2 * i + 1]);
    }
  uint16_t* out = p.dx + (long long)blockIdx.x * p.cols + t * 8;
  const long long out_step = (long long)gridDim.x * p.cols;
  // rstd of 32 rows a lane each, and of the 32 behind them: a load for each row, one row ahead, was what rows waited for
  auto rstd_of = [&](int n) { return n < count ? p.rstd[blockIdx.x + (long long)n * gridDim.x] : 0.0f; };
  float rs = rstd_of((int)lane), rs_next = rstd_of(32 + (int)lane);
  bool late = false;
  int slot = 0;
  uint32_t phase = 0;
  for (int n0 = 0, flip = 0; n0 < count; n0 += R, flip ^= 1) {
    float rstd[R], sum[R];
    uint32_t at[R];                                            // the rows' slots
    if ((n0 & 31) == 0 && n0 > 0) {
      rs = rs_next;
      rs_next = rstd_of(n0 + 32 + (int)lane);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) rstd[r] = __shfl_sync(0xFFFFFFFFu, rs, (n0 + r) & 31);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      sum[r] = 0.0f;
      at[r] = (uint32_t)slot * slot_bytes + t * 16;
      if (n0 + r < count) {
        if (!late && !fp4dev::mbar_wait_bounded(bar0 + 8 * slot, phase)) {
          late = true;                                         // reported; the remaining waits are skipped
          atomicOr(error, 1u);
        }
        if (++slot == ring_rows) {
          slot = 0;
          phase ^= 1u;
        }
        const float2 r2 = make_float2(rstd[r], rstd[r]);
        float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
          if (t + k * TPR < p.chunks) {
            float2 a[4], b[4];
            unpack2(*reinterpret_cast<const uint4*>(ring + at[r] + k * TPR * 16), a);
            unpack2(*reinterpret_cast<const uint4*>(ring + at[r] + row_bytes + k * TPR * 16), b);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 xh = __fmul2_rn(b[i], r2);
              s2 = __ffma2_rn(__fmul2_rn(a[i], w[k][i]), xh, s2);
              acc[k][i] = __ffma2_rn(a[i], xh, acc[k][i]);
            }
          }
        }
        sum[r] = __fadd_rn(s2.x, s2.y);
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) sum[r] += __shfl_xor_sync(0xFFFFFFFFu, sum[r], d);
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (lane == 0) part[flip][r][warp] = sum[r];
    __syncthreads();                                           // one barrier for R rows: two sets of sums
    if (t == 0 && n0 > 0)
      for (int r = 0; r < R && fp4ring::may_ask(late, fetched, count); ++r) fetch();
#pragma unroll
    for (int r = 0; r < R; ++r) sum[r] = lane < warps ? part[flip][r][lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) sum[r] += __shfl_xor_sync(0xFFFFFFFFu, sum[r], d);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (n0 + r < count) {
        // dx = g * rstd + (xh * (-rstd * c) + dresidual)
        const float kf = __fmul_rn(-rstd[r], __fmul_rn(sum[r], p.inv_cols));
        const float2 r2 = make_float2(rstd[r], rstd[r]), k2 = make_float2(kf, kf);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
          if (t + k * TPR < p.chunks) {
            float2 a[4], b[4], e[4];
            unpack2(*reinterpret_cast<const uint4*>(ring + at[r] + k * TPR * 16), a);
            unpack2(*reinterpret_cast<const uint4*>(ring + at[r] + row_bytes + k * TPR * 16), b);
            if (arrays == 3) {
              unpack2(*reinterpret_cast<const uint4*>(ring + at[r] + 2 * row_bytes + k * TPR * 16), e);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) e[i] = make_float2(0.0f, 0.0f);
            }
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 v = __ffma2_rn(__fmul2_rn(a[i], w[k][i]), r2, __ffma2_rn(__fmul2_rn(b[i], r2), k2, e[i]));
              o[i] = pack_bf16(v.x, v.y);
            }
            *reinterpret_cast<uint4*>(out + k * TPR * 8) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        out += out_step;
      }
    }
  }
  if (late && t == 0)                                          // no copy may land after the block has gone
    for (uint32_t n = fp4ring::first_open(fetched, ring_rows); n < (uint32_t)fetched; ++n)
      fp4dev::mbar_wait_bounded(bar0 + 8 * fp4ring::slot_of(n, ring_rows), fp4ring::parity_of(n, ring_rows));
  store_partials<CPT>(p, acc, t, TPR);
}

// dweight[c] = sum over the partials' rows, in a fixed order: 32 columns a CTA, 32 rows at a time.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* partials, float* out, uint32_t parts,
                                                          uint32_t cols) {
  __shared__ float s[32][33];
  pdl_trigger();
  pdl_wait();
  const uint32_t x = threadIdx.x & 31u, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  float v = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (uint32_t r = y; r < parts; r += 32) v = __fadd_rn(v, partials[(long long)r * cols + c]);
  }
  s[y][x] = v;
  __syncthreads();
  v = s[x][y];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  if (x == 0 && blockIdx.x * 32 + y < cols) out[blockIdx.x * 32 + y] = v;
}

// How a row is spread: chunks a thread, threads a row (a multiple of 32), rows a block.
struct RowShape {
  int cpt;
  uint32_t tpr, slots;
};
// Rows of up to 128 chunks (1024 elements) are a warp's own; longer ones take four chunks a thread, in blocks
// of at least 128 threads.
RowShape row_shape(int64_t chunks) {
  if (chunks <= 128) return {(int)((chunks + 31) / 32), 32u, 8u};
  const uint32_t tpr = (uint32_t)((chunks + 127) / 128 * 32);
  return {4, tpr, tpr >= 128 ? 1u : 256u / tpr};
}

template <int CPT, int MOST, int BLOCKS = 1>
cudaError_t run_norm(const NormArgs& p, int fmt, uint32_t grid, cudaStream_t st) {
  const dim3 block(p.tpr * p.slots);
  return fmt == FP8_E4M3_CODES
             ? launch_kernel(rmsnorm_fp8_kernel<0, CPT, MOST, BLOCKS>, dim3(grid), block, 0, st, false, 1u, p)
             : launch_kernel(rmsnorm_fp8_kernel<1, CPT, MOST, BLOCKS>, dim3(grid), block, 0, st, false, 1u, p);
}

template <int CPT>
cudaError_t run_short(const NormBwdArgs& p, int parts, cudaStream_t st) {
  return launch_kernel(rmsnorm_backward_short_kernel<CPT>, dim3(parts), dim3(256), (p.slots - 1) * p.cols * sizeof(float),
                       st, false, 1u, p);
}

// The long rows' ring: two blocks an SM where each holds four rows of three arrays, else one.
constexpr int64_t kRingBytes = 222 * 1024;
int long_blocks(int64_t cols) { return 4 * cols * 6 <= kRingBytes / 2 ? 2 : 1; }

template <int R>
cudaError_t run_long(const NormBwdArgs& p, int parts, unsigned* error, cudaStream_t st) {
  auto kernel = rmsnorm_backward_long_kernel<R>;
  static SmemLimit limit;
  const cudaError_t attr = limit.raise(kernel, (int)kRingBytes + 256);
  if (attr != cudaSuccess) return attr;
  const int64_t slot = (int64_t)p.cols * 2 * (p.dres != nullptr ? 3 : 2);
  const int rows = (int)std::min<int64_t>(16, kRingBytes / long_blocks(p.cols) / slot);
  return launch_kernel(kernel, dim3(parts), dim3(p.tpr), (size_t)(rows * (slot + 8)), st, false, 1u, p, rows, error);
}

}  // namespace

cudaError_t launch_rmsnorm_fp8(const RmsNormParams& q, int num_sms, cudaStream_t st) {
  NormArgs p;
  p.x = static_cast<const uint16_t*>(q.x);
  p.residual = static_cast<const uint16_t*>(q.residual);
  p.weight = q.weight;
  p.rows = q.rows;
  p.ldx = q.ldx;
  p.ldr = q.ldr;
  p.ldc = q.ldc;
  p.eps = (double)q.eps;
  p.inv_cols = 1.0 / (double)q.cols;
  p.codes = q.codes;
  p.scales = q.scales;
  p.residual_out = static_cast<uint16_t*>(q.residual_out);
  p.norm_out = static_cast<uint16_t*>(q.norm_out);
  p.rstd = q.rstd;
  p.cols = (uint32_t)q.cols;
  p.chunks = (uint32_t)(q.cols / 8);
  p.groups = (uint32_t)fp8_groups(q.cols);
  p.main_ctas = 0;
  p.weight_f32 = q.weight_f32;
  p.sf_mma = q.sf_mma;
  // With fewer rows than SMs nothing hides a row's latency but its own width: as many threads as it has chunks.
  RowShape shape = row_shape(p.chunks);
  if (q.rows < num_sms) {
    const int cpt = p.chunks <= 1024 ? 1 : 2;
    shape = {cpt, (p.chunks + 32 * cpt - 1) / (32 * cpt) * 32, 1u};
  }
  p.tpr = shape.tpr;
  p.slots = shape.slots;
  p.main_ctas = (uint32_t)((q.rows + shape.slots - 1) / shape.slots);
  const uint32_t grid = p.main_ctas + (p.sf_mma && q.rows % 128 != 0 ? 1u : 0u);
  if (shape.tpr == 32) {
    switch (shape.cpt) {
      case 1: return run_norm<1, kShortThreads>(p, q.fmt, grid, st);
      case 2: return run_norm<2, kShortThreads>(p, q.fmt, grid, st);
      case 3: return run_norm<3, kShortThreads>(p, q.fmt, grid, st);
      default: return run_norm<4, kShortThreads>(p, q.fmt, grid, st);
    }
  }
  switch (shape.cpt) {
    case 1: return run_norm<1, 1024>(p, q.fmt, grid, st);
    case 2: return run_norm<2, 1024>(p, q.fmt, grid, st);
    default:
      return shape.tpr <= 384 ? run_norm<4, 384, 3>(p, q.fmt, grid, st) : run_norm<4, 512, 2>(p, q.fmt, grid, st);
  }
}

// Blocks of the backward kernel, each a row of partial sums.
int rmsnorm_backward_parts(int64_t rows, int64_t cols, int num_sms) {
  const int64_t slots = cols <= 1024 ? 8 : 1;
  const int64_t most = (int64_t)num_sms * (cols <= 1024 ? 2 : long_blocks(cols));
  return (int)std::min<int64_t>(most, (rows + slots - 1) / slots);
}

cudaError_t launch_rmsnorm_backward(const RmsNormBackwardParams& q, int num_sms, cudaStream_t st) {
  NormBwdArgs p;
  p.dy = static_cast<const uint16_t*>(q.dy);
  p.h = static_cast<const uint16_t*>(q.h);
  p.weight = q.weight;
  p.rstd = q.rstd;
  p.dres = static_cast<const uint16_t*>(q.dresidual);
  p.dx = static_cast<uint16_t*>(q.dx);
  p.partials = q.partials;
  p.rows = q.rows;
  p.lddy = q.lddy;
  p.ldh = q.ldh;
  p.lddr = q.lddr;
  p.inv_cols = 1.0f / (float)q.cols;
  p.cols = (uint32_t)q.cols;
  p.chunks = (uint32_t)(q.cols / 8);
  p.weight_f32 = q.weight_f32;
  const int parts = rmsnorm_backward_parts(q.rows, q.cols, num_sms);
  cudaError_t e;
  if (p.chunks <= 128) {
    p.tpr = 32;
    p.slots = 8;
    switch ((p.chunks + 31) / 32) {
      case 1: e = run_short<1>(p, parts, st); break;
      case 2: e = run_short<2>(p, parts, st); break;
      case 3: e = run_short<3>(p, parts, st); break;
      default: e = run_short<4>(p, parts, st); break;
    }
  } else {
    p.tpr = (p.chunks + 63) / 64 * 32;
    p.slots = 1;
    // two rows a barrier where the ring holds eight of them
    e = 8 * (int64_t)p.cols * 6 <= kRingBytes / 2 ? run_long<2>(p, parts, q.error, st) : run_long<1>(p, parts, q.error, st);
  }
  if (e != cudaSuccess) return e;
  return launch_kernel(column_sum_kernel, dim3((p.cols + 31) / 32), dim3(1024), 0, st, false, 1u,
                       (const float*)q.partials, q.dweight, (uint32_t)parts, p.cols);
}

}  // namespace fp4lib
