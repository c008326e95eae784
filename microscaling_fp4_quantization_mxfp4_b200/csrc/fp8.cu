// Block-scaled FP8 quantization (E4M3 / E5M2 codes, one E8M0 scale per 128 elements) and its inverse.
// The formats and the scale rule are in fp8_device.cuh.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "fp4_device.cuh"
#include "fp4_internal.h"
#include "fp8_device.cuh"
#include "fp8_internal.h"

namespace fp4lib {
namespace {

using namespace fp8dev;

// ------------------------------------------------------- blocks along rows --
// Half a warp per block: 16 lanes x 8 elements (one 16-byte load each), 8-byte code stores (128 contiguous
// bytes a block).  Bound by HBM: 2 bytes in, 1 out per element.  Each warp takes kUnroll pairs of adjacent
// blocks with all loads in flight at once.
constexpr int kRowThreads = 256;
constexpr int kUnroll = 4;

struct RowArgs {
  const uint16_t* x;
  long long rows, ld, ldc;
  uint8_t* codes;
  uint8_t* scales;
  uint32_t groups, chunks;      // 128-element blocks and 8-element chunks in a row
  uint32_t items;               // rows * groups
  uint32_t main_ctas;           // CTAs beyond these zero the scale rows that pad the tensor-core layout
  int sf_mma;
};

template <int FMT>
__global__ void __launch_bounds__(kRowThreads) fp8_quantize_rows_kernel(RowArgs p) {
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x >= p.main_ctas) {
    zero_pad_rows(p.scales, p.rows, p.groups);
    return;
  }
  const uint32_t lane = threadIdx.x & 31u, half = lane >> 4, c16 = lane & 15u;
  const uint32_t warp = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);       // threads may pass 32 bits, warps do not
  const uint32_t first = warp * (2 * kUnroll) + half;               // blocks first, first + 2, ... in row order
  uint4 v[kUnroll];
  uint32_t row[kUnroll], g[kUnroll];
  bool on[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (u == 0) {
      row[0] = first / p.groups;
      g[0] = first - row[0] * p.groups;
    } else {
      row[u] = row[u - 1];
      g[u] = g[u - 1] + 2;
      while (g[u] >= p.groups) {
        g[u] -= p.groups;
        ++row[u];
      }
    }
    on[u] = first + 2 * u < p.items && g[u] * 16 + c16 < p.chunks;
    v[u] = make_uint4(0, 0, 0, 0);
    if (on[u]) v[u] = *reinterpret_cast<const uint4*>(p.x + (long long)row[u] * p.ld + (g[u] * 16 + c16) * 8);
  }
  uint32_t m[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) m[u] = pair_bits(max_abs8(v[u]));
  float inv[kUnroll];
  int own;
  bool stores;
  const uint32_t byte = block_scales<FMT>(m, inv, own, stores);
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (on[u]) {
      float2 e[4];
      unpack2(v[u], e);
      *reinterpret_cast<uint2*>(p.codes + (long long)row[u] * p.ldc + (g[u] * 16 + c16) * 8) = codes8<FMT>(e, inv[u]);
    }
  }
  if (stores && first + 2 * own < p.items) {
    uint32_t r = row[0], b = g[0];
#pragma unroll
    for (int u = 1; u < kUnroll; ++u)
      if (own == u) {
        r = row[u];
        b = g[u];
      }
    uint8_t* out = p.scales + sf_offset(p.sf_mma, r, b, p.groups);
    *out = (uint8_t)byte;
    if (p.sf_mma && b + 1 == p.groups)                              // groups that pad the layout to 4
      for (uint32_t k = 1; (b + k) & 3u; ++k) out[k] = 0;
  }
}

// ------------------------------------------- blocks along columns, and tiles --
// 128 x 128 elements a CTA, copied to shared memory by cp.async (zeros past the matrix).  TILE = false: every
// column of the tile is one block of the transpose.  TILE = true: one scale for the tile, its codes written
// along the rows and, unless codes_t is null, along the columns.  In the column phase a lane reads two adjacent
// columns (32 lanes: 64 columns, no bank conflicts) of 32 rows; the codes pass through the tile's own buffer, so
// that eight lanes store a whole 128-byte row of the transpose (32 bytes a lane, straight from registers,
// touched 32 lines an instruction: 46.6 us for 16301 x 4096).  Bound by HBM (3 or 4 bytes an element).  What is
// in flight is the other CTAs' tiles: five an SM (48 registers) took 34.2 us, six, which spill, 35.6, three
// persistent ones with a second buffer for the next tile 37.1.
constexpr int kTileThreads = 256;
constexpr int kTileLoads = 8;           // 16-byte chunks a thread
constexpr int kTileBlocks = 5;          // CTAs an SM

struct TileArgs {
  const uint16_t* x;
  long long rows, cols, ld, ldc, ldc_t;
  uint8_t* codes;
  uint8_t* scales;
  uint8_t* codes_t;
  uint8_t* scales_t;
  long long groups, groups_t;
  uint32_t tiles_x;             // tiles side by side
  int sf_mma;
};

template <int FMT, bool TILE>
__global__ void __launch_bounds__(kTileThreads, kTileBlocks) fp8_quantize_tile_kernel(TileArgs p) {
  __shared__ __align__(128) uint32_t tile[128 * 64];        // bf16 pairs, row-major
  __shared__ uint32_t red[4 * 64];                          // column maxima of the four 32-row groups / warps' maxima
  pdl_trigger();
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const long long rt = blockIdx.x / p.tiles_x, ct = blockIdx.x - rt * p.tiles_x;
  const long long r0 = rt * 128, c0 = ct * 128;
  pdl_wait();
  if (r0 >= p.rows || c0 >= p.cols) {
    // a tile of the layout's padding: its scales are zero
    if (t < 128) {
      if (TILE && r0 < p.rows) p.scales[sf_offset(1, r0 + t, ct, p.groups)] = 0;
      if (c0 < p.cols && p.scales_t != nullptr) p.scales_t[sf_offset(1, c0 + t, rt, p.groups_t)] = 0;
    }
    return;
  }
  {
    const long long row = r0 + (t >> 4), col = c0 + (t & 15) * 8;
    const uint16_t* src = p.x + row * p.ld + col;
    const uint32_t dst = fp4dev::smem_addr(tile) + t * 16;
#pragma unroll
    for (int i = 0; i < kTileLoads; ++i) {
      const bool in = row + 16 * i < p.rows && col < p.cols;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * kTileThreads * 16),
                   "l"(in ? src + 16 * i * p.ld : p.x), "r"(in ? 16 : 0)
                   : "memory");
    }
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
  }
  __syncthreads();
  uint32_t byte = 0;
  if (TILE) {
    uint4 v[kTileLoads];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kTileLoads; ++i) {
      v[i] = reinterpret_cast<const uint4*>(tile)[t + i * kTileThreads];
      m = __vmaxu2(m, max_abs8(v[i]));
    }
    m = __reduce_max_sync(0xFFFFFFFFu, pair_bits(m));
    if (lane == 0) red[warp] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int w = 0; w < kTileThreads / 32; ++w) m = max(m, red[w]);
    byte = scale_byte<FMT>(m);
    const float inv = inv_scale(byte);
    const int r = t >> 4, c = (t & 15) * 8;
    uint8_t* dst = p.codes + (r0 + r) * p.ldc + c0 + c;
#pragma unroll
    for (int i = 0; i < kTileLoads; ++i) {
      if (r0 + r + 16 * i < p.rows && c0 + c < p.cols) {
        float2 e[4];
        unpack2(v[i], e);
        *reinterpret_cast<uint2*>(dst + 16 * i * p.ldc) = codes8<FMT>(e, inv);
      }
    }
    if (t < 128) {
      if (r0 + t < p.rows) p.scales[sf_offset(p.sf_mma, r0 + t, ct, p.groups)] = (uint8_t)byte;
      else if (p.sf_mma) p.scales[sf_offset(1, r0 + t, ct, p.groups)] = 0;
    }
    if (p.codes_t == nullptr) return;
  }
  // columns: lane -> pair of columns in half `warp & 1`, rows 32 * (warp >> 1) .. + 31
  const int pr = (warp & 1) * 32 + lane, rg = warp >> 1;
  uint32_t w[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) w[i] = tile[(rg * 32 + i) * 64 + pr];
  uint32_t blo = byte, bhi = byte;
  if (!TILE) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) m = max_abs2(m, w[i]);
    red[rg * 64 + pr] = m;
    __syncthreads();
    m = __vmaxu2(__vmaxu2(red[pr], red[64 + pr]), __vmaxu2(red[128 + pr], red[192 + pr]));
    blo = scale_byte<FMT>(m << 16);
    bhi = scale_byte<FMT>(m & 0xFFFF0000u);
  }
  const float2 inv = make_float2(inv_scale(blo), inv_scale(bhi));
  uint32_t lo[8], hi[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float2 e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      e[i] = __fmul2_rn(make_float2(fp4dev::bf16_lo(w[4 * k + i]), fp4dev::bf16_hi(w[4 * k + i])), inv);
    lo[k] = cvt4<FMT>(e[0].x, e[1].x, e[2].x, e[3].x);
    hi[k] = cvt4<FMT>(e[0].y, e[1].y, e[2].y, e[3].y);
  }
  const long long c = c0 + 2 * pr;                        // even, and cols is a multiple of 8: both inside or both out
  if (rg == 0 && (c < p.cols || p.sf_mma)) {
    const bool in = c < p.cols;                           // else a row that pads the layout
    p.scales_t[sf_offset(p.sf_mma, c, rt, p.groups_t)] = in ? (uint8_t)blo : 0;
    p.scales_t[sf_offset(p.sf_mma, c + 1, rt, p.groups_t)] = in ? (uint8_t)bhi : 0;
  }
  if (TILE) __syncthreads();                              // the tile has been read (the maxima's barrier, without TILE)
  // 128 rows of 128 codes, 16-byte piece j of row r at j ^ (r / 2 mod 8): the two rows of a lane, and then a
  // row's eight pieces, fall on distinct banks
  uint4* out = reinterpret_cast<uint4*>(tile);
  const int sw = pr & 7;
  out[2 * pr * 8 + ((2 * rg) ^ sw)] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  out[2 * pr * 8 + ((2 * rg + 1) ^ sw)] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
  out[(2 * pr + 1) * 8 + ((2 * rg) ^ sw)] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  out[(2 * pr + 1) * 8 + ((2 * rg + 1) ^ sw)] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
  __syncthreads();
  const int piece = t & 7;
  const long long left = p.rows - (r0 + piece * 16);      // elements of the transpose's rows from this piece on
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (t >> 3) + 32 * i;
    if (c0 + r >= p.cols || left <= 0) break;
    const uint4 v = out[r * 8 + (piece ^ ((r >> 1) & 7))];
    uint8_t* dst = p.codes_t + (c0 + r) * p.ldc_t + r0 + piece * 16;
    if (left >= 16) {
      *reinterpret_cast<uint4*>(dst) = v;
    } else {
      const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int b = 0; b < 15; ++b)
        if (b < left) dst[b] = (uint8_t)(q[b / 4] >> (8 * (b & 3)));
    }
  }
}

// ------------------------------------------------------------- dequantize --
// One thread per 8 codes of a row, nothing read past its end: value = code * 2^(byte - 127) in fp32 (exact wherever the product
// is a normal fp32 number), rounded to bf16 on request.
struct DeqArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  void* out;
  long long rows, cols, ldc;
  uint32_t chunks, groups;
  uint64_t items;
  int sf_mma, fmt, out_bf16, vec;
};

__device__ __forceinline__ float code_value(uint32_t c, int fmt) {
  uint32_t h2;
  if (fmt == 0) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)c));
  else asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)c));
  const uint16_t h = (uint16_t)h2;
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

__global__ void __launch_bounds__(256) fp8_dequantize_kernel(DeqArgs p) {
  pdl_trigger();
  pdl_wait();
  for (uint64_t it = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; it < p.items;
       it += (uint64_t)gridDim.x * blockDim.x) {
    const uint64_t row = it / p.chunks;
    const uint32_t c = (uint32_t)(it - row * p.chunks) * 8;
    const uint32_t byte = p.scales[sf_offset(p.sf_mma, (long long)row, c >> 7, p.groups)];
    const float s = byte == kNanByte ? __uint_as_float(0x7FFFFFFFu) : fp4dev::mx_scale_value(byte);
    const uint8_t* src = p.codes + row * p.ldc + c;
    uint2 q = make_uint2(0, 0);
    if (c + 8 <= p.cols) {
      q = *reinterpret_cast<const uint2*>(src);
    } else {                                  // a row's last codes: the bytes behind them need not be the caller's
      for (int i = 0; i < 8; ++i)
        if (c + i < p.cols) (i < 4 ? q.x : q.y) |= (uint32_t)src[i] << (8 * (i & 3));
    }
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = i < 4 ? q.x : q.y;
      v[i] = __fmul_rn(code_value((w >> (8 * (i & 3))) & 0xFFu, p.fmt), s);
    }
    const long long o = (long long)row * p.cols + c;
    if (p.out_bf16) {
      __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.out) + o;
      if (p.vec) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(v[2 * i])) |
                 ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(v[2 * i + 1])) << 16);
        *reinterpret_cast<uint4*>(y) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        for (int i = 0; i < 8; ++i)
          if (c + i < p.cols) y[i] = __float2bfloat16_rn(v[i]);
      }
    } else {
      float* y = static_cast<float*>(p.out) + o;
      if (p.vec) {
        reinterpret_cast<float4*>(y)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(y)[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        for (int i = 0; i < 8; ++i)
          if (c + i < p.cols) y[i] = v[i];
      }
    }
  }
}

}  // namespace

cudaError_t launch_fp8_quantize_rows(const Fp8QuantizeParams& q, cudaStream_t st) {
  RowArgs p;
  p.x = static_cast<const uint16_t*>(q.x);
  p.rows = q.rows;
  p.ld = q.ld;
  p.ldc = q.ldc;
  p.codes = q.codes;
  p.scales = q.scales;
  p.groups = (uint32_t)fp8_groups(q.cols);
  p.chunks = (uint32_t)(q.cols / 8);
  p.items = (uint32_t)(q.rows * p.groups);
  p.sf_mma = q.sf_mma;
  constexpr uint32_t per_cta = kRowThreads / 32 * 2 * kUnroll;
  p.main_ctas = (p.items + per_cta - 1) / per_cta;
  const uint32_t grid = p.main_ctas + (q.sf_mma && q.rows % 128 != 0 ? 1u : 0u);
  return q.fmt == FP8_E4M3_CODES
             ? launch_kernel(fp8_quantize_rows_kernel<0>, dim3(grid), dim3(kRowThreads), 0, st, false, 1u, p)
             : launch_kernel(fp8_quantize_rows_kernel<1>, dim3(grid), dim3(kRowThreads), 0, st, false, 1u, p);
}

template <bool TILE>
static cudaError_t launch_tiles(const Fp8QuantizeParams& q, cudaStream_t st) {
  TileArgs p;
  p.x = static_cast<const uint16_t*>(q.x);
  p.rows = q.rows;
  p.cols = q.cols;
  p.ld = q.ld;
  p.ldc = q.ldc;
  p.ldc_t = q.ldc_t;
  p.codes = q.codes;
  p.scales = q.scales;
  p.codes_t = q.codes_t;
  p.scales_t = q.scales_t;
  p.groups = fp8_groups(q.cols);
  p.groups_t = fp8_groups(q.rows);
  p.sf_mma = q.sf_mma;
  int64_t gx = p.groups, gy = p.groups_t;
  if (q.sf_mma) {                     // the groups that pad the layout to 4 are tiles of their own
    if (TILE) gx = (gx + 3) / 4 * 4;
    if (q.scales_t != nullptr) gy = (gy + 3) / 4 * 4;
  }
  p.tiles_x = (uint32_t)gx;
  const dim3 grid((unsigned)(gx * gy));
  return q.fmt == FP8_E4M3_CODES
             ? launch_kernel(fp8_quantize_tile_kernel<0, TILE>, grid, dim3(kTileThreads), 0, st, false, 1u, p)
             : launch_kernel(fp8_quantize_tile_kernel<1, TILE>, grid, dim3(kTileThreads), 0, st, false, 1u, p);
}

cudaError_t launch_fp8_quantize_cols(const Fp8QuantizeParams& q, cudaStream_t st) { return launch_tiles<false>(q, st); }
cudaError_t launch_fp8_quantize_tiles(const Fp8QuantizeParams& q, cudaStream_t st) { return launch_tiles<true>(q, st); }

cudaError_t launch_fp8_dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t rows, int64_t cols,
                                  int fmt, int sf_mma, void* out, int out_bf16, cudaStream_t st) {
  DeqArgs p;
  p.codes = codes;
  p.scales = scales;
  p.out = out;
  p.rows = rows;
  p.cols = cols;
  p.ldc = ldc;
  p.chunks = (uint32_t)((cols + 7) / 8);
  p.groups = (uint32_t)fp8_groups(cols);
  p.items = (uint64_t)rows * p.chunks;
  p.sf_mma = sf_mma;
  p.fmt = fmt;
  p.out_bf16 = out_bf16;
  p.vec = cols % 8 == 0;
  const uint64_t ctas = (p.items + 255) / 256;
  const unsigned grid = (unsigned)std::min<uint64_t>(ctas, 1u << 20);
  return launch_kernel(fp8_dequantize_kernel, dim3(grid), dim3(256), 0, st, false, 1u, p);
}

}  // namespace fp4lib
