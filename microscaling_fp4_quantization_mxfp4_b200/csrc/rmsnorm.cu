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
// Sums, statistics and y are fp32; the only roundings to fewer bits are the outputs' own.
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

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(a)) |
         ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(b)) << 16);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
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

// Sum over the TPR threads of a row (every thread of the block takes part; `part` holds one float per
// warp).  Warp shuffles, then the row's warps in order.
template <int TPR, int THREADS>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int d = (TPR < 32 ? TPR : 32) / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  if (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) part[warp] = v;
    __syncthreads();
    constexpr int W = TPR / 32;
    const int w0 = warp / W * W;
    v = part[w0];
#pragma unroll
    for (int i = 1; i < W; ++i) v += part[w0 + i];
  }
  return v;
}

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;
  const void* weight;
  long long rows, ldx, ldr, ldc;
  float eps, fcols;
  uint8_t* codes;
  uint8_t* scales;
  uint16_t* residual_out;
  uint16_t* norm_out;
  float* rstd;
  uint32_t cols, chunks, groups, main_ctas;
  int weight_f32, fmt, sf_mma;
};

// TPR threads a row, CPT 8-element chunks a thread: the row stays in registers between the sum of
// squares and the quantization, so x and the residual are read once.  Bound by HBM (7 bytes an element
// with a residual); one row of few: by the latency of load -> sum -> store.
template <int TPR, int CPT>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) rmsnorm_fp8_kernel(NormArgs p) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kRows = kThreads / TPR;
  __shared__ float part[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x >= p.main_ctas) {
    zero_pad_rows(p.scales, p.rows, p.groups);
    return;
  }
  const uint32_t t = threadIdx.x % TPR;
  const long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
  const bool live = row < p.rows;
  uint4 h[CPT];
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const uint32_t c = t + k * TPR;
    h[k] = make_uint4(0, 0, 0, 0);
    if (live && c < p.chunks) h[k] = *reinterpret_cast<const uint4*>(p.x + row * p.ldx + c * 8);
  }
  if (p.residual != nullptr) {
    uint4 r[CPT];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const uint32_t c = t + k * TPR;
      r[k] = make_uint4(0, 0, 0, 0);
      if (live && c < p.chunks) r[k] = *reinterpret_cast<const uint4*>(p.residual + row * p.ldr + c * 8);
    }
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const uint32_t c = t + k * TPR;
      float a[8], b[8];
      fp4dev::unpack8(h[k], a);
      fp4dev::unpack8(r[k], b);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = __fadd_rn(a[i], b[i]);
      h[k] = pack8(a);
      if (live && c < p.chunks) *reinterpret_cast<uint4*>(p.residual_out + row * p.cols + c * 8) = h[k];
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    float a[8];
    fp4dev::unpack8(h[k], a);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __fmaf_rn(a[i], a[i], ss);
  }
  ss = row_sum<TPR, kThreads>(ss, part);
  const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(ss, p.fcols), p.eps));
  if (live && t == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const uint32_t c = t + k * TPR;
    const bool on = live && c < p.chunks;
    float y[8];
    fp4dev::unpack8(h[k], y);
    uint32_t m = 0;
    if (on) {
      float w[8];
      load_weight8(p.weight, p.weight_f32, c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] = __fmul_rn(__fmul_rn(y[i], rstd), w[i]);
        m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
      }
    }
    m = max_half_warp(m);
    const uint32_t byte = p.fmt == 0 ? scale_byte<0>(m) : scale_byte<1>(m);
    const float inv = inv_scale(byte);
    const uint32_t g = c >> 4;
    if (on) {
      *reinterpret_cast<uint2*>(p.codes + row * p.ldc + c * 8) = p.fmt == 0 ? codes8<0>(y, inv) : codes8<1>(y, inv);
      if (p.norm_out != nullptr) *reinterpret_cast<uint4*>(p.norm_out + row * p.cols + c * 8) = pack8(y);
    }
    if (live && g < p.groups) {
      const uint32_t j = c & 15u;
      if (j == 0) p.scales[sf_offset(p.sf_mma, row, g, p.groups)] = (uint8_t)byte;
      else if (p.sf_mma && g + 1 == p.groups && j <= ((4u - (p.groups & 3u)) & 3u))
        p.scales[sf_offset(1, row, g + j, p.groups)] = 0;            // groups that pad the layout to 4
    }
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
  float fcols;
  uint32_t cols, chunks;
  int weight_f32;
};

// Every CTA walks rows blockIdx, blockIdx + gridDim, ... (kRows of them at a time) and keeps its
// columns' sums of dy * xh in registers; they leave once, as one row of `partials` per row slot.
template <int TPR, int CPT>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) rmsnorm_backward_kernel(NormBwdArgs p) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kRows = kThreads / TPR;
  __shared__ float part[2][kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const uint32_t t = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  float acc[CPT][8];
#pragma unroll
  for (int k = 0; k < CPT; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[k][i] = 0.0f;
  int flip = 0;
  for (long long r0 = (long long)blockIdx.x * kRows; r0 < p.rows; r0 += (long long)gridDim.x * kRows, flip ^= 1) {
    const long long row = r0 + slot;
    const bool live = row < p.rows;
    const float rstd = live ? p.rstd[row] : 0.0f;
    uint4 d[CPT], h[CPT];
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const uint32_t c = t + k * TPR;
      d[k] = h[k] = make_uint4(0, 0, 0, 0);
      if (live && c < p.chunks) {
        d[k] = *reinterpret_cast<const uint4*>(p.dy + row * p.lddy + c * 8);
        h[k] = *reinterpret_cast<const uint4*>(p.h + row * p.ldh + c * 8);
      }
    }
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const uint32_t c = t + k * TPR;
      if (live && c < p.chunks) {
        float a[8], b[8], w[8];
        fp4dev::unpack8(d[k], a);
        fp4dev::unpack8(h[k], b);
        load_weight8(p.weight, p.weight_f32, c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = __fmul_rn(b[i], rstd);
          s = __fmaf_rn(__fmul_rn(a[i], w[i]), xh, s);
          acc[k][i] = __fmaf_rn(a[i], xh, acc[k][i]);
        }
      }
    }
    s = row_sum<TPR, kThreads>(s, part[flip]);       // two buffers: one barrier a row
    const float c1 = __fdiv_rn(s, p.fcols);
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const uint32_t c = t + k * TPR;
      if (live && c < p.chunks) {
        float a[8], b[8], w[8], r[8];
        fp4dev::unpack8(d[k], a);
        fp4dev::unpack8(h[k], b);
        load_weight8(p.weight, p.weight_f32, c, w);
        if (p.dres != nullptr) {
          fp4dev::unpack8(*reinterpret_cast<const uint4*>(p.dres + row * p.lddr + c * 8), r);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) r[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float g = __fmul_rn(a[i], w[i]), xh = __fmul_rn(b[i], rstd);
          a[i] = __fmaf_rn(rstd, __fmaf_rn(-xh, c1, g), r[i]);
        }
        *reinterpret_cast<uint4*>(p.dx + row * p.cols + c * 8) = pack8(a);
      }
    }
  }
  float* out = p.partials + ((long long)blockIdx.x * kRows + slot) * p.cols;
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const uint32_t c = t + k * TPR;
    if (c < p.chunks) {
      reinterpret_cast<float4*>(out + c * 8)[0] = make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
      reinterpret_cast<float4*>(out + c * 8)[1] = make_float4(acc[k][4], acc[k][5], acc[k][6], acc[k][7]);
    }
  }
}

// dweight[c] = sum over the partials' rows, in a fixed order: 32 columns a CTA, 32 rows at a time.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* partials, float* out, uint32_t parts,
                                                          uint32_t cols) {
  __shared__ float s[32][33];
  pdl_trigger();
  pdl_wait();
  const uint32_t x = threadIdx.x & 31u, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  float v = 0.0f;
  if (c < cols)
    for (uint32_t r = y; r < parts; r += 32) v = __fadd_rn(v, partials[(long long)r * cols + c]);
  s[y][x] = v;
  __syncthreads();
  v = s[x][y];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  if (x == 0 && blockIdx.x * 32 + y < cols) out[blockIdx.x * 32 + y] = v;
}

// Threads a row: the least power of two with at most `cpt` chunks a thread.
int threads_for(int64_t chunks, int cpt, int most) {
  int t = 32;
  while (t < most && (int64_t)t * cpt < chunks) t *= 2;
  return t;
}

template <int TPR, int CPT>
cudaError_t run_norm(const NormArgs& a, cudaStream_t st) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  NormArgs p = a;
  p.main_ctas = (uint32_t)((a.rows + kThreads / TPR - 1) / (kThreads / TPR));
  const uint32_t grid = p.main_ctas + (a.sf_mma && a.rows % 128 != 0 ? 1u : 0u);
  return launch_kernel(rmsnorm_fp8_kernel<TPR, CPT>, dim3(grid), dim3(kThreads), 0, st, false, 1u, p);
}

// Chunks a thread of the backward kernel, and the threads of a row that follow from it.
constexpr int kBwdChunks = 2;
void backward_shape(int64_t cols, int* tpr, int* cpt) {
  const int64_t chunks = cols / 8;
  *tpr = threads_for(chunks, kBwdChunks, 512);
  *cpt = (int64_t)*tpr * kBwdChunks >= chunks ? kBwdChunks : 4;
}

template <int TPR, int CPT>
cudaError_t run_backward(const NormBwdArgs& p, int parts, cudaStream_t st) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  return launch_kernel(rmsnorm_backward_kernel<TPR, CPT>, dim3(parts / (kThreads / TPR)), dim3(kThreads), 0, st, false,
                       1u, p);
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
  p.eps = q.eps;
  p.fcols = (float)q.cols;
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
  p.fmt = q.fmt;
  p.sf_mma = q.sf_mma;
  // With a row for every SM the rows hide each other's latency and two chunks a thread move more bytes
  // per instruction; with fewer rows than SMs the row itself is spread over as many threads as it has chunks.
  const int cpt = q.rows < num_sms ? 1 : 2;
  const int tpr = threads_for(p.chunks, cpt, 1024);
  if (cpt == 1 && (int64_t)tpr >= p.chunks) {
    switch (tpr) {
      case 32: return run_norm<32, 1>(p, st);
      case 64: return run_norm<64, 1>(p, st);
      case 128: return run_norm<128, 1>(p, st);
      case 256: return run_norm<256, 1>(p, st);
      case 512: return run_norm<512, 1>(p, st);
      default: return run_norm<1024, 1>(p, st);
    }
  }
  switch (tpr) {
    case 32: return run_norm<32, 2>(p, st);
    case 64: return run_norm<64, 2>(p, st);
    case 128: return run_norm<128, 2>(p, st);
    case 256: return run_norm<256, 2>(p, st);
    case 512: return run_norm<512, 2>(p, st);
    default: return run_norm<1024, 2>(p, st);
  }
}

int rmsnorm_backward_parts(int64_t rows, int64_t cols, int num_sms) {
  int tpr, cpt;
  backward_shape(cols, &tpr, &cpt);
  const int threads = tpr < 256 ? 256 : tpr, slots = threads / tpr;
  const int64_t most = (int64_t)num_sms * (1024 / threads);           // CTAs that fill the device
  return (int)std::min<int64_t>(most, (rows + slots - 1) / slots) * slots;
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
  p.fcols = (float)q.cols;
  p.cols = (uint32_t)q.cols;
  p.chunks = (uint32_t)(q.cols / 8);
  p.weight_f32 = q.weight_f32;
  const int parts = rmsnorm_backward_parts(q.rows, q.cols, num_sms);
  int tpr, cpt;
  backward_shape(q.cols, &tpr, &cpt);
  cudaError_t e;
  switch (tpr) {
    case 32: e = run_backward<32, 2>(p, parts, st); break;
    case 64: e = run_backward<64, 2>(p, parts, st); break;
    case 128: e = run_backward<128, 2>(p, parts, st); break;
    case 256: e = run_backward<256, 2>(p, parts, st); break;
    default: e = cpt == 2 ? run_backward<512, 2>(p, parts, st) : run_backward<512, 4>(p, parts, st); break;
  }
  if (e != cudaSuccess) return e;
  return launch_kernel(column_sum_kernel, dim3((p.cols + 31) / 32), dim3(1024), 0, st, false, 1u,
                       (const float*)q.partials, q.dweight, (uint32_t)parts, p.cols);
}

}  // namespace fp4lib
