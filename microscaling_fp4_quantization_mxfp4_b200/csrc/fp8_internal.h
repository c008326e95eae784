// Host-side internal interface of the 8-bit operators (quantizers, product, RMS norm) between the
// C-ABI layer (api.cu) and their launchers.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace fp4lib {

// Raises a kernel's limit of dynamic shared memory, once a device: a function's attributes are each device's
// own.  One object a kernel.
class SmemLimit {
 public:
  template <typename K>
  cudaError_t raise(K* kernel, int bytes) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool kept = dev >= 0 && dev < kDevices;
    if (kept && raised_[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    const cudaError_t set = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (kept && set == cudaSuccess) raised_[dev].store(true, std::memory_order_relaxed);
    return set;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<bool> raised_[kDevices] = {};
};

enum { FP8_E4M3_CODES = 0, FP8_E5M2_CODES = 1 };

// Blocks of 128 elements along a row of length n.
inline int64_t fp8_groups(int64_t n) { return (n + 127) / 128; }

struct Fp8QuantizeParams {
  const void* x;                // bf16 [rows, cols], row stride ld
  int64_t rows, cols, ld;
  int fmt;                      // FP8_E4M3_CODES or FP8_E5M2_CODES
  uint8_t* codes;               // along the rows (null: not written)
  int64_t ldc;
  uint8_t* scales;
  uint8_t* codes_t;             // of the transpose (null: not written)
  int64_t ldc_t;
  uint8_t* scales_t;
  int sf_mma;
};
// 1 x 128 blocks along the rows (codes, scales).
cudaError_t launch_fp8_quantize_rows(const Fp8QuantizeParams& p, cudaStream_t st);
// 1 x 128 blocks of the transpose, i.e. along the columns (codes_t, scales_t).
cudaError_t launch_fp8_quantize_cols(const Fp8QuantizeParams& p, cudaStream_t st);
// 128 x 128 tiles (codes, scales and, unless null, codes_t, scales_t).
cudaError_t launch_fp8_quantize_tiles(const Fp8QuantizeParams& p, cudaStream_t st);
cudaError_t launch_fp8_dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t rows, int64_t cols,
                                  int fmt, int sf_mma, void* out, int out_bf16, cudaStream_t st);

struct Fp8GemmParams {
  const uint8_t* a;
  int64_t lda;
  const uint8_t* a_sf;
  const uint8_t* b;
  int64_t ldb;
  const uint8_t* b_sf;
  int64_t M, N, K;
  int a_fmt, b_fmt;
  void* y;
  int64_t ldy;
  int y_bf16;
  unsigned* error;
};
// cudaErrorNotSupported if the driver entry point for tensor maps is missing.
cudaError_t launch_fp8_gemm(const Fp8GemmParams& p, int num_sms, cudaStream_t st);

constexpr int64_t kMaxNormCols = 16384;

struct RmsNormParams {
  const void* x;                // bf16 [rows, cols], row stride ldx
  int64_t ldx;
  const void* residual;         // bf16, row stride ldr; null: none
  int64_t ldr;
  const void* weight;           // [cols], bf16 or fp32
  int weight_f32;
  int64_t rows, cols;
  float eps;
  int fmt;
  uint8_t* codes;
  int64_t ldc;
  uint8_t* scales;
  int sf_mma;
  void* residual_out;           // bf16 [rows, cols] contiguous; null without residual
  float* rstd;                  // [rows]; null: not written
  void* norm_out;               // bf16 [rows, cols] contiguous; null: not written
};
cudaError_t launch_rmsnorm_fp8(const RmsNormParams& p, int num_sms, cudaStream_t st);

struct RmsNormBackwardParams {
  const void* dy;               // bf16 [rows, cols], row stride lddy
  int64_t lddy;
  const void* h;                // bf16 [rows, cols], row stride ldh
  int64_t ldh;
  const void* weight;
  int weight_f32;
  const float* rstd;
  const void* dresidual;        // bf16, row stride lddr; null: none
  int64_t lddr;
  int64_t rows, cols;
  void* dx;                     // bf16 [rows, cols] contiguous
  float* dweight;               // [cols]
  float* partials;              // [rmsnorm_backward_parts(...), cols]
  unsigned* error;              // device error word
};
int rmsnorm_backward_parts(int64_t rows, int64_t cols, int num_sms);
cudaError_t launch_rmsnorm_backward(const RmsNormBackwardParams& p, int num_sms, cudaStream_t st);

}  // namespace fp4lib
