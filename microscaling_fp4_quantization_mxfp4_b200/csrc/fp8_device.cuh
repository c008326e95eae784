// Device-side building blocks of the 8-bit operators: E4M3 / E5M2 codes under one power-of-two
// (E8M0) scale per block of 128 elements.
//
// The scale exponent is the least E >= -127 with amax <= Fmax * 2^E, where Fmax = 1.75 * 2^TOP
// (448 for E4M3, TOP = 8; 57344 for E5M2, TOP = 15): no element saturates, and as 2^-E is exact the
// only rounding of an element is the one to its code.  The byte is E + 127 (0 for a zero block).  A
// block that holds an infinity or a NaN gets byte 255 (the NaN of E8M0) and NaN codes, so that an
// overflow upstream shows in every product it enters.
//
// Magnitudes are compared as the unsigned bit patterns of |x|: they order like the values, with NaN
// above infinity above the finite ones, so one integer maximum gives amax and the non-finite test.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4_device.cuh"

namespace fp8dev {

constexpr uint32_t kBlock = 128;
constexpr uint32_t kNanByte = 255u;

template <int FMT>
struct Format {
  static constexpr int kTop = FMT == 0 ? 8 : 15;     // largest value 1.75 * 2^kTop
};

// Scale byte of a block whose largest |x| has the fp32 bit pattern `bits`.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t bits) {
  const int f = (int)(bits >> 23);
  const int b = max(f - Format<FMT>::kTop + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0), 0);
  return f == 255 ? kNanByte : (uint32_t)b;
}
// 2^(127 - byte); for the NaN byte a NaN, which makes every code of the block one.
__device__ __forceinline__ float inv_scale(uint32_t byte) {
  return byte == kNanByte ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float((254u - byte) << 23);
}

// Two codes, `a` in the low byte (round to nearest even; NaN stays NaN).
template <int FMT>
__device__ __forceinline__ uint32_t cvt2(float a, float b) {
  uint16_t r;
  if (FMT == 0) asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  else asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return (uint32_t)r;
}
template <int FMT>
__device__ __forceinline__ uint32_t cvt4(float a, float b, float c, float d) {
  return cvt2<FMT>(a, b) | (cvt2<FMT>(c, d) << 16);
}
// Eight elements times `inv` -> eight codes.
template <int FMT>
__device__ __forceinline__ uint2 codes8(const float2 (&v)[4], float inv) {
  const float2 s = make_float2(inv, inv);
  const float2 a = __fmul2_rn(v[0], s), b = __fmul2_rn(v[1], s), c = __fmul2_rn(v[2], s), d = __fmul2_rn(v[3], s);
  return make_uint2(cvt4<FMT>(a.x, a.y, b.x, b.y), cvt4<FMT>(c.x, c.y, d.x, d.y));
}
// Eight bf16 elements as fp32 pairs.
__device__ __forceinline__ void unpack2(const uint4& v, float2 (&x)[4]) {
  x[0] = make_float2(fp4dev::bf16_lo(v.x), fp4dev::bf16_hi(v.x));
  x[1] = make_float2(fp4dev::bf16_lo(v.y), fp4dev::bf16_hi(v.y));
  x[2] = make_float2(fp4dev::bf16_lo(v.z), fp4dev::bf16_hi(v.z));
  x[3] = make_float2(fp4dev::bf16_lo(v.w), fp4dev::bf16_hi(v.w));
}

// Two bf16 magnitudes at once: the larger of each half, as 16-bit patterns.
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }
__device__ __forceinline__ uint32_t max_abs8(const uint4& v) {
  return max_abs2(max_abs2(max_abs2(v.x & 0x7FFF7FFFu, v.y), v.z), v.w);
}
// Larger half of a 16-bit pair as an fp32 bit pattern.
__device__ __forceinline__ uint32_t pair_bits(uint32_t m) { return max(m << 16, m & 0xFFFF0000u); }

// Larger magnitude of three, NaN if one is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Scale bytes of the N (at most 4) blocks that each half warp holds, 8 elements a lane and block: m[j] is
// the lane's part of block j's maximum.  The butterfly halves the blocks with the lanes, so that four maxima
// take five shuffles instead of sixteen and each lane works out one byte, that of block `own` (which may be N
// or more: no block); four more hand out the inverse scales.  `first`: the lane that stores the byte.
template <int FMT, int N>
__device__ __forceinline__ uint32_t block_scales(const uint32_t (&m)[N], float (&inv)[N], int& own, bool& first) {
  const int lane = threadIdx.x & 31;
  uint32_t k;
  if (N == 1) {
    k = m[0];
    k = max(k, __shfl_xor_sync(0xFFFFFFFFu, k, 8));
    k = max(k, __shfl_xor_sync(0xFFFFFFFFu, k, 4));
    own = 0;
    first = (lane & 15) == 0;
  } else if (N == 2) {
    const bool b = (lane & 8) != 0;
    k = max(b ? m[1 % N] : m[0], __shfl_xor_sync(0xFFFFFFFFu, b ? m[0] : m[1 % N], 8));
    k = max(k, __shfl_xor_sync(0xFFFFFFFFu, k, 4));
    own = b ? 1 : 0;
    first = (lane & 7) == 0;
  } else {
    const bool b = (lane & 8) != 0, c = (lane & 4) != 0;
    const uint32_t m3 = N == 4 ? m[N - 1] : 0u;
    const uint32_t k0 = max(b ? m[2 % N] : m[0], __shfl_xor_sync(0xFFFFFFFFu, b ? m[0] : m[2 % N], 8));
    const uint32_t k1 = max(b ? m3 : m[1 % N], __shfl_xor_sync(0xFFFFFFFFu, b ? m[1 % N] : m3, 8));
    k = max(c ? k1 : k0, __shfl_xor_sync(0xFFFFFFFFu, c ? k0 : k1, 4));
    own = (lane >> 2) & 3;
    first = (lane & 3) == 0;
  }
  k = max(k, __shfl_xor_sync(0xFFFFFFFFu, k, 2));
  k = max(k, __shfl_xor_sync(0xFFFFFFFFu, k, 1));
  const uint32_t byte = scale_byte<FMT>(k);
  const float mine = inv_scale(byte);
  if (N == 1) {
    inv[0] = mine;
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) inv[j] = __shfl_sync(0xFFFFFFFFu, mine, (lane & 16) | (j * (N == 2 ? 8 : 4)));
  }
  return byte;
}

__device__ __forceinline__ long long sf_offset(int sf_mma, long long row, long long g, long long groups) {
  return sf_mma ? fp4dev::sf_mma_offset(row, g, (groups + 3) >> 2) : row * groups + g;
}

// Zero scale words (four groups each) of the rows that pad the tensor-core layout to 128, by one
// thread block.
__device__ __forceinline__ void zero_pad_rows(uint8_t* scales, long long rows, long long groups) {
  const long long gt = (groups + 3) >> 2, pad = ((rows + 127) & ~127ll) - rows;
  for (long long i = threadIdx.x; i < pad * gt; i += blockDim.x) {
    const long long r = rows + i / gt, t = i % gt;
    *reinterpret_cast<uint32_t*>(scales + fp4dev::sf_mma_offset(r, 4 * t, gt)) = 0u;
  }
}

}  // namespace fp8dev
