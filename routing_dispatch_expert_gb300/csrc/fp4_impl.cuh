// Microscaled 4-bit formats: the block scales and codes of rows quantised at run time, shared by the
// quantise kernel (fp4_quant.cu), the dispatch copy (dispatch.cu) and the epilogue of the 4-bit grouped
// GEMM (gemm_a4.cu), so that a row has the same codes on every path.
//
//   NVFP4 (blocks of 16)  scale = e4m3(RN(amax / RN(6 g))), step = RN(scale * g), codes e2m1(RN(x / step));
//                         g is the matrix scale; every rounding to nearest even, saturating; codes 0
//                         where the step is 0.
//   MXFP4 (blocks of 32)  scale = 2^(floor(log2 amax) - 2), at least 2^-127, held as its e8m0 exponent
//                         byte; codes e2m1(x / scale): exact quotients, the scale is a power of two.
// A block that holds an infinity or a NaN gets the NaN scale (0x7F, 0xFF) and zero codes: its products
// are NaN, never a finite number made of an infinity. The magnitudes are compared as their bit patterns,
// under which every NaN is larger than every number.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {
namespace fp4 {

constexpr int kNv = 0;  // MOE_FP4_NV
constexpr int kMx = 1;  // MOE_FP4_MX

template <int FMT>
constexpr int kBlock = FMT == kNv ? 16 : 32;

constexpr uint32_t kInfBits = 0x7F800000u;

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  const __half_raw r = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&r));
}

__device__ __forceinline__ float e8m0_value(uint32_t code) {
  if (code == 0xFF) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(code ? code << 23 : 0x00400000u);
}

// The scale byte of a block from its largest magnitude (as float bits), and what x is multiplied or
// divided by for its codes: NVFP4 the step (divide; 0: zero codes), MXFP4 the reciprocal (multiply,
// exact; 0: zero codes).
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax_bits, float g, float& by) {
  if (FMT == kNv) {
    if (amax_bits >= kInfBits) {
      by = 0.f;
      return 0x7F;
    }
    const uint32_t code =
        __nv_cvt_float_to_fp8(__fdiv_rn(__uint_as_float(amax_bits), __fmul_rn(6.0f, g)), __NV_SATFINITE, __NV_E4M3);
    by = __fmul_rn(e4m3_value(code), g);
    return code;
  }
  if (amax_bits >= kInfBits) {
    by = 0.f;
    return 0xFF;
  }
  const int code = max((int)(amax_bits >> 23) - 2, 0);
  by = __uint_as_float((uint32_t)(254 - code) << 23);  // 2^(127 - code): at most 2^127
  return (uint32_t)code;
}

// Codes of 8 elements (element 2i in the low nibble of byte i). The NVFP4 quotient is the IEEE one: a
// value next to the midpoint of two codes falls as the definition says.
template <int FMT>
__device__ __forceinline__ uint32_t codes8(const float* x, float by) {
  if (FMT == kNv && by == 0.f) return 0;
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 v;
    if (FMT == kNv) {
      v.x = __fdiv_rn(x[2 * i], by);
      v.y = __fdiv_rn(x[2 * i + 1], by);
    } else {
      v.x = x[2 * i] * by;
      v.y = x[2 * i + 1] * by;
    }
    out |= (uint32_t)__nv_cvt_float2_to_fp4x2(v, __NV_E2M1, cudaRoundNearest) << (8 * i);
  }
  return FMT == kMx && by == 0.f ? 0 : out;
}

// Fp32 values of the 8 codes of a word, times a factor that rounds once (the codes and their block scale
// have 7 significant bits together: their product is exact).
__device__ __forceinline__ void values8(uint32_t codes, float scale, float g, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((codes >> (8 * i)) & 0xFF), __NV_E2M1);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * i] = __fmul_rn(__fmul_rn(f.x, scale), g);
    v[2 * i + 1] = __fmul_rn(__fmul_rn(f.y, scale), g);
  }
}

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

template <int FMT>
__device__ __forceinline__ uint32_t amax8(const float* x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(x[i]));
  return m;
}

// Largest magnitude over the lanes of a block when each lane holds 8 consecutive elements: 2 lanes
// (NVFP4) or 4 (MXFP4). All lanes of the warp take part.
template <int FMT>
__device__ __forceinline__ uint32_t block_amax(uint32_t m) {
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  if (FMT == kMx) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  return m;
}

}  // namespace fp4
}  // namespace moe
