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

// RN(a / b) for many a with one b, r = RN(1 / b): the product a r is corrected twice by its residual. After the
// first correction it is a faithful quotient, and one more of a faithful quotient with a correctly rounded
// reciprocal gives the rounded one (P. Markstein, IBM Journal of Research and Development 34, 1990). Held for
// ordinary b only, where no residual underflows, and for |a| below 1e18, where no quotient overflows (a quotient of
// infinity would be corrected to a NaN); others take the division itself.
__device__ __forceinline__ bool ordinary(float b) { return b > 1e-20f && b < 1e20f; }
constexpr uint32_t kOrdinaryMax = 0x5D5E0B6Bu;  // the bits of 1e18
// The residual is taken as q b - a and its product subtracted, which keeps the sign of a zero.
__device__ __forceinline__ float2 quotient(float2 a, float2 b, float2 r) {
  const float2 na = __fmul2_rn(a, make_float2(-1.f, -1.f)), nr = make_float2(-r.x, -r.y);
  float2 q = __fmul2_rn(a, r);
  q = __ffma2_rn(__ffma2_rn(q, b, na), nr, q);
  return __ffma2_rn(__ffma2_rn(q, b, na), nr, q);
}

// What the NVFP4 scales of a matrix are made with: 6 g and its reciprocal.
struct Scale {
  float g, d, r;
  __device__ __forceinline__ explicit Scale(const float* p) {
    g = p ? *p : 1.0f;
    d = __fmul_rn(6.0f, g);
    r = __frcp_rn(d);
  }
};

// The scale byte of a block from its largest magnitude (as float bits), and what x is multiplied or
// divided by for its codes: NVFP4 the step (divide; 0: zero codes), MXFP4 the reciprocal (multiply,
// exact; 0: zero codes).
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax_bits, const Scale& sc, float& by) {
  if (FMT == kNv) {
    if (amax_bits >= kInfBits) {
      by = 0.f;
      return 0x7F;
    }
    const float amax = __uint_as_float(amax_bits);
    const float t = ordinary(sc.d) && amax_bits < kOrdinaryMax
                        ? quotient(make_float2(amax, 0.f), make_float2(sc.d, sc.d), make_float2(sc.r, sc.r)).x
                        : __fdiv_rn(amax, sc.d);
    const uint32_t code = __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
    by = __fmul_rn(e4m3_value(code), sc.g);
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

__device__ __forceinline__ uint32_t pack8(const float* y) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    out |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(y[2 * i], y[2 * i + 1]), __NV_E2M1, cudaRoundNearest) << (8 * i);
  return out;
}

// Codes of 8 elements (element 2i in the low nibble of byte i). MXFP4: x times a power of two is exact.
// NVFP4: the code of RN(x / step); quotients that are exactly the midpoint of two codes are common (a step is a few
// bits times g, and g is usually made of one of the elements), so the product with a reciprocal alone, 2 ulp off,
// would not do. The quotient by correction takes 6 instructions for two elements. A block whose scale saturates (numbers
// past 6 * 448 g) has quotients of any size. amax_bits: the block's largest magnitude.
template <int FMT>
__device__ __forceinline__ uint32_t codes8(const float* x, float by, uint32_t amax_bits) {
  if (by == 0.f) return 0;
  float y[8];
  if (FMT == kMx) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * by;
    return pack8(y);
  }
  if (ordinary(by) && amax_bits < kOrdinaryMax) {
    const float r = __frcp_rn(by);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 v = quotient(make_float2(x[i], x[i + 1]), make_float2(by, by), make_float2(r, r));
      y[i] = v.x;
      y[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], by);
  }
  return pack8(y);
}

// f g for a result that is rounded again, to 16 bits: rounded to odd (of the two fp32 numbers around a product that
// is none, the one whose last bit is set), so that the second rounding gives what one alone would.
__device__ __forceinline__ float product_to_odd(float f, float g) {
  const float low = __fmul_rd(f, g);
  return __float_as_uint(low) & 1 ? low : __fmul_ru(f, g);
}

// Fp32 values of the 8 codes of a word, times the matrix scale (the codes and their block scale have 7 significant bits
// together: their product is exact). ODD: for a 16-bit result.
template <bool ODD>
__device__ __forceinline__ void values8(uint32_t codes, float scale, float g, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((codes >> (8 * i)) & 0xFF), __NV_E2M1);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const float x = __fmul_rn(f.x, scale), y = __fmul_rn(f.y, scale);
    v[2 * i] = ODD ? product_to_odd(x, g) : __fmul_rn(x, g);
    v[2 * i + 1] = ODD ? product_to_odd(y, g) : __fmul_rn(y, g);
  }
}

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

// 8 consecutive elements of type TYPE (MOE_TYPE_*) as they lie in memory, their largest magnitude as fp32 bits,
// and their fp32 values. Magnitudes of the 16-bit types are compared two at a time as integers.
template <int TYPE>
struct Eight {
  uint4 w;
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
  }
  __device__ __forceinline__ void clear() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t amax() const {
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    const uint32_t m = __vmaxu2(__vimax3_u16x2(w.x & kAbs, w.y & kAbs, w.z & kAbs), w.w & kAbs);
    const uint32_t h = max(m & 0xFFFFu, m >> 16);
    if (TYPE == MOE_TYPE_BF16) return h << 16;
    const __half_raw r{(unsigned short)h};
    return __float_as_uint(__half2float(__half(r)));
  }
  __device__ __forceinline__ void values(float* v) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (TYPE == MOE_TYPE_BF16) {
        v[2 * i] = bf16_lo(u[i]);
        v[2 * i + 1] = bf16_hi(u[i]);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
};
template <>
struct Eight<MOE_TYPE_F32> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    a = q[0];
    b = q[1];
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ uint32_t amax() const {
    return max(__vimax3_u32(__vimax3_u32(abs_bits(a.x), abs_bits(a.y), abs_bits(a.z)), abs_bits(a.w), abs_bits(b.x)),
               __vimax3_u32(abs_bits(b.y), abs_bits(b.z), abs_bits(b.w)));
  }
  __device__ __forceinline__ void values(float* v) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

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
