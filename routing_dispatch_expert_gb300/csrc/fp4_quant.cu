// Rows to microscaled 4 bits, and back to the values they stand for (formats in fp4_impl.cuh).
//
// One pass over the rows: a lane holds 8 or 16 consecutive elements, so a warp's loads and stores are
// contiguous; a block of 16 or 32 elements is 1 to 4 lanes, which share its largest magnitude by shuffles.
// Bound by HBM, but for 16-bit rows to NVFP4, whose quotients make about 100 instructions of 8 elements.
// 16384 x 7168 on one GB300 (bytes in and out over the time; a copy moves 6788 GB/s): bf16 to MXFP4 43 - 46 us
// (6.5 - 6.9 TB/s), to NVFP4 54 - 56 us (5.3 - 5.6); fp32 to either 74 - 80 us (6.7 - 7.1); back to fp32 80 - 82 us (6.5),
// to bf16 45 - 48 us (6.2 - 6.7).
#include <type_traits>

#include "common.cuh"
#include "fp4_impl.cuh"
#include "kernels.h"

namespace moe {
namespace fp4 {

constexpr int kThreads = 256;

// A thread has units of 8 elements (a whole NVFP4 block of 16 where their loads are 16 bytes: one scale a lane
// instead of two equal ones, 65 -> 56 us for 16384 x 7168 bf16 rows, whose bound is instructions), kThreads apart:
// their loads are all in flight together.
constexpr int kUnits = 4;
template <int FMT, int TYPE>
constexpr int kEights = FMT == kNv && TYPE != MOE_TYPE_F32 ? 2 : 1;  // of a unit

// `per_row` units a row (blocks never straddle a warp: cols is a multiple of 32); PACKED: rows follow one another.
template <int FMT, int TYPE, bool PACKED>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const void* __restrict__ x, int64_t ldx, uint32_t units,
                                                            uint32_t per_row, const float* __restrict__ g,
                                                            uint32_t* __restrict__ q, uint8_t* __restrict__ s) {
  constexpr int W = kEights<FMT, TYPE>, N = kUnits / W;
  const uint32_t u0 = blockIdx.x * (kThreads * N) + threadIdx.x;
  const Scale gs(FMT == kNv ? g : nullptr);
  Eight<TYPE> x8[N][W];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t u = u0 + i * kThreads;
    if (u < units) {
      const uint32_t row = PACKED ? 0 : u / per_row;
#pragma unroll
      for (int w = 0; w < W; ++w) x8[i][w].load(x, row * ldx + 8 * W * (int64_t)(u - row * per_row) + 8 * w);
    } else {
#pragma unroll
      for (int w = 0; w < W; ++w) x8[i][w].clear();
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t u = u0 + i * kThreads;
    const uint32_t m = W == 2 ? max(x8[i][0].amax(), x8[i][W - 1].amax()) : block_amax<FMT>(x8[i][0].amax());
    if (u >= units) continue;
    float by, v[8];
    const uint32_t code = block_scale<FMT>(m, gs, by);
    uint32_t c[W];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      x8[i][w].values(v);
      c[w] = codes8<FMT>(v, by, m);
    }
    if (W == 2) {
      reinterpret_cast<uint2*>(q)[u] = make_uint2(c[0], c[W - 1]);
      s[u] = (uint8_t)code;
    } else {
      q[u] = c[0];
      constexpr uint32_t kLanes = kBlock<FMT> / 8;
      if (u % kLanes == 0) s[u / kLanes] = (uint8_t)code;
    }
  }
}

template <int FMT, int TYPE, bool WIDE>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint32_t* __restrict__ q,
                                                              const uint8_t* __restrict__ s,
                                                              const float* __restrict__ g, uint32_t units,
                                                              void* __restrict__ y) {
  const uint32_t u0 = blockIdx.x * (kThreads * kUnits) + threadIdx.x;
  const float gs = FMT == kNv && g ? *g : 1.0f;
  uint32_t c[kUnits], b[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const uint32_t u = u0 + i * kThreads;
    c[i] = u < units ? q[u] : 0;
    b[i] = u < units ? s[u / (kBlock<FMT> / 8)] : 0;
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const uint32_t u = u0 + i * kThreads;
    if (u >= units) return;
    float v[8];
    // MXFP4 values are exact in fp32: no matrix scale
    values8<FMT == kNv && TYPE != MOE_TYPE_F32>(c[i], FMT == kNv ? e4m3_value(b[i]) : e8m0_value(b[i]), gs, v);
    if (TYPE == MOE_TYPE_F32) {
      float* o = static_cast<float*>(y) + 8 * (int64_t)u;
      if (WIDE) {
        st_global_v8(o, reinterpret_cast<const uint32_t*>(v));
      } else {  // y is 16-byte but not 32-byte aligned
        reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
      continue;
    }
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (TYPE == MOE_TYPE_BF16) {
        w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
      } else {
        const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + 8 * (int64_t)u) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace fp4

cudaError_t launch_quantize_fp4(const void* x, int type, int64_t rows, int64_t cols, int64_t ldx, int format,
                                const float* g, void* q, void* s, cudaStream_t stream) {
  if (rows == 0 || cols == 0) return cudaSuccess;
  using namespace fp4;
  using std::integral_constant;
  auto pick = [&](auto format_c, auto type_c) {
    constexpr int F = decltype(format_c)::value, T = decltype(type_c)::value, W = kEights<F, T>;
    const uint32_t per_row = (uint32_t)(cols / (8 * W)), units = (uint32_t)(rows * per_row);
    const uint32_t blocks = (uint32_t)cdiv(units, kThreads * (kUnits / W));
    auto kernel = rows == 1 || ldx == cols ? quantize_kernel<F, T, true> : quantize_kernel<F, T, false>;
    kernel<<<blocks, kThreads, 0, stream>>>(x, ldx, units, per_row, g, static_cast<uint32_t*>(q), static_cast<uint8_t*>(s));
    return cudaGetLastError();
  };
  auto with_type = [&](auto format_c) {
    return type == MOE_TYPE_F32    ? pick(format_c, integral_constant<int, MOE_TYPE_F32>{})
           : type == MOE_TYPE_BF16 ? pick(format_c, integral_constant<int, MOE_TYPE_BF16>{})
                                   : pick(format_c, integral_constant<int, MOE_TYPE_F16>{});
  };
  return format == kNv ? with_type(integral_constant<int, kNv>{}) : with_type(integral_constant<int, kMx>{});
}

cudaError_t launch_dequantize_fp4(const void* q, const void* s, const float* g, int64_t rows, int64_t cols, int format,
                                  int type, void* y, cudaStream_t stream) {
  if (rows == 0 || cols == 0) return cudaSuccess;
  const uint32_t units = (uint32_t)(rows * (cols / 8));
  const uint32_t blocks = (uint32_t)cdiv(units, fp4::kThreads * fp4::kUnits);
  auto go = [&](auto kernel) {
    kernel<<<blocks, fp4::kThreads, 0, stream>>>(static_cast<const uint32_t*>(q), static_cast<const uint8_t*>(s), g,
                                                 units, y);
    return cudaGetLastError();
  };
  using namespace fp4;
  using std::integral_constant;
  auto with_type = [&](auto format_c) {
    constexpr int F = decltype(format_c)::value;
    if (type == MOE_TYPE_F32)
      return reinterpret_cast<uintptr_t>(y) % 32 == 0 ? go(dequantize_kernel<F, MOE_TYPE_F32, true>)
                                                      : go(dequantize_kernel<F, MOE_TYPE_F32, false>);
    return type == MOE_TYPE_BF16 ? go(dequantize_kernel<F, MOE_TYPE_BF16, false>)
                                 : go(dequantize_kernel<F, MOE_TYPE_F16, false>);
  };
  return format == kNv ? with_type(integral_constant<int, kNv>{}) : with_type(integral_constant<int, kMx>{});
}

}  // namespace moe
