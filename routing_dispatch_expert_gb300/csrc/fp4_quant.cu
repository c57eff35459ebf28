// Rows to microscaled 4 bits, and back to the values they stand for (formats in fp4_impl.cuh).
//
// One pass over the rows: a lane holds 8 consecutive elements, so a warp's loads (16 or 32 bytes a lane)
// and stores (4 bytes of codes a lane) are contiguous; a block of 16 or 32 elements is 2 or 4 lanes,
// which share its largest magnitude by shuffles. HBM-bound.
#include "common.cuh"
#include "fp4_impl.cuh"
#include "kernels.h"

namespace moe {
namespace fp4 {

constexpr int kThreads = 256;

template <int TYPE>  // MOE_TYPE_*
__device__ __forceinline__ void load8(const void* p, int64_t at, float* v) {
  if (TYPE == MOE_TYPE_F32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = q[0], b = q[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    return;
  }
  const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
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

// One thread per 8 elements; `per_row` of them a row (a multiple of 4: blocks never straddle a warp).
template <int FMT, int TYPE>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const void* __restrict__ x, int64_t ldx, uint32_t units,
                                                            uint32_t per_row, const float* __restrict__ g,
                                                            uint32_t* __restrict__ q, uint8_t* __restrict__ s) {
  const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
  const bool in = u < units;
  const float gs = g ? *g : 1.0f;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (in) {
    const uint32_t row = u / per_row;
    load8<TYPE>(x, row * ldx + 8 * (int64_t)(u - row * per_row), v);
  }
  const uint32_t m = block_amax<FMT>(amax8<FMT>(v));
  if (!in) return;
  float by;
  const uint32_t code = block_scale<FMT>(m, gs, by);
  q[u] = codes8<FMT>(v, by);
  constexpr uint32_t kLanes = kBlock<FMT> / 8;
  if (u % kLanes == 0) s[u / kLanes] = (uint8_t)code;
}

template <int FMT, int TYPE>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint32_t* __restrict__ q,
                                                              const uint8_t* __restrict__ s,
                                                              const float* __restrict__ g, uint32_t units,
                                                              void* __restrict__ y) {
  const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
  if (u >= units) return;
  const uint32_t b = s[u / (kBlock<FMT> / 8)];
  float v[8];
  values8(q[u], FMT == kNv ? e4m3_value(b) : e8m0_value(b), FMT == kNv && g ? *g : 1.0f, v);
  if (TYPE == MOE_TYPE_F32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(y) + 8 * (int64_t)u);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (TYPE == MOE_TYPE_BF16) {
      w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + 8 * (int64_t)u) = make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace fp4

cudaError_t launch_quantize_fp4(const void* x, int type, int64_t rows, int64_t cols, int64_t ldx, int format,
                                const float* g, void* q, void* s, cudaStream_t stream) {
  if (rows == 0 || cols == 0) return cudaSuccess;
  const uint32_t per_row = (uint32_t)(cols / 8), units = (uint32_t)(rows * (cols / 8));
  const uint32_t blocks = (uint32_t)cdiv(units, fp4::kThreads);
  auto go = [&](auto kernel) {
    kernel<<<blocks, fp4::kThreads, 0, stream>>>(x, ldx, units, per_row, g, static_cast<uint32_t*>(q),
                                                 static_cast<uint8_t*>(s));
    return cudaGetLastError();
  };
  using namespace fp4;
  if (format == kNv)
    return type == MOE_TYPE_F32    ? go(quantize_kernel<kNv, MOE_TYPE_F32>)
           : type == MOE_TYPE_BF16 ? go(quantize_kernel<kNv, MOE_TYPE_BF16>)
                                   : go(quantize_kernel<kNv, MOE_TYPE_F16>);
  return type == MOE_TYPE_F32    ? go(quantize_kernel<kMx, MOE_TYPE_F32>)
         : type == MOE_TYPE_BF16 ? go(quantize_kernel<kMx, MOE_TYPE_BF16>)
                                 : go(quantize_kernel<kMx, MOE_TYPE_F16>);
}

cudaError_t launch_dequantize_fp4(const void* q, const void* s, const float* g, int64_t rows, int64_t cols, int format,
                                  int type, void* y, cudaStream_t stream) {
  if (rows == 0 || cols == 0) return cudaSuccess;
  const uint32_t units = (uint32_t)(rows * (cols / 8));
  const uint32_t blocks = (uint32_t)cdiv(units, fp4::kThreads);
  auto go = [&](auto kernel) {
    kernel<<<blocks, fp4::kThreads, 0, stream>>>(static_cast<const uint32_t*>(q), static_cast<const uint8_t*>(s), g,
                                                 units, y);
    return cudaGetLastError();
  };
  using namespace fp4;
  if (format == kNv)
    return type == MOE_TYPE_F32    ? go(dequantize_kernel<kNv, MOE_TYPE_F32>)
           : type == MOE_TYPE_BF16 ? go(dequantize_kernel<kNv, MOE_TYPE_BF16>)
                                   : go(dequantize_kernel<kNv, MOE_TYPE_F16>);
  return type == MOE_TYPE_F32    ? go(dequantize_kernel<kMx, MOE_TYPE_F32>)
         : type == MOE_TYPE_BF16 ? go(dequantize_kernel<kMx, MOE_TYPE_BF16>)
                                 : go(dequantize_kernel<kMx, MOE_TYPE_F16>);
}

}  // namespace moe
