// What the kernels of the norm (rms_norm.cu) and of its gradient (rms_norm_backward.cu) share.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace moe {
namespace rn {

using rows::Chunk;
using rows::kChunk;
using rows::kMap1;
using rows::kMap2;
using rows::kMap4;
using rows::kMap8;
using rows::kOdd;

constexpr int kNone = -1;

template <int LANES = 32>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A chunk of the weight; ones where there is none.
template <int TYPE, int MAP, int LANES>
__device__ __forceinline__ void load_weight(const void* w, int w_f32, int c0, int cols, int lane, float (&f)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.f;
  } else if (w_f32) {
    Chunk<MOE_TYPE_F32, MAP, LANES> c;
    c.load(w, c0, cols, lane);
    c.values(f);
  } else {
    Chunk<TYPE, MAP, LANES> c;
    c.load(w, c0, cols, lane);
    c.values(f);
  }
}

template <int V>
using Int = std::integral_constant<int, V>;

// Narrow rows take an access of 8 columns a lane where they are whole ones, else number by number.
inline bool by_words(int cols) { return cols > 128 || cols % 8 == 0; }

// f(type, the other type, map, lanes of a row) of rows of `type` beside rows of `other` (kNone, the same, or fp32);
// aligned: all are whole 16 bytes, even: all begin an even number of elements apart
template <class F>
cudaError_t with_types(int type, int other, bool aligned, bool even, int lanes, F&& f) {
  auto mapped = [&](auto T, auto O) {
    constexpr int kAligned = decltype(T)::value == MOE_TYPE_F32 || decltype(O)::value == MOE_TYPE_F32 ? kMap4 : kMap8;
    auto odd = [&](auto M) {
      if (lanes == 4) return f(T, O, M, Int<4>{});
      if (lanes == 8) return f(T, O, M, Int<8>{});
      if (lanes == 16) return f(T, O, M, Int<16>{});
      return f(T, O, M, Int<32>{});
    };
    if constexpr (decltype(T)::value != MOE_TYPE_F32) {
      if (!aligned && even) return odd(Int<kMap2>{});
    }
    if (!aligned) return odd(Int<kMap1>{});
    if (lanes == 4) return f(T, O, Int<kMap8>{}, Int<4>{});
    if (lanes == 8) return f(T, O, Int<kMap8>{}, Int<8>{});
    if (lanes == 16) return f(T, O, Int<kMap8>{}, Int<16>{});
    return f(T, O, Int<kAligned>{}, Int<32>{});
  };
  auto beside = [&](auto T) {
    if (other == kNone) return mapped(T, Int<kNone>{});
    if (other == MOE_TYPE_F32) return mapped(T, Int<MOE_TYPE_F32>{});
    return mapped(T, T);
  };
  if (type == MOE_TYPE_F32) return beside(Int<MOE_TYPE_F32>{});
  if (type == MOE_TYPE_BF16) return beside(Int<MOE_TYPE_BF16>{});
  return beside(Int<MOE_TYPE_F16>{});
}

}  // namespace rn
}  // namespace moe
