// Rows of fp32, bf16 or fp16 numbers as the kernels of the norm (rms_norm.cu, rms_norm_backward.cu) and of the rows' way
// back (unpermute.cu) read and write them: a warp takes 256 consecutive columns (a chunk) at a time, a lane 8 of them,
// held as fp32.
//
// Which 8 depends on how the rows lie in memory (MAP):
//   kMap8  rows that are whole 16 bytes and begin on 16, 16-bit numbers: columns 8 lane .. 8 lane + 7, one 16-byte
//          access
//   kMap4  the same for fp32: columns 4 lane .. + 3 and 128 + 4 lane .. + 3, so that both accesses are whole lines;
//          16-bit rows beside fp32 ones take two 8-byte accesses for it
//   kMap1  rows of any width that begin anywhere: columns lane + 32 i, one number an access. A warp's access is then 64
//          or 128 consecutive bytes; with 8 consecutive numbers a lane it would be 32 pieces of four lines. Of narrow
//          rows that share a warp, LANES lanes each, columns lane + LANES i.
//   kMap2  rows of an even number of 16-bit numbers, whose begins are as far apart: the same by two numbers an access,
//          columns 2 lane + 64 i and the next one; fp32 rows beside them take two numbers of 8 bytes
// Every chunk is 256 columns in all of them, so a lane's columns are the same in every row, and the blocks of 128
// columns that share an 8-bit scale are half a chunk.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"

namespace moe {
namespace rows {

constexpr int kMap8 = 0, kMap4 = 1, kMap1 = 2, kMap2 = 3;
template <int MAP>
constexpr bool kOdd = MAP == kMap1 || MAP == kMap2;  // rows that are not whole 16 bytes
constexpr int kChunk = 256;

template <int TYPE>
constexpr int kSize = TYPE == MOE_TYPE_F32 ? 4 : 2;

// Column of a lane's i-th number within the chunk.
template <int MAP, int LANES = 32>
__device__ __forceinline__ int column(int lane, int i) {
  return MAP == kMap8   ? 8 * lane + i
         : MAP == kMap4 ? 128 * (i / 4) + 4 * lane + i % 4
         : MAP == kMap2 ? 2 * LANES * (i / 2) + 2 * lane + i % 2
                        : LANES * i + lane;
}

template <int TYPE>
__device__ __forceinline__ float value(uint32_t bits) {
  if (TYPE == MOE_TYPE_F32) return __uint_as_float(bits);
  if (TYPE == MOE_TYPE_BF16) return __uint_as_float(bits << 16);
  return __half2float(__ushort_as_half((unsigned short)bits));
}
template <int TYPE>
__device__ __forceinline__ uint32_t bits_of(float v) {  // rounded to nearest even
  if (TYPE == MOE_TYPE_F32) return __float_as_uint(v);
  if (TYPE == MOE_TYPE_BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  return __half_as_ushort(__float2half_rn(v));
}
template <int TYPE>
__device__ __forceinline__ uint32_t load_bits(const void* p, int64_t at) {
  if (TYPE == MOE_TYPE_F32) return static_cast<const uint32_t*>(p)[at];
  return static_cast<const uint16_t*>(p)[at];
}
template <int TYPE>
__device__ __forceinline__ void store_bits(void* p, int64_t at, uint32_t v) {
  if (TYPE == MOE_TYPE_F32)
    static_cast<uint32_t*>(p)[at] = v;
  else
    static_cast<uint16_t*>(p)[at] = (uint16_t)v;
}

template <int TYPE>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (TYPE == MOE_TYPE_BF16) return pack_bf16x2(lo, hi);
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <int TYPE>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (TYPE == MOE_TYPE_BF16) return make_float2(bf16_lo(w), bf16_hi(w));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// A lane's 8 numbers of a chunk as they lie in memory: nothing is done with them until values(), so the loads of
// several chunks and tensors are in flight together. c0: first column of the chunk; columns at and past cols are 0.
template <int TYPE, int MAP, int LANES = 32>
struct Chunk {
  static constexpr bool kWide = TYPE == MOE_TYPE_F32;
  uint32_t w[MAP == kMap1 || kWide ? 8 : 4];

  __device__ __forceinline__ void load(const void* row, int c0, int cols, int lane) {
    if constexpr (MAP == kMap1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c0 + column<MAP, LANES>(lane, i);
        w[i] = c < cols ? load_bits<TYPE>(row, c) : 0u;
      }
    } else if constexpr (MAP == kMap2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + column<MAP, LANES>(lane, 2 * i);
        const char* p = static_cast<const char*>(row) + (int64_t)c * kSize<TYPE>;
        if constexpr (kWide) {
          const uint2 v = c < cols ? *reinterpret_cast<const uint2*>(p) : make_uint2(0u, 0u);
          w[2 * i] = v.x, w[2 * i + 1] = v.y;
        } else {
          w[i] = c < cols ? *reinterpret_cast<const uint32_t*>(p) : 0u;
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < (kWide || MAP == kMap4 ? 2 : 1); ++h) {
        const int c = c0 + column<MAP>(lane, 4 * h);
        const char* p = static_cast<const char*>(row) + (int64_t)c * kSize<TYPE>;
        if constexpr (!kWide && MAP == kMap4) {
          uint2 v = make_uint2(0u, 0u);
          if (c < cols) v = *reinterpret_cast<const uint2*>(p);
          w[2 * h] = v.x, w[2 * h + 1] = v.y;
        } else {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (c < cols) v = *reinterpret_cast<const uint4*>(p);
          w[4 * h] = v.x, w[4 * h + 1] = v.y, w[4 * h + 2] = v.z, w[4 * h + 3] = v.w;
        }
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (MAP == kMap1 || kWide ? 8 : 4); ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
    if constexpr (MAP == kMap1 || kWide) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = value<TYPE>(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = unpack2<TYPE>(w[i]);
        f[2 * i] = v.x, f[2 * i + 1] = v.y;
      }
    }
  }
};

// A lane's 8 numbers to a row, each rounded once; columns at and past cols are left alone.
template <int TYPE, int MAP, int LANES = 32>
__device__ __forceinline__ void store(void* row, int c0, int cols, int lane, const float (&f)[8]) {
  constexpr bool kWide = TYPE == MOE_TYPE_F32;
  if constexpr (MAP == kMap1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + column<MAP, LANES>(lane, i);
      if (c < cols) store_bits<TYPE>(row, c, bits_of<TYPE>(f[i]));
    }
  } else if constexpr (MAP == kMap2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + column<MAP, LANES>(lane, 2 * i);
      char* p = static_cast<char*>(row) + (int64_t)c * kSize<TYPE>;
      if (c >= cols) continue;
      if constexpr (kWide)
        *reinterpret_cast<float2*>(p) = make_float2(f[2 * i], f[2 * i + 1]);
      else
        *reinterpret_cast<uint32_t*>(p) = pack2<TYPE>(f[2 * i], f[2 * i + 1]);
    }
  } else {
#pragma unroll
    for (int h = 0; h < (kWide || MAP == kMap4 ? 2 : 1); ++h) {
      const int c = c0 + column<MAP>(lane, 4 * h);
      char* p = static_cast<char*>(row) + (int64_t)c * kSize<TYPE>;
      if (c >= cols) continue;
      const float* g = f + 4 * h;
      if constexpr (kWide)
        *reinterpret_cast<float4*>(p) = make_float4(g[0], g[1], g[2], g[3]);
      else if constexpr (MAP == kMap4)
        *reinterpret_cast<uint2*>(p) = make_uint2(pack2<TYPE>(g[0], g[1]), pack2<TYPE>(g[2], g[3]));
      else
        *reinterpret_cast<uint4*>(p) = make_uint4(pack2<TYPE>(f[0], f[1]), pack2<TYPE>(f[2], f[3]),
                                                  pack2<TYPE>(f[4], f[5]), pack2<TYPE>(f[6], f[7]));
    }
  }
}

// The first n of 16 bytes of global memory into shared memory, zeros behind them: complete once the group they are
// committed in is waited for.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void copy8(uint32_t to, const void* from, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(n) : "memory");
}

// Zeros from byte `from` of base, which is on 16 bytes, up to byte `to`, by this thread of so many. Both are whole
// elements.
template <int SIZE>
__device__ __forceinline__ void clear(void* base, int64_t from, int64_t to, int64_t thread, int64_t threads) {
  using Part = typename std::conditional<SIZE == 4, uint32_t, typename std::conditional<SIZE == 2, uint16_t, uint8_t>::type>::type;
  char* const p = static_cast<char*>(base);
  const int64_t lo = min((from + 15) & ~(int64_t)15, to), hi = max(to & ~(int64_t)15, lo);
  for (int64_t i = from + SIZE * thread; i < lo; i += SIZE * threads) *reinterpret_cast<Part*>(p + i) = 0;
  for (int64_t i = lo + 16 * thread; i < hi; i += 16 * threads) *reinterpret_cast<uint4*>(p + i) = make_uint4(0u, 0u, 0u, 0u);
  for (int64_t i = hi + SIZE * thread; i < to; i += SIZE * threads) *reinterpret_cast<Part*>(p + i) = 0;
}

// Whether a row length or distance of n numbers of this type is whole 16 bytes.
inline bool whole(int type, int64_t n) { return n % (type == MOE_TYPE_F32 ? 4 : 8) == 0; }

// Lanes of a row, 8 columns each: narrow rows share a warp.
inline int lanes_of(int64_t cols) { return cols <= 32 ? 4 : cols <= 64 ? 8 : cols <= 128 ? 16 : 32; }

}  // namespace rows
}  // namespace moe
