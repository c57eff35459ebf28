// Root-mean-square norm of the sum of a row and its residual, with an output in 8 bits, and its gradient.
//
//   t = x + r,  n = t * rstd,  rstd = 1 / sqrt(mean(t^2) + eps),  y = n * w
//   scale of 128 columns = amax |y| / 448 (at least 2^-126; 1 where all are 0), code = e4m3(RN(y RN(1 / scale)))
//   with g = dy * w:  dt = rstd * (g - n * mean(g n)) + (the gradient that reaches t from elsewhere)
//                     dw = sum over the rows of dy * n
//
// Everything is fp32: the sum is normalised and quantised before it is rounded for the residual stream, and each output
// is rounded once. The gradient is that of the norm of the t it is given; rstd is made again from t, which it reads
// anyway, instead of being stored.
//
// Both are bound by HBM: a row is read once and held on the SM between its reduction and its outputs. One GB300, out of
// HBM (a copy's rate is 6.78 TB/s), x and residual of one type, the gradient with the residual stream's:
//   16384 x 7168 bf16 to bf16 and e4m3 162 us, 6.5 TB/s        its gradient 143 us, 6.6 TB/s
//   8192 x 7168 fp32                   137 us, 6.9 TB/s                     138 us, 6.8 TB/s
//   8192 x 7167 bf16 / fp32            101, 4.6 / 138 us, 6.8               139, 3.4 / 161 us, 5.8
//   65536 x 512 bf16 / 65536 x 64      41, 6.6 / 6.6 us, 5.1                53, 5.0 / 11.6 us, 2.9
//   65536 x 511 bf16 / 65536 x 33      53, 5.0 / 6.5 us, 2.7               87, 3.1 / 14.7 us, 1.2
//   one row of 4096                    2.7 us, launch                       5.5 us, two launches
// Odd 16-bit rows are bound by their number-by-number accesses, narrow ones of the gradient by a barrier a row and its
// sums. Forward: three blocks of 448 threads an SM for 7168 columns, so that one block's loads run beside another's
// sums; that takes 42 registers, with the weight loaded behind the reduction (two blocks: 192 us). Backward: one
// round of blocks, rows copied ahead into shared memory (rows held in registers instead, one block an SM: 167 us; two,
// spilling: 226). Rows of up to 128 columns share a warp (65536 x 64 bf16 6.6 us, with a warp a row 16.7; 65536 x 33 6.5
// and 18.8, its gradient 14.7 and 39).
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace moe {
namespace rn {

using rows::Chunk;
using rows::kChunk;
using rows::kMap1;
using rows::kMap4;
using rows::kMap8;

constexpr int kNone = -1;
constexpr uint32_t kInfBits = 0x7F800000u;

struct Args {
  const void* x;
  const void* r;
  const void* w;
  void* y;
  void* total;
  uint8_t* q;
  float* s;
  int64_t rows, ldx, ldr;
  int cols, w_f32;
  float eps;
};

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

// Codes and scales of a chunk: two blocks of 128 columns. The codes are made with the reciprocal, 1.5 ulp of fp32 off
// the quotient: that moves a code only where y / scale is that close to a midpoint, which unlike for rows of few bits
// is rare here, and takes one instruction instead of eight. The largest magnitude is taken over the bits, under which a
// NaN is larger than every number: a block that holds an infinity or a NaN stands for NaN throughout.
template <int MAP, int LANES>
__device__ __forceinline__ void quantize(const Args& a, int64_t row, int c0, int cols, int lane, const float (&y)[8]) {
  constexpr bool kOne = MAP == kMap8 || LANES < 32;  // a lane's columns lie in one block
  uint32_t m[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int h = kOne ? 0 : i / 4;
    m[h] = max(m[h], __float_as_uint(y[i]) & 0x7FFFFFFFu);
  }
  if (kOne) {
#pragma unroll
    for (int o = (LANES < 16 ? LANES : 16) / 2; o > 0; o >>= 1) m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
  } else {
    m[0] = __reduce_max_sync(0xffffffffu, m[0]);
    m[1] = __reduce_max_sync(0xffffffffu, m[1]);
  }
  const int nb = (a.cols + 127) / 128;
  float v[8];
#pragma unroll
  for (int h = 0; h < (kOne ? 1 : 2); ++h) {
    constexpr int kN = kOne ? 8 : 4;
    float scale = 1.f;
    if (m[h]) scale = m[h] > kInfBits ? __uint_as_float(m[h]) : fmaxf(__fdiv_rn(__uint_as_float(m[h]), 448.0f), 1.1754944e-38f);
    const float by = __frcp_rn(scale);
#pragma unroll
    for (int i = 0; i < kN; ++i) v[4 * h + i] = y[4 * h + i] * by;
    const int b = c0 / 128 + (kOne ? lane / 16 : h);
    if ((kOne ? lane % 16 : lane) == 0 && b < nb && cols > 0) a.s[row * nb + b] = scale;
  }
  uint32_t code[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) code[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  uint8_t* q = a.q + row * a.cols + c0;
  if constexpr (MAP == kMap8) {
    if (c0 + 8 * lane < cols)
      *reinterpret_cast<uint2*>(q + 8 * lane) = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
  } else if constexpr (MAP == kMap4) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (c0 + 128 * h + 4 * lane < cols)
        *reinterpret_cast<uint32_t*>(q + 128 * h + 4 * lane) = code[2 * h] | code[2 * h + 1] << 16;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = rows::column<MAP, LANES>(lane, i);
      if (c0 + c < cols) q[c] = (uint8_t)(code[i / 2] >> (8 * (i & 1)));
    }
  }
}

// blockDim.x / 32 warps a row, warp w with chunks w, w + W, ..; blockDim.y rows a block. With LANES < 32 a warp
// has 32 / LANES narrow rows.
template <int XT, int RT, int MAP, bool FP8, int CPW, int LANES, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) norm_kernel(const Args a) {
  __shared__ float part[32];
  constexpr int kRT = RT == kNone ? XT : RT;
  const int lane = (threadIdx.x & 31) % LANES, warp = threadIdx.x >> 5, W = LANES == 32 ? blockDim.x >> 5 : 1;
  const int64_t row = ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * (32 / LANES) + (threadIdx.x & 31) / LANES;
  const int cols = row < a.rows ? a.cols : 0;
  float t[CPW][8];
  {
    Chunk<XT, MAP, LANES> x[CPW];
    Chunk<kRT, MAP, LANES> r[CPW];
    const char* xr = static_cast<const char*>(a.x) + row * a.ldx * rows::kSize<XT>;
    const char* rr = RT == kNone ? nullptr : static_cast<const char*>(a.r) + row * a.ldr * rows::kSize<kRT>;
#pragma unroll
    for (int j = 0; j < CPW; ++j) {
      const int c0 = (warp + j * W) * kChunk;
      x[j].load(xr, c0, cols, lane);
      if (RT != kNone) r[j].load(rr, c0, cols, lane);
    }
#pragma unroll
    for (int j = 0; j < CPW; ++j) {
      x[j].values(t[j]);
      if (RT != kNone) {
        float f[8];
        r[j].values(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[j][i] += f[i];
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < CPW; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(t[j][i], t[j][i], ss);
  ss = lanes_sum<LANES>(ss);
  if (W > 1) {
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = lanes_sum(lane < W ? part[lane] : 0.f);
  }
  const float rstd = __frsqrt_rn(__fdiv_rn(ss, (float)a.cols) + a.eps);
#pragma unroll
  for (int j = 0; j < CPW; ++j) {
    const int c0 = (warp + j * W) * kChunk;
    if (LANES == 32 && c0 >= cols) break;
    if (RT != kNone && a.total)
      rows::store<kRT, MAP, LANES>(static_cast<char*>(a.total) + row * a.cols * rows::kSize<kRT>, c0, cols, lane, t[j]);
    float y[8], w[8];
    load_weight<XT, MAP, LANES>(a.w, a.w_f32, c0, a.cols, lane, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = t[j][i] * rstd * w[i];
    if (a.y) rows::store<XT, MAP, LANES>(static_cast<char*>(a.y) + row * a.cols * rows::kSize<XT>, c0, cols, lane, y);
    if (FP8) quantize<MAP, LANES>(a, row, c0, cols, lane, y);
  }
}

struct BackArgs {
  const void* dy;
  const void* t;
  const void* dt;
  const void* w;
  void* dx;
  void* dr;
  float* part;   // [blocks][cols] or nullptr: no gradient of the weight
  int64_t rows, ldt;
  int cols, w_f32;
  float eps;
  int stage, stages;  // rows that are not whole 16 bytes: words of a stage, and stages
};

constexpr int kGroups = 8;  // warps with rows of their own in a block, where a warp holds one row or several

// A thread's numbers of the rows to come: stages of dy, t and dt, each kWords 16-byte words a chunk. Word w of a stage
// lies at w * threads + thread, so a warp's words are consecutive. A thread reads back what it copied itself: no
// barrier.
template <int TYPE, int TT, int CPW>
struct Ring {
  static constexpr int kDy = TYPE == MOE_TYPE_F32 ? 2 : 1, kT = TT == MOE_TYPE_F32 ? 2 : 1;
  static constexpr int kWords = CPW * (kDy + 2 * kT);
  static constexpr int bytes(int threads, int stages) { return 16 * kWords * threads * stages; }
};

constexpr int kMaxRing = 208 * 1024;  // bytes of a block's stages, at most

// Rows in flight a thread: two, or one where two would not fit (wide fp32 rows).
template <int TYPE, int TT, int CPW, int THREADS>
constexpr int kStages = Ring<TYPE, TT, CPW>::bytes(THREADS, 2) <= kMaxRing ? 2 : 1;

// Rows that are not whole 16 bytes: a row's warps (or its lanes) copy it as the 16-byte words that cover it, and read
// their numbers out of those behind a barrier. Its first word may begin in the row before, its last one is copied up to the row's
// end.
__host__ __device__ __forceinline__ int covering(int cols, int size) { return (cols * size + 15 + 15) / 16; }  // words, at most

// Persistent: a thread has the same columns in every row, so it keeps the weight and the weight's gradient of them in
// registers, while later rows are copied into shared memory. One row at a time by all warps of a block, or, with GROUPS
// > 1, a row by each warp, or 32 / LANES narrow ones.
template <int TYPE, int TT, int MAP, int CPW, int LANES, int GROUPS, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 256 ? 4 : THREADS <= 512 ? 2 : 1) back_kernel(const BackArgs a) {
  extern __shared__ uint4 ring[];
  __shared__ float2 part[2][32];
  __shared__ float dw_part[GROUPS > 1 ? GROUPS : 1][GROUPS > 1 ? kChunk : 1];
  using R = Ring<TYPE, TT, CPW>;
  constexpr int S = kStages<TYPE, TT, CPW, THREADS>;
  const int lane = (threadIdx.x & 31) % LANES, warp = GROUPS > 1 ? 0 : threadIdx.x >> 5;
  const int W = GROUPS > 1 ? 1 : blockDim.x >> 5;
  const int group = GROUPS > 1 ? threadIdx.x >> 5 : 0;
  float w[CPW][8], dw[CPW][8];
#pragma unroll
  for (int j = 0; j < CPW; ++j) {
    load_weight<TYPE, MAP, LANES>(a.w, a.w_f32, (warp + j * W) * kChunk, a.cols, lane, w[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
  }
  using Dy = std::integral_constant<int, TYPE>;
  using T = std::integral_constant<int, TT>;
  const char* const from[3] = {static_cast<const char*>(a.dy), static_cast<const char*>(a.t), static_cast<const char*>(a.dt)};
  const int64_t pitch[3] = {(int64_t)a.cols * rows::kSize<TYPE>, a.ldt * rows::kSize<TT>, (int64_t)a.cols * rows::kSize<TT>};
  // first word of dy, t and dt in a stage
  const int words[3] = {0, MAP == kMap1 ? covering(a.cols, rows::kSize<TYPE>) : CPW * R::kDy,
                        MAP == kMap1 ? covering(a.cols, rows::kSize<TYPE>) + covering(a.cols, rows::kSize<TT>)
                                     : CPW * (R::kDy + R::kT)};
  constexpr int kRows = 32 / LANES;  // of a warp
  const int sub = (threadIdx.x & 31) / LANES;  // the lane's row of those
  uint4* const mine = MAP == kMap1 ? ring + (group * kRows + sub) * a.stages * a.stage : ring;  // of this row
  auto copy = [&](auto type, int which, int slot, int64_t row) {
    constexpr int kType = decltype(type)::value;
    const char* p = from[which] + row * pitch[which];
    if constexpr (MAP == kMap1) {
      const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15), end = off + a.cols * rows::kSize<kType>;
      for (int b = 16 * (GROUPS > 1 ? lane : threadIdx.x); b < end; b += 16 * LANES * W)
        rows::copy16(smem_u32(mine + slot * a.stage + words[which]) + b, p - off + b, min(16, end - b));
    } else {
      constexpr bool kHalves = kType != MOE_TYPE_F32 && MAP == kMap4;  // 8 bytes and 8 bytes of one word
      constexpr int kN = kType == MOE_TYPE_F32 ? 2 : 1;
#pragma unroll
      for (int j = 0; j < CPW; ++j)
#pragma unroll
        for (int n = 0; n < (kHalves ? 2 : kN); ++n) {
          const int c = (warp + j * W) * kChunk + rows::column<MAP>(lane, 4 * n);
          const bool there = c < a.cols && (LANES == 32 || row < a.rows);
          const char* src = there ? p + (int64_t)c * rows::kSize<kType> : from[which];
          const int word = (slot * R::kWords + words[which] + j * kN + (kHalves ? 0 : n)) * blockDim.x + threadIdx.x;
          if constexpr (kHalves)
            rows::copy8(smem_u32(ring + word) + 8 * n, src, there ? 8 : 0);
          else
            rows::copy16(smem_u32(ring + word), src, there ? 16 : 0);
        }
    }
  };
  auto numbers = [&](auto type, int which, int slot, int64_t row, int j, float (&f)[8]) {
    constexpr int kType = decltype(type)::value;
    Chunk<kType, MAP, LANES> c;
    if constexpr (MAP == kMap1) {
      const int off = (int)(reinterpret_cast<uintptr_t>(from[which] + row * pitch[which]) & 15);
      c.load(reinterpret_cast<const char*>(mine + slot * a.stage + words[which]) + off, (warp + j * W) * kChunk, a.cols, lane);
    } else {
      constexpr int kN = kType == MOE_TYPE_F32 ? 2 : 1;
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        const uint4 v = ring[(slot * R::kWords + words[which] + j * kN + n) * blockDim.x + threadIdx.x];
        c.w[4 * n] = v.x, c.w[4 * n + 1] = v.y, c.w[4 * n + 2] = v.z, c.w[4 * n + 3] = v.w;
      }
    }
    c.values(f);
  };
  const int64_t step = (int64_t)gridDim.x * GROUPS * kRows;
  int64_t first = ((int64_t)blockIdx.x * GROUPS + group) * kRows;  // the warp's
  auto fetch = [&](int slot, int64_t at) {
    if (at < a.rows) {
      const int64_t row = at + sub;
      if (MAP != kMap1 || LANES == 32 || row < a.rows) {
        copy(Dy{}, 0, slot, row);
        copy(T{}, 1, slot, row);
        if (a.dt) copy(T{}, 2, slot, row);
      }
    }
    rows::copies_commit();
  };
  auto meet = [&]() {  // the warps of a row
    if (GROUPS > 1)
      __syncwarp();
    else
      __syncthreads();
  };
  const int stages = MAP == kMap1 ? a.stages : S;
  if (MAP != kMap1 || stages == 2) fetch(0, first);
  if (MAP != kMap1 && S == 2) fetch(1, first + step);
  for (int turn = 0, slot = 0; first < a.rows; first += step, turn ^= 1, slot = slot + 1 == stages ? 0 : slot + 1) {
    if constexpr (MAP == kMap1) {
      if (stages == 1) {
        meet();  // the row before has been read
        fetch(0, first);
      }
      rows::copies_wait<0>();
      meet();  // this row has come, and the one before has been read
      if (stages == 2) fetch(slot ^ 1, first + step);
    } else {
      rows::copies_wait<S - 1>();
    }
    const int64_t row = first + sub;
    const int cols = LANES == 32 || row < a.rows ? a.cols : 0;
    float ss = 0.f, gt = 0.f;
#pragma unroll
    for (int j = 0; j < CPW; ++j) {
      float g[8], v[8];
      numbers(Dy{}, 0, slot, row, j, g);
      numbers(T{}, 1, slot, row, j, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(v[i], v[i], ss);
        gt = fmaf(g[i] * w[j][i], v[i], gt);
      }
    }
    ss = lanes_sum<LANES>(ss);
    gt = lanes_sum<LANES>(gt);
    if (W > 1) {  // one barrier a row: the next row's sums go to the other half
      if (lane == 0) part[turn][warp] = make_float2(ss, gt);
      __syncthreads();
      const float2 p = lane < W ? part[turn][lane] : make_float2(0.f, 0.f);
      ss = lanes_sum(p.x);
      gt = lanes_sum(p.y);
    }
    const float rstd = __frsqrt_rn(__fdiv_rn(ss, (float)a.cols) + a.eps);
    const float dot = __fdiv_rn(gt, (float)a.cols) * rstd;  // mean(g n)
#pragma unroll
    for (int j = 0; j < CPW; ++j) {
      const int c0 = (warp + j * W) * kChunk;
      if (LANES == 32 && c0 >= cols) break;
      float g[8], v[8], d[8];
      numbers(Dy{}, 0, slot, row, j, g);
      numbers(T{}, 1, slot, row, j, v);
      if (a.dt) {
        numbers(T{}, 2, slot, row, j, d);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = v[i] * rstd;
        if (LANES == 32 || cols) dw[j][i] = fmaf(g[i], n, dw[j][i]);
        d[i] = fmaf(rstd, fmaf(-n, dot, g[i] * w[j][i]), d[i]);
      }
      if (a.dx) rows::store<TYPE, MAP, LANES>(static_cast<char*>(a.dx) + row * a.cols * rows::kSize<TYPE>, c0, cols, lane, d);
      if (a.dr) rows::store<TT, MAP, LANES>(static_cast<char*>(a.dr) + row * a.cols * rows::kSize<TT>, c0, cols, lane, d);
    }
    if constexpr (MAP != kMap1) fetch(slot, first + S * step);
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!a.part) return;
  if constexpr (GROUPS > 1) {  // a warp's rows, then the block's warps, in order
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int o = LANES; o < 32; o <<= 1) dw[0][i] += __shfl_xor_sync(0xffffffffu, dw[0][i], o);
      if ((threadIdx.x & 31) < LANES) dw_part[group][rows::column<MAP, LANES>(lane, i)] = dw[0][i];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += 32 * GROUPS) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < GROUPS; ++k) sum += dw_part[k][c];
      a.part[(int64_t)blockIdx.x * a.cols + c] = sum;
    }
  } else {
#pragma unroll
    for (int j = 0; j < CPW; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (warp + j * W) * kChunk + rows::column<MAP>(lane, i);
        if (c < a.cols) a.part[(int64_t)blockIdx.x * a.cols + c] = dw[j][i];
      }
  }
}

// The weight's gradient from the blocks' sums, in block order: 32 columns a block, 32 warps over the sums.
__global__ void __launch_bounds__(1024) dweight_kernel(const float* part, int n, int cols, int type, void* dw) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // it is launched beside the other kernel's end
  float sum = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int b = warp; b < n; b += 32) sum += part[(int64_t)b * cols + c];
  }
  sums[warp][lane] = sum;
  __syncthreads();
  sum = lanes_sum(sums[lane][warp]);
  if (lane == 0 && blockIdx.x * 32 + warp < cols) {
    const int at = blockIdx.x * 32 + warp;
    if (type == MOE_TYPE_F32)
      rows::store_bits<MOE_TYPE_F32>(dw, at, rows::bits_of<MOE_TYPE_F32>(sum));
    else if (type == MOE_TYPE_BF16)
      rows::store_bits<MOE_TYPE_BF16>(dw, at, rows::bits_of<MOE_TYPE_BF16>(sum));
    else
      rows::store_bits<MOE_TYPE_F16>(dw, at, rows::bits_of<MOE_TYPE_F16>(sum));
  }
}

template <int V>
using Int = std::integral_constant<int, V>;

// Narrow rows take an access of 8 columns a lane where they are whole ones, else number by number.
bool by_words(int cols) { return cols > 128 || cols % 8 == 0; }

// f(type, the other type, map, lanes of a row) of rows of `type` beside rows of `other` (kNone, the same, or fp32)
template <class F>
cudaError_t with_types(int type, int other, bool aligned, int lanes, F&& f) {
  auto mapped = [&](auto T, auto O) {
    constexpr int kAligned = decltype(T)::value == MOE_TYPE_F32 || decltype(O)::value == MOE_TYPE_F32 ? kMap4 : kMap8;
    if (!aligned) {
      if (lanes == 4) return f(T, O, Int<kMap1>{}, Int<4>{});
      if (lanes == 8) return f(T, O, Int<kMap1>{}, Int<8>{});
      if (lanes == 16) return f(T, O, Int<kMap1>{}, Int<16>{});
      return f(T, O, Int<kMap1>{}, Int<32>{});
    }
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

cudaError_t launch_rms_norm(const RmsNormDesc& d, cudaStream_t stream) {
  rn::Args a;
  a.x = d.x;
  a.r = d.residual;
  a.w = d.weight;
  a.y = d.y;
  a.total = d.total;
  a.q = static_cast<uint8_t*>(d.q);
  a.s = d.s;
  a.rows = d.rows;
  a.ldx = d.ldx;
  a.ldr = d.ldr;
  a.cols = d.cols;
  a.w_f32 = d.weight_type == MOE_TYPE_F32;
  a.eps = d.eps;
  const bool aligned = rows::whole(d.type, d.cols) && (d.rows == 1 || rows::whole(d.type, d.ldx)) &&
                       (d.rows == 1 || !d.residual || rows::whole(d.type, d.ldr)) && rn::by_words(d.cols);
  const int chunks = (int)cdiv(d.cols, rows::kChunk);
  // two chunks a warp wherever there are two (65536 x 384 bf16 31 us, with one 36; 32768 x 2048 with codes 91 and 97;
  // 32768 x 512 fp32 with codes 44.8 and 44.1); eight rows a block where a warp holds one or several
  const int cpw = chunks > 1 ? 2 : 1;
  const int W = (int)cdiv(chunks, cpw), G = W == 1 ? 8 : 1;
  const int lanes = rows::lanes_of(d.cols);
  return rn::with_types(d.type, d.residual ? d.residual_type : rn::kNone, aligned, lanes, [&](auto T, auto R, auto M, auto L) {
    constexpr int kT = decltype(T)::value, kR = decltype(R)::value, kM = decltype(M)::value, kL = decltype(L)::value;
    auto go = [&](auto kernel) {
      kernel<<<(unsigned)cdiv(d.rows, G * (32 / kL)), dim3(32 * W, G), 0, stream>>>(a);
      return cudaGetLastError();
    };
    auto sized = [&](auto Q) {
      constexpr bool kQ = decltype(Q)::value != 0;
      if constexpr (kL == 32) {
        if (cpw == 2)
          return W <= 16 ? go(rn::norm_kernel<kT, kR, kM, kQ, 2, 32, 512, 3>) : go(rn::norm_kernel<kT, kR, kM, kQ, 2, 32, 1024, 1>);
      }
      return go(rn::norm_kernel<kT, kR, kM, kQ, 1, kL, 256, 4>);
    };
    return d.q ? sized(rn::Int<1>{}) : sized(rn::Int<0>{});
  });
}

namespace rn {

// Chunks of a warp, and warps of a row (2048 columns: 83 us with two chunks, 88 with one; 512 columns: 63 and 53).
int back_chunks(int cols) { return cols > 4 * rows::kChunk ? 2 : 1; }
int back_warps(int cols) { return (int)cdiv(cdiv(cols, rows::kChunk), back_chunks(cols)); }

}  // namespace rn

// Blocks of the gradient's kernel, at most: as many as run at once (fewer where shared memory holds fewer), each at
// least one row.
int rms_norm_backward_blocks(int64_t rows, int cols) {
  const int W = rn::back_warps(cols), G = W == 1 ? rn::kGroups : 1;
  const int per_sm = W * G <= 8 ? 32 / (W * G) : W <= 14 ? 28 / W : W <= 16 ? 2 : 1;
  // a block of few rows has little to add up: four at least for another block an SM (1000 x 4096 bf16 14.2 us, without
  // 16.4)
  const int64_t few = cdiv(cdiv(rows, G), (int64_t)kNumSMsHint * 4);
  return (int)std::max<int64_t>(1, std::min<int64_t>(cdiv(rows, G), kNumSMsHint * std::min<int64_t>(per_sm, few)));
}

cudaError_t launch_rms_norm_backward(const RmsNormBackwardDesc& d, int* launches, cudaStream_t stream) {
  rn::BackArgs a;
  a.dy = d.dy;
  a.t = d.total;
  a.dt = d.dtotal;
  a.w = d.weight;
  a.dx = d.dx;
  a.dr = d.dresidual;
  a.part = d.dweight ? static_cast<float*>(d.ws) : nullptr;
  a.rows = d.rows;
  a.ldt = d.ldt;
  a.cols = d.cols;
  a.w_f32 = d.weight_type == MOE_TYPE_F32;
  a.eps = d.eps;
  const bool aligned = rows::whole(d.type, d.cols) && (d.rows == 1 || rows::whole(d.type, d.ldt)) && rn::by_words(d.cols);
  const int W = rn::back_warps(d.cols);
  int grid = rms_norm_backward_blocks(d.rows, d.cols);
  *launches = d.dweight ? 2 : 1;
  auto fit = [&](int smem) {  // blocks an SM's shared memory holds, each with 10 KB of its own at most
    grid = (int)std::min<int64_t>(grid, (int64_t)kNumSMsHint * std::max(1, 226 * 1024 / (smem + (W == 1 ? 10 : 2) * 1024)));
  };
  const int lanes = rows::lanes_of(d.cols);
  cudaError_t e = rn::with_types(d.type, d.total_type, aligned, lanes, [&](auto T, auto R, auto M, auto L) {
    constexpr int kT = decltype(T)::value, kM = decltype(M)::value, kL = decltype(L)::value;
    constexpr int kR = decltype(R)::value == rn::kNone ? kT : decltype(R)::value;
    auto go = [&](auto C, auto G, auto N, int threads) {
      constexpr int kC = decltype(C)::value, kN = decltype(N)::value, kG = decltype(G)::value;
      auto kernel = rn::back_kernel<kT, kR, kM, kC, kL, kG, kN>;
      static PerDevice<bool> attr;  // one for each kernel
      bool set = false;
      cudaError_t r = per_device<bool>(
          attr,
          [&](bool& v) {
            const cudaError_t x = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, rn::kMaxRing);
            v = x == cudaSuccess;
            return x;
          },
          &set);
      if (r != cudaSuccess) return r;
      int smem = rn::Ring<kT, kR, kC>::bytes(threads, rn::kStages<kT, kR, kC, kN>);
      if (kM == rows::kMap1) {
        a.stage = rn::covering(d.cols, rows::kSize<kT>) + (d.dtotal ? 2 : 1) * rn::covering(d.cols, rows::kSize<kR>);
        const int held = kG * (32 / kL);  // rows of a block
        a.stages = 2 * held * a.stage * 16 <= rn::kMaxRing ? 2 : 1;
        smem = a.stages * held * a.stage * 16;
      }
      fit(smem);
      grid = (int)std::min<int64_t>(grid, cdiv(d.rows, kG * (32 / kL)));
      kernel<<<grid, threads, smem, stream>>>(a);
      return cudaGetLastError();
    };
    if (d.cols <= rows::kChunk) return go(rn::Int<1>{}, rn::Int<rn::kGroups>{}, rn::Int<32 * rn::kGroups>{}, 32 * rn::kGroups);
    if constexpr (kL == 32) {
      // odd rows so wide that an SM holds one block of them: one chunk a warp, for twice the warps (8192 x 7167 fp32
      // 161 us, with two chunks 201)
      if (kM == rows::kMap1 && d.cols > 4 * rows::kChunk && d.cols <= 32 * rows::kChunk &&
          2 * (rn::covering(d.cols, rows::kSize<kT>) + (d.dtotal ? 2 : 1) * rn::covering(d.cols, rows::kSize<kR>)) * 16 > 110 * 1024)
        return go(rn::Int<1>{}, rn::Int<1>{}, rn::Int<1024>{}, 32 * (int)cdiv(d.cols, rows::kChunk));
      if (rn::back_chunks(d.cols) == 1) return go(rn::Int<1>{}, rn::Int<1>{}, rn::Int<256>{}, 32 * W);
      if (W <= 8) return go(rn::Int<2>{}, rn::Int<1>{}, rn::Int<256>{}, 32 * W);
      if (W <= 14) return go(rn::Int<2>{}, rn::Int<1>{}, rn::Int<448>{}, 32 * W);
      if (W <= 16) return go(rn::Int<2>{}, rn::Int<1>{}, rn::Int<512>{}, 32 * W);
      return go(rn::Int<2>{}, rn::Int<1>{}, rn::Int<1024>{}, 32 * W);
    }
    return cudaErrorInvalidValue;  // narrow rows have one warp
  });
  if (e != cudaSuccess || !d.dweight) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)cdiv(d.cols, 32));
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rn::dweight_kernel, (const float*)a.part, grid, d.cols, d.weight_type, d.dweight);
}

}  // namespace moe
