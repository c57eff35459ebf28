// Rows back from expert order to token order, added up with the route weights, and the gradient of that.
//
//   y[t] = base[t] + sum_j w[t, j] yd[p[t, j]]                      in slot order, fp32, rounded once
//   dyd[p[t, j]] = w[t, j] dy[t],   dw[t, j] = <yd[p[t, j]], dy[t]>  fp32
//
// Both go token by token, so that the k uses of a token's row meet; the k rows elsewhere are read (and written) once.
// The rows of a chunk are all loaded before any is worked on, and a token's positions are looked up once for many
// chunks.
//
// Bound by HBM. One GB300, k 8 (a copy's rate is 6.78 TB/s), with weights and base, and the gradient with the weights':
//   16384 x 7168 bf16 345 us, 6.8 TB/s   601 us, 6.6        8192 x 7168 fp32 331 us   589 us
//   65536 x 64 bf16    20 us, 4.4         28 us, 5.4        65536 x 33 bf16 22.5 us   40 us
//   8192 x 7166 bf16  210 us, 5.6        331 us, 6.0        8192 x 7167 bf16 257 us, 4.6   416 us, 4.8
// 16-bit rows that are not whole 16 bytes are bound by their accesses of one number or two. 64 x 512, k 2: 2.4 us, launch.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace moe {
namespace un {

using std::integral_constant;

// Rows and weights of the slots j0 .. j0 + KB - 1 of token t, in each of its LANES lanes; -1 past the last slot, and
// for positions outside the T k rows.
template <int KB, int LANES>
__device__ __forceinline__ void slots(const int32_t* inv_pos, const float* weights, int64_t t, int64_t T, int k, int j0,
                                      int (&row)[KB], float (&w)[KB]) {
  if constexpr (LANES == 32) {
    const int lane = threadIdx.x & 31;
    const bool in = lane < KB && j0 + lane < k;
    int r = in ? inv_pos[t * k + j0 + lane] : -1;
    if (r >= T * k) r = -1;
    const float v = in && weights ? weights[t * k + j0 + lane] : 1.f;
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      row[j] = __shfl_sync(0xffffffffu, r, j);
      w[j] = __shfl_sync(0xffffffffu, v, j);
    }
  } else {
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      const bool in = t < T && j0 + j < k;
      row[j] = in ? inv_pos[t * k + j0 + j] : -1;
      if (row[j] >= T * k) row[j] = -1;
      w[j] = in && weights ? weights[t * k + j0 + j] : 1.f;
    }
  }
}

// Blocks of 256 threads an SM holds: the registers of KB rows in flight, by the times. Rows number by number take a
// register a number (65536 x 511 bf16, the gradient: two slots 80 us with four blocks, 98 with three; four slots 142 with
// three, 163 with four; eight slots 272 with two, 652 with three), by pairs one for two (8192 x 7166: 210 us with two
// blocks, 259 with three; the narrow rows of 65536 x 66 33.5 and 28.0). A few spilled words do not decide it: eight slots
// of whole 16-bit rows spill 68 bytes at three blocks and run at a copy's rate.
template <int TYPE, int MAP, int KB, int LANES = 32>
constexpr int kBlocks = MAP == rows::kMap2   ? (KB < 8 ? 4 : LANES == 32 ? 2 : 3)
                        : MAP == rows::kMap1 ? (KB == 8 ? 2 : KB == 4 ? 3 : 4)
                        : TYPE == MOE_TYPE_F32 ? (KB == 8 ? 2 : 3)
                                               : (KB == 8 ? 3 : 4);

struct AddArgs {
  const void* yd;
  const void* base;      // or nullptr
  const float* weights;  // [T, k] or nullptr
  const int32_t* inv_pos;
  void* y;
  int64_t T;
  int cols, chunks, k;
  int piece, pieces;  // chunks of a warp's work, and those works of a row
};

// A warp a piece of a token's row, or LANES lanes a whole narrow row: fp32, the base first and then the slots in order.
// KB: slots at a time, a power of two at or above k, at most 8.
template <int TYPE, int MAP, int KB, int LANES>
__global__ void __launch_bounds__(256, (kBlocks<TYPE, MAP, KB, LANES>)) unpermute_kernel(const AddArgs a) {
  constexpr int kTokens = 32 / LANES;
  const int lane = threadIdx.x & 31, sub = lane % LANES;
  const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  const int64_t items = LANES == 32 ? a.T * a.pieces : cdiv(a.T, kTokens);
  const int64_t pitch = (int64_t)a.cols * rows::kSize<TYPE>;
  for (int64_t it = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; it < items; it += warps) {
    const int64_t t = LANES == 32 ? it / a.pieces : it * kTokens + lane / LANES;
    const int first = LANES == 32 ? (int)(it - t * a.pieces) * a.piece : 0;
    const int last = LANES == 32 ? min(a.chunks, first + a.piece) : 1;
    const int cols = t < a.T ? a.cols : 0;
    int row[KB];
    float w[KB];
    slots<KB, LANES>(a.inv_pos, a.weights, t, a.T, a.k, 0, row, w);
    for (int c = first; c < last; ++c) {
      const int c0 = c * rows::kChunk;
      float sum[8];
      for (int j0 = 0; j0 < a.k; j0 += KB) {
        if (KB == 8 && a.k > KB) slots<KB, LANES>(a.inv_pos, a.weights, t, a.T, a.k, j0, row, w);
        rows::Chunk<TYPE, MAP, LANES> b, v[KB];
        if (j0 == 0) {
          if (a.base)
            b.load(static_cast<const char*>(a.base) + t * pitch, c0, cols, sub);
          else
            b.clear();
        }
#pragma unroll
        for (int j = 0; j < KB; ++j)
          if (row[j] >= 0) v[j].load(static_cast<const char*>(a.yd) + row[j] * pitch, c0, cols, sub);
        if (j0 == 0) b.values(sum);
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          if (row[j] < 0) continue;
          float f[8];
          v[j].values(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] = fmaf(w[j], f[i], sum[i]);
        }
        if (KB < 8) break;  // k is at most KB
      }
      rows::store<TYPE, MAP, LANES>(static_cast<char*>(a.y) + t * pitch, c0, cols, sub, sum);
    }
  }
}

struct SpreadArgs {
  const void* dy;
  const void* yd;        // or nullptr: no gradient of the weights
  const float* weights;  // [T, k] or nullptr
  const int32_t* inv_pos;
  const int32_t* held_at;
  void* dyd;
  float* dweights;  // [T, k] or nullptr
  int64_t T;
  int cols, chunks, k;
};

// A group of W warps a token (blockDim.x / 32, blockDim.y groups a block where W is 1), or LANES lanes a narrow row:
// its row of dy to its k rows of dyd, and their products with yd's rows, summed over the lanes and then the warps. At
// the end all threads clear the rows that hold nothing.
template <int TYPE, int MAP, int KB, int LANES>
__global__ void __launch_bounds__(256, (kBlocks<TYPE, MAP, KB>)) spread_kernel(const SpreadArgs a) {
  constexpr int kTokens = 32 / LANES;
  __shared__ float part[8][KB];
  const int lane = threadIdx.x & 31, sub = lane % LANES, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
  const int64_t pitch = (int64_t)a.cols * rows::kSize<TYPE>;
  const int64_t group = (int64_t)blockIdx.x * blockDim.y + threadIdx.y, groups = (int64_t)gridDim.x * blockDim.y;
  for (int64_t g0 = group * kTokens; g0 < a.T; g0 += groups * kTokens) {
    const int64_t t = g0 + lane / LANES;
    const int cols = t < a.T ? a.cols : 0;
    for (int j0 = 0; j0 < a.k; j0 += KB) {
      int row[KB];
      float w[KB], dot[KB];
      slots<KB, LANES>(a.inv_pos, a.weights, t, a.T, a.k, j0, row, w);
#pragma unroll
      for (int j = 0; j < KB; ++j) dot[j] = 0.f;
      for (int c = warp; c < a.chunks; c += W) {
        const int c0 = c * rows::kChunk;
        rows::Chunk<TYPE, MAP, LANES> dy, v[KB];
        dy.load(static_cast<const char*>(a.dy) + t * pitch, c0, cols, sub);
        if (a.yd) {
#pragma unroll
          for (int j = 0; j < KB; ++j)
            if (row[j] >= 0) v[j].load(static_cast<const char*>(a.yd) + row[j] * pitch, c0, cols, sub);
        }
        float g[8];
        dy.values(g);
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          if (row[j] < 0) continue;
          float f[8];
          if (a.yd) {
            v[j].values(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[j] = fmaf(g[i], f[i], dot[j]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = w[j] * g[i];
          rows::store<TYPE, MAP, LANES>(static_cast<char*>(a.dyd) + row[j] * pitch, c0, cols, sub, f);
        }
      }
      if (!a.dweights) continue;
      float mine = 0.f;
#pragma unroll
      for (int j = 0; j < KB; ++j) {
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
        if (LANES < KB && sub == j % LANES && t < a.T && j0 + j < a.k) a.dweights[t * a.k + j0 + j] = dot[j];
        if (sub == j) mine = dot[j];
      }
      if (LANES < KB) continue;  // narrow rows have one warp
      if (W == 1) {
        if (t < a.T && sub < KB && j0 + sub < a.k) a.dweights[t * a.k + j0 + sub] = mine;
        continue;
      }
      if (lane < KB) part[warp][lane] = mine;
      __syncthreads();
      if (threadIdx.x < KB && j0 + threadIdx.x < a.k) {
        float sum = 0.f;
        for (int i = 0; i < W; ++i) sum += part[i][threadIdx.x];
        a.dweights[t * a.k + j0 + threadIdx.x] = sum;
      }
      __syncthreads();
    }
  }
  const int64_t held = min(max((int64_t)*a.held_at, (int64_t)0), a.T * a.k), threads = (int64_t)blockDim.x * blockDim.y;
  rows::clear<rows::kSize<TYPE>>(a.dyd, held * pitch, a.T * a.k * pitch,
                                 blockIdx.x * threads + threadIdx.y * blockDim.x + threadIdx.x, gridDim.x * threads);
}

// f(type, map, slots at a time, lanes of a row). Rows of up to 128 columns share a warp (65536 x 64 bf16 20 us, with a warp
// a row 45; 65536 x 33 22.5 and 69); two or four slots leave registers for more blocks (65536 x 512, k 2: 52 us, with eight
// 58; 65536 x 511, k 4: 92 and 112).
template <class F>
cudaError_t with_rows(int type, int64_t cols, int k, F&& f) {
  const bool whole = rows::whole(type, cols);
  auto typed = [&](auto T) {
    constexpr int kT = decltype(T)::value;
    constexpr int kAligned = kT == MOE_TYPE_F32 ? rows::kMap4 : rows::kMap8;
    using One = integral_constant<int, rows::kMap1>;
    using Two = integral_constant<int, kT == MOE_TYPE_F32 ? rows::kMap1 : rows::kMap2>;
    using Whole = integral_constant<int, kAligned>;
    using Eight = integral_constant<int, rows::kMap8>;  // narrow rows: 8 columns a lane whatever the type
    integral_constant<int, 2> two;
    integral_constant<int, 4> four;
    const int lanes = rows::lanes_of(cols);
    integral_constant<int, 8> eight;
    integral_constant<int, 16> sixteen;
    integral_constant<int, 32> all;
    if (!whole || (lanes < 32 && cols % 8)) {
      auto by = [&](auto M) {
        auto odd = [&](auto L) { return k <= 2 ? f(T, M, two, L) : k <= 4 ? f(T, M, four, L) : f(T, M, eight, L); };
        return lanes == 4 ? odd(four) : lanes == 8 ? odd(eight) : lanes == 16 ? odd(sixteen) : odd(all);
      };
      return cols % 2 ? by(One{}) : by(Two{});
    }
    if (lanes <= 8) return k <= 2 ? f(T, Eight{}, two, eight) : f(T, Eight{}, eight, eight);
    if (lanes == 16) return k <= 2 ? f(T, Eight{}, two, sixteen) : f(T, Eight{}, eight, sixteen);
    return k <= 2 ? f(T, Whole{}, two, all) : k <= 4 ? f(T, Whole{}, four, all) : f(T, Whole{}, eight, all);
  };
  if (type == MOE_TYPE_F32) return typed(integral_constant<int, MOE_TYPE_F32>{});
  if (type == MOE_TYPE_BF16) return typed(integral_constant<int, MOE_TYPE_BF16>{});
  return typed(integral_constant<int, MOE_TYPE_F16>{});
}

}  // namespace un

cudaError_t launch_unpermute(const UnpermuteDesc& d, cudaStream_t stream) {
  un::AddArgs a;
  a.yd = d.yd;
  a.base = d.base;
  a.weights = d.weights;
  a.inv_pos = d.inv_pos;
  a.y = d.y;
  a.T = d.T;
  a.cols = d.cols;
  a.chunks = (int)cdiv(d.cols, rows::kChunk);
  a.k = d.k;
  // a warp's work: up to 16 chunks of a row, fewer where there would be less than 32 works an SM (7168 columns of 16384
  // tokens: 339 us with 14 chunks, 343 with 7 or 4, 480 with one, whose rows' numbers are then looked up for every
  // chunk)
  const int64_t pieces = std::max<int64_t>(cdiv(a.chunks, 16), std::min<int64_t>(a.chunks, cdiv(32 * num_sms(), a.T)));
  a.piece = (int)cdiv(a.chunks, pieces);
  a.pieces = (int)cdiv(a.chunks, a.piece);
  return un::with_rows(d.type, d.cols, d.k, [&](auto T, auto M, auto K, auto L) {
    constexpr int kL = decltype(L)::value;
    const int64_t items = kL == 32 ? a.T * a.pieces : cdiv(a.T, 32 / kL);
    const unsigned blocks = (unsigned)std::min<int64_t>(cdiv(items, 8), (int64_t)num_sms() * 16);
    un::unpermute_kernel<decltype(T)::value, decltype(M)::value, decltype(K)::value, kL><<<blocks, 256, 0, stream>>>(a);
    return cudaGetLastError();
  });
}

cudaError_t launch_unpermute_backward(const UnpermuteBackwardDesc& d, cudaStream_t stream) {
  un::SpreadArgs a;
  a.dy = d.dy;
  a.yd = d.dweights ? d.yd : nullptr;
  a.weights = d.weights;
  a.inv_pos = d.inv_pos;
  a.held_at = d.held;
  a.dyd = d.dyd;
  a.dweights = d.dweights;
  a.T = d.T;
  a.cols = d.cols;
  a.chunks = (int)cdiv(d.cols, rows::kChunk);
  a.k = d.k;
  // warps of a token: four, up to eight where few tokens would leave SMs idle (16384 tokens of 7168 columns: 600 us
  // with four or two, 637 with eight: every token ends in a barrier and a sum over the warps)
  const int64_t most = std::min<int64_t>(8, std::max<int64_t>(4, cdiv(24 * num_sms(), a.T)));
  const int W = (int)cdiv(a.chunks, cdiv(a.chunks, most)), G = W == 1 ? 8 : 1;
  return un::with_rows(d.type, d.cols, d.k, [&](auto T, auto M, auto K, auto L) {
    constexpr int kL = decltype(L)::value;
    const unsigned blocks = (unsigned)std::min<int64_t>(cdiv(a.T, G * (32 / kL)), (int64_t)num_sms() * 64 / (W * G));
    un::spread_kernel<decltype(T)::value, decltype(M)::value, decltype(K)::value, kL>
        <<<blocks, dim3(32 * W, G), 0, stream>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace moe
