// Gradient of the root-mean-square norm (rms_norm.cu).
//
//   t: the total that was normalised, n = t * rstd, rstd = 1 / sqrt(mean(t^2) + eps), g = dy * w
//   dt = rstd * (g - n * mean(g n)) + (the gradient that reaches t from elsewhere)
//   dw = sum over the rows of dy * n
//
// fp32, each output rounded once. rstd is made again from t, which is read anyway, instead of being stored.
//
// Bound by HBM: a row is read once and held on the SM between its sums and its outputs. One GB300, out of HBM (a copy's
// rate is 6.78 TB/s), with the residual stream's gradient:
//   16384 x 7168 bf16  143 us, 6.6 TB/s     8192 x 7168 fp32  138 us, 6.8 TB/s
//   65536 x 512 bf16    53 us, 5.0          65536 x 64 bf16   11.6 us, 2.9
//   8192 x 7166 bf16   104 us, 4.5          65536 x 34 bf16   13 us, 1.4
//   8192 x 7167 bf16   139 us, 3.4          8192 x 7167 fp32  161 us, 5.8
//   65536 x 33 bf16   14.7 us, 1.2          one row of 4096   5.5 us, two launches
// 16-bit rows that are not whole 16 bytes are bound by their accesses of one number or two, in shared memory (dy and t
// twice) and to HBM. Narrow rows share a warp and wait for no other (65536 x 33 14.7 us, with a warp a row 39); they are
// bound by instructions, two sums over the lanes a row, odd ones by reads of one number, and by the second launch over up
// to 608 blocks' sums; whole ones of one 16-bit type spill 120 bytes at the 64 registers that four blocks an SM leave.
// One round of blocks, rows copied ahead into shared memory (rows held in registers instead, one block an SM: 167 us;
// two, spilling: 226).
#include <algorithm>

#include "rms_norm.cuh"

namespace moe {
namespace rn {

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
// their numbers out of those behind a barrier (of the warp, where it has rows of its own). Its first word may begin in
// the row before, its last one is copied up to the row's end.
__host__ __device__ __forceinline__ int covering(int cols, int size) {  // words, at most
  return (cols * size + 15 + 15) / 16;
}

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
  const int words[3] = {0, kOdd<MAP> ? covering(a.cols, rows::kSize<TYPE>) : CPW * R::kDy,
                        kOdd<MAP> ? covering(a.cols, rows::kSize<TYPE>) + covering(a.cols, rows::kSize<TT>)
                                     : CPW * (R::kDy + R::kT)};
  constexpr int kRows = 32 / LANES;  // of a warp
  const int sub = (threadIdx.x & 31) / LANES;  // the lane's row of those
  uint4* const mine = kOdd<MAP> ? ring + (group * kRows + sub) * a.stages * a.stage : ring;  // of this row
  auto copy = [&](auto type, int which, int slot, int64_t row) {
    constexpr int kType = decltype(type)::value;
    const char* p = from[which] + row * pitch[which];
    if constexpr (kOdd<MAP>) {
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
    if constexpr (kOdd<MAP>) {
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
      if (!kOdd<MAP> || LANES == 32 || row < a.rows) {
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
  const int stages = kOdd<MAP> ? a.stages : S;
  if (!kOdd<MAP> || stages == 2) fetch(0, first);
  if (!kOdd<MAP> && S == 2) fetch(1, first + step);
  for (int turn = 0, slot = 0; first < a.rows; first += step, turn ^= 1, slot = slot + 1 == stages ? 0 : slot + 1) {
    if constexpr (kOdd<MAP>) {
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
    if constexpr (!kOdd<MAP>) fetch(slot, first + S * step);
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

// Chunks of a warp, and warps of a row (2048 columns: 83 us with two chunks, 88 with one; 512 columns: 63 and 53).
int back_chunks(int cols) { return cols > 4 * rows::kChunk ? 2 : 1; }
int back_warps(int cols) { return (int)cdiv(cdiv(cols, rows::kChunk), back_chunks(cols)); }

}  // namespace rn

// Blocks of the gradient's kernel, at most: as many as run at once (fewer where shared memory holds fewer), each at
// least one row. An SM's registers hold 32 warps of 64 a thread, 28 of the 72 that rows of 9 to 14 warps take.
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
  const bool even = d.cols % 2 == 0 && (d.rows == 1 || d.ldt % 2 == 0);
  const int lanes = rows::lanes_of(d.cols);
  cudaError_t e = rn::with_types(d.type, d.total_type, aligned, even, lanes, [&](auto T, auto R, auto M, auto L) {
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
      if (rows::kOdd<kM>) {
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
      if (rows::kOdd<kM> && d.cols > 4 * rows::kChunk && d.cols <= 32 * rows::kChunk &&
          2 * (rn::covering(d.cols, rows::kSize<kT>) + (d.dtotal ? 2 : 1) * rn::covering(d.cols, rows::kSize<kR>)) * 16 > 110 * 1024)
        return go(rn::Int<1>{}, rn::Int<1>{}, rn::Int<1024>{}, 32 * (int)cdiv(d.cols, rows::kChunk));
      if (rn::back_chunks(d.cols) == 1) return go(rn::Int<1>{}, rn::Int<1>{}, rn::Int<256>{}, 32 * W);
      if (W <= 8) return go(rn::Int<2>{}, rn::Int<1>{}, rn::Int<256>{}, 32 * W);
      // up to 14 warps, two blocks an SM have 72 registers a thread instead of 64 (16384 x 7168 bf16 143 us, with the
      // kernel for 16 warps 149; 8192 x 7166 104.5 and 113.8; 8192 x 4608 55 and 57)
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
