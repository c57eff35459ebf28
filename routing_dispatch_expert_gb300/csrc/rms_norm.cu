// Root-mean-square norm of the sum of a row and its residual, with an output in 8 bits. (Its gradient is in
// rms_norm_backward.cu.)
//
//   t = x + r,  n = t * rstd,  rstd = 1 / sqrt(mean(t^2) + eps),  y = n * w
//   scale of 128 columns = amax |y| / 448 (at least 2^-126; 1 where all are 0), code = e4m3(RN(y / scale))
//
// Everything is fp32: the sum is normalised and quantised before it is rounded for the residual stream, and each output
// is rounded once.
//
// Bound by HBM: a row is read once and held on the SM between its reduction and its outputs. One GB300, out of HBM (a
// copy's rate is 6.78 TB/s), x and residual of one type:
//   16384 x 7168 bf16 to bf16 and e4m3   163 us, 6.5 TB/s     8192 x 7168 fp32   137 us, 6.9 TB/s
//   65536 x 512 bf16                      41 us, 6.6          65536 x 64 bf16    6.6 us, 5.1
//   8192 x 7166 bf16 (with codes)         94 us, 5.0 (100)    65536 x 34 bf16    5.8 us, 3.1
//   8192 x 7167 bf16 (with codes)        101 us, 4.6 (135)    65536 x 33 bf16    6.5 us, 2.7
//   one row of 4096                      2.7 us, launch
//   16384 x 7168 bf16, fp32 residual     202 us, 7.0 TB/s (240 with codes, 6.4)
// 16-bit rows that are not whole 16 bytes are bound by their accesses of one number or two. Three blocks of 448 threads
// an SM for 7168 columns, so that one block's loads run beside another's sums: 40 registers, for which the weight is
// loaded behind the reduction and the kernels with codes spill up to 36 bytes (two blocks: 192 us). Rows of up to 128
// columns share a warp (65536 x 64 bf16 6.6 us, with a warp a row 16.7; 65536 x 33 6.5 and 18.8).
#include <cuda_fp8.h>

#include <algorithm>

#include "rms_norm.cuh"

namespace moe {
namespace rn {

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

// Codes and scales of a chunk: two blocks of 128 columns. The codes are e4m3(RN(y / scale)), those of the FP8 layer's
// rows. 1 / scale is taken as by + rest, by rounded down and rest what it lacks, and the quotient as fma(y, by, y * rest):
// the product by a constant in two parts of Brisebarre and Muller, "Correctly rounded multiplication by arbitrary
// precision constants" (2008). It is RN(y / scale) unless the quotient lies within 2^-46 of itself from the middle of two
// fp32 numbers (scales below 2^100; past them rest loses bits). rest is not negative, so zeros keep their sign. 16384 x
// 7168 to codes 163 us; with a division a number 174; by the rounded reciprocal alone 162, one code in 10^6 another, next
// to a midpoint. The largest magnitude is taken over the bits, under which a NaN is larger than every number: a block
// that holds an infinity or a NaN stands for NaN throughout.
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
    const float by = __frcp_rd(scale), e = fmaf(-by, scale, 1.f);  // 1 / scale = by / (1 - e) = by (1 + e + e^2 + ..)
    const float rest = by > 0.f ? fmaf(e, e, e) * by : 0.f;         // 0 under an infinite scale
#pragma unroll
    for (int i = 0; i < kN; ++i) v[4 * h + i] = fmaf(y[4 * h + i], by, y[4 * h + i] * rest);
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
  } else if constexpr (MAP == kMap2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = rows::column<MAP, LANES>(lane, 2 * i);
      if (c0 + c < cols) *reinterpret_cast<uint16_t*>(q + c) = (uint16_t)code[i];
    }
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
  const bool even = d.cols % 2 == 0 && (d.rows == 1 || (d.ldx % 2 == 0 && (!d.residual || d.ldr % 2 == 0)));
  const int lanes = rows::lanes_of(d.cols);
  return rn::with_types(d.type, d.residual ? d.residual_type : rn::kNone, aligned, even, lanes, [&](auto T, auto R, auto M, auto L) {
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

}  // namespace moe
