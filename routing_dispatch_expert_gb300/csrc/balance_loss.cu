// The router's load-balance loss, its per-expert counts and mean probabilities, and its gradient.
//
// For a sequence s with n unmasked tokens, E experts and k choices a token:
//   p[t, e]  softmax over the experts of logits[t], or sigmoid(logits[t, e]) / sum over the experts
//   c[e]     assignments of the n tokens to expert e,    P[e] = mean over the n tokens of p[t, e]
//   L_s      = alpha * E / (k n) * sum_e c[e] P[e]
//   dL_s/dlogits[t, e] = alpha * E / (k n^2) * p[t, e] * d[t, e] * (c[e] - sum_j p[t, j] c[j])
// with d = 1 (softmax) or 1 - sigmoid(logits[t, e]); the counts carry no gradient.
//
// Both scores are one formula: p = w / sum w with w = exp(l - m) (softmax, m the row's maximum) or
// w = 1 / (e^c + e^(c - l)), c = min(m, 0): the sigmoid times e^-c, so that a row whose sigmoids all
// underflow keeps its ratios. A row of nothing but -inf has no probabilities: its p are 0.
//
// One GB300, 65536 tokens x 256 experts, k 8, 24 sequences, sigmoid, logits out of HBM: forward fp32 22.5 us (3.1 TB/s:
// 70 MB at a copy's rate are 10 us), bf16 21.3; backward 23.6 us (5.7 TB/s of 6.8) and 18.9. 512 tokens x 8 experts: 3.7
// and 2.7 us, launch and memory latency. The forward pass is bound by latency, not by instructions or HBM (38% and 36% of
// their peaks): an SM has work for 63% of the kernel's time and issues in 57% of those cycles, a third of its warps'
// waiting is for loads. It counts before the main loop, joins its warps at every piece of a sequence, and the second
// kernel adds 5 us. bf16 rows take as many memory instructions as fp32 ones (8 bytes a lane). Two rows in flight a warp
// instead of one, and three blocks an SM, changed nothing or spilled.
//
// Precision: fp32 throughout. That is the probabilities (weights() below: at most 2e-6 relative), their sums over
// tokens, the means, the sum over experts and the loss, and the gradient's factor dloss alpha E / (k n^2) c[e]. 64 bits
// for sums and factors would go through a pipe 60 times slower. Measured against 64 bits on the batch above: loss 7.6e-8
// and gradient up to 1.8e-7 relative, where sums, means and factors in 64 bits leave 6.8e-8 and up to 1.2e-7.
//
// Both directions read the logits once from HBM. A token is held by L lanes (L = E / 4 rounded up to a
// power of two, at most 32; each lane groups of 4 consecutive experts), and the sums over tokens are
// kept in registers while the tokens stream by; they are joined over the block in a fixed order, then
// over the blocks by a second kernel in block order, so results do not depend on timing.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace bl {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
  const void* logits;
  const int32_t* topk_idx;
  const int32_t* offsets;  // [S + 1] or nullptr: one sequence of all T tokens
  const uint8_t* mask;     // [T] or nullptr
  int T, E, k, S;
  int per_block;   // tokens of a block
  float alpha;
  float* psum;     // [blocks + S][E]
  int32_t* pcnt;   // [blocks + S][E]
  int32_t* pn;     // [blocks + S]
  float* loss;     // [S]
  int32_t* counts; // [S][E]
  float* mean;     // [S][E]
  int32_t* tokens; // [S]
};

// Approximate instructions, 2 ulp and 1: part of the 2e-6 above. Flushing to zero costs nothing here (what underflows is
// below 1e-38 of the row's largest) and saves the scaling around either.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// a float of another block of the cluster, by its shared::cluster address
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// first token of sequence s, within [0, T] whatever the offsets hold
__device__ __forceinline__ int seq_begin(const int32_t* offsets, int s, int S, int T) {
  if (!offsets) return s <= 0 ? 0 : T;
  return min(max(offsets[s], 0), T);
}
// last sequence in [0, S) that begins at or before token t (0 if none does)
__device__ __forceinline__ int seq_of(const int32_t* offsets, int S, int T, int t) {
  int lo = 0, hi = S - 1;
  if (!offsets) return 0;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seq_begin(offsets, mid, S, T) <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// The same for a whole warp and one token: the lanes look at 32 sequences at a time, one load instead of a chain of
// log2 S (offsets ascend, so the sequences that begin at or before t are the first ones).
__device__ __forceinline__ int seq_of_warp(const int32_t* offsets, int S, int T, int t) {
  if (!offsets) return 0;
  if (S > 1024) return seq_of(offsets, S, T, t);
  int n = 0;
  for (int s0 = 0; s0 < S; s0 += 32) {
    const int s = s0 + (threadIdx.x & 31);
    n += __popc(__ballot_sync(0xffffffffu, s < S && seq_begin(offsets, s, S, T) <= t));
  }
  return max(n - 1, 0);
}

// This lane's experts of a token, 4 (sub + L j) + i (j < EPL / 4, i < 4), as they lie in memory: nothing is done
// with them until values(), so that the loads of a token are in flight while another one is worked on.
template <bool BF16, int L, int EPL>
struct Row {
  uint32_t w[BF16 ? EPL / 2 : EPL];
  __device__ __forceinline__ void load(const void* logits, int64_t row, int E, int sub) {
    const bool vec = (E & 3) == 0;
#pragma unroll
    for (int j = 0; j < EPL / 4; ++j) {
      const int e = 4 * (sub + L * j);
      const int64_t at = row * E + e;
      if (BF16) {
        const uint16_t* p = static_cast<const uint16_t*>(logits) + at;
        if (vec && e < E) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          w[2 * j] = v.x, w[2 * j + 1] = v.y;
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i)  // 0xFF80: -inf
            w[2 * j + i] = (e + 2 * i < E ? p[2 * i] : 0xFF80u) | (e + 2 * i + 1 < E ? p[2 * i + 1] : 0xFF80u) << 16;
        }
      } else {
        const uint32_t* p = static_cast<const uint32_t*>(logits) + at;
        if (vec && e < E) {
          const uint4 v = *reinterpret_cast<const uint4*>(p);
          w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[4 * j + i] = e + i < E ? p[i] : 0xFF800000u;
        }
      }
    }
  }
  __device__ __forceinline__ void values(float (&l)[EPL]) const {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      l[i] = !BF16 ? __uint_as_float(w[i]) : i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
  }
};

template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  if (L == 32) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
  }
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// l becomes w, and 1 / sum w is returned: the probabilities are w times it. With DERIV d becomes 1 - sigmoid(l).
// The exponent is one fused multiply-add, fma(l, log2 e, -c log2 e): its own rounding is |x| 2^-24 for an exponent
// x, that of c log2 e is the same for the whole row and cancels; ex2.approx and rcp.approx add 2 ulp and 1. In all
// below 2e-6 down to probabilities of 1e-8 of the largest. The rounding that cancels is up to c 2^-25 in the exponent:
// harmless for c of 1e6 (a factor of 2^0.05 in every w), but past 1e9, where rows masked with a large negative number
// are, it would take every w to 0 or infinity. So the row is shifted first where c is large: l - c is exact or off by
// 2^-24 of the difference. A row of nothing but -inf has a sum of 0 and no probabilities; a NaN makes its whole row NaN.
constexpr float kShift = 1048576.0f;
template <bool SIGMOID, bool DERIV, int L, int EPL>
__device__ __forceinline__ float weights(float (&l)[EPL], float (&d)[DERIV ? EPL : 1]) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < EPL; ++i) m = fmaxf(m, l[i]);
  m = lanes_max<L>(m);
  float c = m == -INFINITY ? 0.f : m;
  if (SIGMOID) c = fminf(c, 0.f);
  float ec = 0.f;
  if (fabsf(c) > kShift) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] -= c;
    c = 0.f;  // and e^c is 0
  } else if (SIGMOID) {
    ec = ex2(c * kLog2e);
  }
  const float c2 = c * kLog2e;
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    if (SIGMOID) {
      const float u = ex2(fmaf(l[i], -kLog2e, c2));  // e^(c - l); inf for l = -inf: w = 0
      const float w = reciprocal(ec + u);
      // 1 - sigmoid = e^-l / (1 + e^-l); 1 in fp32 once u > 2^25, where u * w could be inf * 0
      if (DERIV) d[i] = u < 1e30f ? u * w : 1.0f;
      l[i] = w;
    } else {
      l[i] = ex2(fmaf(l[i], kLog2e, -c2));
    }
    z += l[i];
  }
  z = lanes_sum<L>(z);
  return z == 0.f ? 0.f : __fdividef(1.0f, z);
}

// loss, counts, mean and token count of sequence s from its sums: called by all threads of a block
// that together hold the experts [e0, e1); returns this thread's part of sum_e c P.
__device__ __forceinline__ float finish_expert(const Args& a, int s, int e, float sum, int cnt, int n) {
  const float mean = n > 0 ? __fdiv_rn(sum, (float)n) : 0.f;
  a.mean[(int64_t)s * a.E + e] = mean;
  a.counts[(int64_t)s * a.E + e] = cnt;
  return (float)cnt * mean;
}
__device__ __forceinline__ void finish_loss(const Args& a, int s, float dot, int n) {
  a.loss[s] = n > 0 ? a.alpha * (float)a.E * __fdiv_rn(dot, (float)a.k * (float)n) : 0.f;
  a.tokens[s] = n;
}

// sum over a block's threads, in a fixed order; the result is in every thread of warp 0
template <int WARPS>
__device__ __forceinline__ float block_sum(float v, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = lanes_sum<32>(v);
  __syncthreads();
  if (lane == 0) red[warp] = v;
  __syncthreads();
  return lanes_sum<32>(lane < WARPS ? red[lane] : 0.f);
}

constexpr int kMaxE = 1024;
constexpr int kHalf = kWarps / 2;

// Sums over the tokens of one block: for each sequence that has tokens in [b * per_block, ...) one
// entry b + s of psum, pcnt and pn (the pairs (b, s) that occur form a staircase, so b + s is unique).
// SINGLE: one block holds every token and writes the results itself.
template <bool SIGMOID, bool BF16, int L, int EPL, bool SINGLE>
__global__ void __launch_bounds__(kThreads, EPL > 8 ? 1 : 2) forward_kernel(const Args a) {
  constexpr int PER_WARP = 32 / L;           // tokens of a warp at a time
  constexpr int STRIDE = kWarps * PER_WARP;  // tokens of the block at a time
  __shared__ float part[kHalf][L * EPL];
  __shared__ int hist[L * EPL];
  __shared__ float red[kWarps];
  __shared__ int n_seq_tokens;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % L;
  const int b0 = blockIdx.x * a.per_block, b1 = min(a.T, b0 + a.per_block);
  if (!SINGLE) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int s = SINGLE ? 0 : seq_of_warp(a.offsets, a.S, a.T, b0), after; s < a.S; s = after) {
    const int begin = seq_begin(a.offsets, s, a.S, a.T);
    if (!SINGLE && begin >= b1) break;
    const int lo = max(begin, b0), hi = min(seq_begin(a.offsets, s + 1, a.S, a.T), b1);
    after = s + 1;
    // the next sequence with a token, past those that are empty
    if (!SINGLE && hi < b1) after = max(after, seq_of_warp(a.offsets, a.S, a.T, max(hi, b0)));
    if (!SINGLE && lo >= hi) continue;
    float acc[EPL], none[1];
    Row<BF16, L, EPL> cur;
#pragma unroll
    for (int i = 0; i < EPL; ++i) acc[i] = 0.f;
    // probabilities: the next token's logits are loaded before this one's are worked on (the first before the counts)
    auto fetch = [&](int base) {
      const int t = base + lane / L;
      const bool in = t < hi && (!a.mask || a.mask[t]);
      if (in) cur.load(a.logits, t, a.E, sub);
      return in;
    };
    int base = lo + warp * PER_WARP;
    bool in = base < hi && fetch(base);
    for (int e = threadIdx.x; e < a.E; e += kThreads) hist[e] = 0;
    if (threadIdx.x == 0) n_seq_tokens = 0;
    __syncthreads();
    // counts: whole numbers, so the order of the atomics does not show
    int n = 0;
    for (int t = lo + threadIdx.x; t < hi; t += kThreads) {
      if (a.mask && !a.mask[t]) continue;
      ++n;
      for (int j = 0; j < a.k; ++j) {
        const int e = a.topk_idx[(int64_t)t * a.k + j];
        if (e >= 0 && e < a.E) atomicAdd(&hist[e], 1);
      }
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0 && n) atomicAdd(&n_seq_tokens, n);
    for (; base < hi; base += STRIDE) {
      float l[EPL];
      const bool now = in;
      cur.values(l);
      if (L < 32 && !now) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) l[i] = -INFINITY;
      }
      in = base + STRIDE < hi && fetch(base + STRIDE);
      if (L == 32 && !now) continue;  // the whole warp
      const float r = weights<SIGMOID, false, L, EPL>(l, none);
      if (L == 32 || now) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) acc[i] = fmaf(l[i], r, acc[i]);
      }
    }
    // tokens of the warp, then warps w and w + 8, then warps 0 .. 7
#pragma unroll
    for (int i = 0; i < EPL; ++i)
#pragma unroll
      for (int o = L; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    auto at = [&](int i) { return 4 * (sub + L * (i / 4)) + i % 4; };
    if (warp >= kHalf && lane < L)
#pragma unroll
      for (int i = 0; i < EPL; ++i) part[warp - kHalf][at(i)] = acc[i];
    __syncthreads();
    if (warp < kHalf && lane < L)
#pragma unroll
      for (int i = 0; i < EPL; ++i) part[warp][at(i)] += acc[i];
    __syncthreads();
    const int64_t entry = (int64_t)blockIdx.x + s;
    float dot = 0.f;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
      float sum = part[0][e];
#pragma unroll
      for (int w = 1; w < kHalf; ++w) sum += part[w][e];
      if (SINGLE) {
        dot += finish_expert(a, s, e, sum, hist[e], n_seq_tokens);
      } else {
        a.psum[entry * a.E + e] = sum;
        a.pcnt[entry * a.E + e] = hist[e];
      }
    }
    if (SINGLE) {
      dot = block_sum<kWarps>(dot, red);
      if (threadIdx.x == 0) finish_loss(a, s, dot, n_seq_tokens);
    } else if (threadIdx.x == 0) {
      a.pn[entry] = n_seq_tokens;
    }
    __syncthreads();
  }
}

// The results of one sequence from its blocks' sums: `ranks` blocks a sequence (a cluster), each with `per` of the
// experts; a block's threads are experts times groups of entries. More blocks only where a sequence has many
// entries (one of 65536 tokens has 304). The kernel is launched beside the first one's end and waits for its
// results here.
constexpr int kFinishThreads = 1024;
__global__ void __launch_bounds__(kFinishThreads) finish_kernel(const Args a, int ranks, int per) {
  __shared__ float sums[kFinishThreads];
  __shared__ int cnts[kFinishThreads];
  __shared__ float red[32];
  __shared__ float dot_part;
  __shared__ int n_tokens;
  const int s = blockIdx.x / ranks, rank = blockIdx.x - s * ranks;
  const int begin = seq_begin(a.offsets, s, a.S, a.T), end = seq_begin(a.offsets, s + 1, a.S, a.T);
  const int f = begin / a.per_block, l = end > begin ? (end - 1) / a.per_block : f - 1;  // first, last block
  const int groups = kFinishThreads / per, group = threadIdx.x / per;
  const int e = rank * per + threadIdx.x % per;
  if (threadIdx.x == 0) n_tokens = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float sum = 0.f;
  int cnt = 0, n = 0;
  if (e < a.E) {
#pragma unroll 4
    for (int b = f + group; b <= l; b += groups) {
      sum += a.psum[((int64_t)b + s) * a.E + e];
      cnt += a.pcnt[((int64_t)b + s) * a.E + e];
    }
  }
  for (int b = f + threadIdx.x; b <= l; b += kFinishThreads) n += a.pn[b + s];
  sums[threadIdx.x] = sum;
  cnts[threadIdx.x] = cnt;
  __syncthreads();
  if (n) atomicAdd(&n_tokens, n);
  __syncthreads();
  float dot = 0.f;
  if (group == 0 && e < a.E) {
    for (int g = 1; g < groups; ++g) {
      sum += sums[g * per + threadIdx.x];
      cnt += cnts[g * per + threadIdx.x];
    }
    dot = finish_expert(a, s, e, sum, cnt, n_tokens);
  }
  dot = block_sum<32>(dot, red);
  if (ranks == 1) {
    if (threadIdx.x == 0) finish_loss(a, s, dot, n_tokens);
    return;
  }
  if (threadIdx.x == 0) dot_part = dot;
  cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    float total = 0.f;
    for (int r = 0; r < ranks; ++r) total += ld_cluster(mapa_shared(smem_u32(&dot_part), (uint32_t)r));
    finish_loss(a, s, total, n_tokens);
  }
  cluster_sync();  // no block leaves while its part is read
}

struct BackArgs {
  const void* logits;
  const int32_t* offsets;
  const uint8_t* mask;
  const int32_t* counts;
  const int32_t* tokens;
  const float* dloss;
  void* dlogits;
  int T, E, S, per_block;
  float scale;  // alpha * E / k
};

template <bool SIGMOID, bool BF16, int L, int EPL>
__global__ void __launch_bounds__(kThreads, EPL > 8 ? 1 : 2) backward_kernel(const BackArgs a) {
  constexpr int PER_WARP = 32 / L;
  constexpr int STRIDE = kWarps * PER_WARP;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % L;
  const int b0 = blockIdx.x * a.per_block, b1 = min(a.T, b0 + a.per_block);
  const bool vec = (a.E & 3) == 0;
  float g[EPL];
  Row<BF16, L, EPL> cur;
  int until = -1;  // g is that of the sequence of the tokens before this one
  bool covered = false;
  auto fetch = [&](int base) {
    const int t = base + lane / L;
    const bool in = t < b1 && (!a.mask || a.mask[t]);
    if (in) cur.load(a.logits, t, a.E, sub);
    return in;
  };
  int base = b0 + warp * PER_WARP;
  bool in = base < b1 && fetch(base);
  for (; base < b1; base += STRIDE) {
    const int t = base + lane / L;
    if (t < b1 && t >= until) {
      const int s = seq_of(a.offsets, a.S, a.T, t);
      const int begin = seq_begin(a.offsets, s, a.S, a.T), end = seq_begin(a.offsets, s + 1, a.S, a.T);
      covered = t >= begin && t < end;
      until = t < begin ? begin : t < end ? end : a.T;
      const float n = (float)max(a.tokens[s], 1);
      const float c = __fdiv_rn(__fdiv_rn(a.scale * a.dloss[s], n), n);
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = 4 * (sub + L * (i / 4)) + i % 4;
        g[i] = e < a.E ? c * (float)a.counts[(int64_t)s * a.E + e] : 0.f;
      }
    }
    float l[EPL], d[SIGMOID ? EPL : 1];
    const bool now = in;
    cur.values(l);
    in = base + STRIDE < b1 && fetch(base + STRIDE);
    const bool zero = !now || !covered;  // padding, or a token of no sequence: whatever its logits hold
    if (L < 32 || !zero) {               // with L = 32 the whole warp has one token
      const float r = weights<SIGMOID, SIGMOID, L, EPL>(l, d);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        l[i] *= r;
        dot = fmaf(l[i], g[i], dot);
      }
      dot = lanes_sum<L>(dot);
#pragma unroll
      for (int i = 0; i < EPL; ++i) l[i] *= SIGMOID ? (g[i] - dot) * d[SIGMOID ? i : 0] : g[i] - dot;
    }
    if (zero) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) l[i] = 0.f;
    }
    if (t >= b1) continue;
#pragma unroll
    for (int j = 0; j < EPL / 4; ++j) {
      const int e = 4 * (sub + L * j);
      const float* o = l + 4 * j;
      const int64_t at = (int64_t)t * a.E + e;
      if (vec && e < a.E) {
        if (BF16)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dlogits) + at) =
              make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(a.dlogits) + at) = make_float4(o[0], o[1], o[2], o[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (e + i >= a.E) break;
          if (BF16)
            static_cast<__nv_bfloat16*>(a.dlogits)[at + i] = __float2bfloat16_rn(o[i]);
          else
            static_cast<float*>(a.dlogits)[at + i] = o[i];
        }
      }
    }
  }
}

// Lanes of a token for E experts, and the shapes that are compiled: (L, EPL) with L * EPL >= E.
int lanes_of(int E) { return E <= 4 ? 1 : E <= 8 ? 2 : E <= 16 ? 4 : E <= 32 ? 8 : E <= 64 ? 16 : 32; }

template <class F>
cudaError_t with_shape(int E, F&& f) {
  using std::integral_constant;
  if (E <= 4) return f(integral_constant<int, 1>{}, integral_constant<int, 4>{});
  if (E <= 8) return f(integral_constant<int, 2>{}, integral_constant<int, 4>{});
  if (E <= 16) return f(integral_constant<int, 4>{}, integral_constant<int, 4>{});
  if (E <= 32) return f(integral_constant<int, 8>{}, integral_constant<int, 4>{});
  if (E <= 64) return f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  if (E <= 128) return f(integral_constant<int, 32>{}, integral_constant<int, 4>{});
  if (E <= 256) return f(integral_constant<int, 32>{}, integral_constant<int, 8>{});
  if (E <= 512) return f(integral_constant<int, 32>{}, integral_constant<int, 16>{});
  return f(integral_constant<int, 32>{}, integral_constant<int, 32>{});
}

// Tokens of a block: at least four rounds of its warps (fewer where the sequences are short: a block works on one
// after the other, about 3 us each), at most what fills the SMs with two blocks each.
int tokens_per_block(int T, int E, int S) {
  const int64_t least = std::min<int64_t>(4 * kWarps * (32 / lanes_of(E)), std::max<int64_t>(1, cdiv(4 * (int64_t)T, S)));
  return (int)std::max<int64_t>(least, cdiv(T, 2 * kNumSMsHint));
}

}  // namespace bl

int64_t balance_loss_entries(int T, int E, int S) { return cdiv(T, bl::tokens_per_block(T, E, S)) + S; }

cudaError_t launch_balance_loss(const BalanceLossDesc& d, int* launches, cudaStream_t stream) {
  bl::Args a;
  a.logits = d.logits;
  a.topk_idx = d.topk_idx;
  a.offsets = d.offsets;
  a.mask = d.mask;
  a.T = d.T;
  a.E = d.E;
  a.k = d.k;
  a.S = d.S;
  a.per_block = bl::tokens_per_block(d.T, d.E, d.S);
  a.alpha = d.alpha;
  const int64_t entries = balance_loss_entries(d.T, d.E, d.S);
  a.psum = static_cast<float*>(d.scratch);
  a.pcnt = reinterpret_cast<int32_t*>(a.psum + entries * d.E);
  a.pn = a.pcnt + entries * d.E;
  a.loss = d.loss;
  a.counts = d.counts;
  a.mean = d.mean;
  a.tokens = d.tokens;
  const bool single = d.T <= a.per_block && d.S <= 4;  // one block, one sequence after the other
  const unsigned blocks = single ? 1u : (unsigned)cdiv(d.T, a.per_block);
  cudaError_t e = bl::with_shape(d.E, [&](auto Lc, auto Ec) {
    constexpr int L = decltype(Lc)::value, EPL = decltype(Ec)::value;
    auto go = [&](auto kernel) {
      kernel<<<blocks, bl::kThreads, 0, stream>>>(a);
      return cudaGetLastError();
    };
    if (d.sigmoid)
      return d.bf16 ? (single ? go(bl::forward_kernel<true, true, L, EPL, true>)
                              : go(bl::forward_kernel<true, true, L, EPL, false>))
                    : (single ? go(bl::forward_kernel<true, false, L, EPL, true>)
                              : go(bl::forward_kernel<true, false, L, EPL, false>));
    return d.bf16 ? (single ? go(bl::forward_kernel<false, true, L, EPL, true>)
                            : go(bl::forward_kernel<false, true, L, EPL, false>))
                  : (single ? go(bl::forward_kernel<false, false, L, EPL, true>)
                            : go(bl::forward_kernel<false, false, L, EPL, false>));
  });
  *launches = 1;
  if (e != cudaSuccess || single) return e;
  int wide = 32;  // experts rounded up to a power of two, and those of a block
  while (wide < d.E) wide *= 2;
  const int64_t each = cdiv(blocks, d.S) + 1;  // entries of a sequence
  int ranks = 1;
  while (ranks < 8 && wide / ranks > 32 && each > 8 * (bl::kFinishThreads / (wide / ranks))) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)d.S * (unsigned)ranks);
  cfg.blockDim = dim3(bl::kFinishThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 2 : 1;
  *launches = 2;
  return cudaLaunchKernelEx(&cfg, bl::finish_kernel, a, ranks, wide / ranks);
}

cudaError_t launch_balance_loss_backward(const BalanceLossBackwardDesc& d, cudaStream_t stream) {
  bl::BackArgs a;
  a.logits = d.logits;
  a.offsets = d.offsets;
  a.mask = d.mask;
  a.counts = d.counts;
  a.tokens = d.tokens;
  a.dloss = d.dloss;
  a.dlogits = d.dlogits;
  a.T = d.T;
  a.E = d.E;
  a.S = d.S;
  a.scale = d.alpha * (float)d.E / (float)d.k;
  const int round = bl::kWarps * (32 / bl::lanes_of(d.E));
  a.per_block = (int)std::max<int64_t>(round, cdiv(cdiv(d.T, 2 * num_sms()), round) * round);
  const unsigned blocks = (unsigned)cdiv(d.T, a.per_block);
  return bl::with_shape(d.E, [&](auto Lc, auto Ec) {
    constexpr int L = decltype(Lc)::value, EPL = decltype(Ec)::value;
    auto go = [&](auto kernel) {
      kernel<<<blocks, bl::kThreads, 0, stream>>>(a);
      return cudaGetLastError();
    };
    if (d.sigmoid)
      return d.bf16 ? go(bl::backward_kernel<true, true, L, EPL>) : go(bl::backward_kernel<true, false, L, EPL>);
    return d.bf16 ? go(bl::backward_kernel<false, true, L, EPL>) : go(bl::backward_kernel<false, false, L, EPL>);
  });
}

}  // namespace moe
