// Gradient of the route weights with respect to the router's logits.
//
// With l the logits of a token, e_j its chosen experts, c the routed scale and g_j the gradient of weight j:
//   softmax           w_j = c p_{e_j}, p = softmax of all logits:   dl_e = c p_e (G_e - sum_j g_j p_{e_j})
//   softmax, renorm.  w_j = c u_j, u = softmax of the chosen ones:  dl_{e_j} = c u_j (g_j - sum_i g_i u_i)
//   sigmoid           w_j = c s_j, s = sigmoid(l_{e_j}):            dl_{e_j} = c s_j (1 - s_j) g_j
//   sigmoid, renorm.  w_j = c u_j, u_j = s_j / sum_i s_i:           dl_{e_j} = c u_j (1 - s_j) (g_j - sum_i g_i u_i)
// G_e adds the g_j of the slots that chose e (an expert chosen twice gets both); 0 where nothing is said. The selection
// and its bias carry no gradient. Slots whose index lies outside [0, E) are left out.
//
// fp32. Sigmoids are taken with e^min(l) factored out of their sum, so that a token whose sigmoids all underflow keeps
// their ratios; a token whose chosen logits are all -inf has no weights and a gradient of 0.
//
// One GB300: 65536 tokens x 256 experts, k 8, fp32: chosen experts alone 20.6 us. Its bytes, dlogits and the 8 logits a
// token, are 11 us at a copy's rate, but the logits come in pieces of 64 bytes: 46 MB are read and 67 written, 17 us.
// Softmax over all 24.6 us (5.5 TB/s of 6.78), bf16 23.9: latency, a token's loads and sums in a row. 4096 x 8: 2.4 us,
// launch. Four tokens a warp instead of one for the chosen experts: 33 -> 20 us; all loads of a token asked for together:
// 30 -> 24.6 us (softmax).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace moe {
namespace rb {

constexpr int kThreads = 256;
constexpr int kMaxE = 1024;
constexpr float kLog2e = 1.4426950408889634f;

// 2 ulp. A probability e^(l - m) is taken as 2^(log2(e) (l - m)): the product's rounding is |x| 2^-24 of an exponent x,
// that is below 2e-6 of a probability of 1e-8, and less of larger ones.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float exponential(float x) { return ex2(x * kLog2e); }

struct Args {
  const void* logits;
  const int32_t* idx;
  const float* dw;
  void* dlogits;
  int64_t T;
  int E, k, renorm;
  float scale;
};

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// One slot of a token: its expert (-1: none) and the gradient of its weight (asked for together), then its logit.
__device__ __forceinline__ void ask_slot(const Args& a, int64_t t, int j, int& e, float& g) {
  const bool in = t < a.T && j < a.k;
  e = in ? a.idx[t * a.k + j] : -1;
  g = in ? a.dw[t * a.k + j] : 0.f;
}
template <int TYPE>
__device__ __forceinline__ float slot_logit(const Args& a, int64_t t, int& e, float& g) {
  if (e >= 0 && e < a.E) return rows::value<TYPE>(rows::load_bits<TYPE>(a.logits, t * a.E + e));
  e = -1;
  g = 0.f;
  return -INFINITY;
}

// The gradients of the slots that chose this lane's expert, and how many they are: an expert chosen twice gets both,
// and each of its slots writes the same sum.
template <int L>
__device__ __forceinline__ void same_expert(int k, int e, float g, float& all, float& n) {
  all = g;
  n = 1.f;
  const uint32_t peers = __match_any_sync(0xffffffffu, e < 0 ? -1 : e + (int)((threadIdx.x & 31) / L) * kMaxE);
  if (!__any_sync(0xffffffffu, e >= 0 && __popc(peers) > 1)) return;
  all = n = 0.f;
  for (int j = 0; j < k; ++j) {
    const int ej = __shfl_sync(0xffffffffu, e, j, L);
    const float gj = __shfl_sync(0xffffffffu, g, j, L);
    if (ej == e) {
      all += gj;
      n += 1.f;
    }
  }
}

// Weights of the chosen experts alone: L lanes a token (k rounded up to a power of two), lane j slot j. The rows of a
// warp's tokens lie one after the other and are zeroed as one; the slots then write over that, behind a barrier of the
// warp.
template <int TYPE, bool SIGMOID, int L>
__global__ void __launch_bounds__(kThreads) chosen_kernel(const Args a) {
  constexpr int kPer = 32 / L;  // tokens of a warp
  const int lane = threadIdx.x & 31, sub = lane % L;
  const int64_t warps = ((int64_t)gridDim.x * kThreads) >> 5;
  const int64_t bytes = (int64_t)kPer * a.E * rows::kSize<TYPE>;  // of a warp's rows
  for (int64_t t0 = (((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5) * kPer; t0 < a.T; t0 += warps * kPer) {
    const int64_t t = t0 + lane / L;
    int e;
    float g;
    ask_slot(a, t, sub, e, g);
    char* out = static_cast<char*>(a.dlogits) + t0 * a.E * rows::kSize<TYPE>;
    if ((bytes & 15) == 0 && t0 + kPer <= a.T) {
      for (int64_t b = 16 * lane; b < bytes; b += 512) *reinterpret_cast<uint4*>(out + b) = make_uint4(0u, 0u, 0u, 0u);
    } else {
      const int64_t n = min((int64_t)kPer, a.T - t0) * a.E;
      for (int64_t i = lane; i < n; i += 32) rows::store_bits<TYPE>(out, i, 0u);
    }
    const float l = slot_logit<TYPE>(a, t, e, g);
    float u, slope = 1.f, all, n;
    if (!SIGMOID) {
      float m = lanes_max<L>(l);
      if (m == -INFINITY) m = 0.f;
      u = exponential(l - m);
    } else {
      // sigmoid(l) e^-c = 1 / (e^c + e^(c - l)) with c = min(max l, 0)
      float c = 0.f;
      if (a.renorm) {
        const float m = lanes_max<L>(l);
        c = m == -INFINITY ? 0.f : fminf(m, 0.f);
      }
      u = e < 0 ? 0.f : __fdividef(1.0f, exponential(c) + exponential(c - l));
      slope = __fdividef(1.0f, 1.0f + exponential(l));
    }
    same_expert<L>(a.k, e, g, all, n);
    if (a.renorm) {  // a softmax over the chosen, or sigmoids divided by their sum
      const float z = lanes_sum<L>(u);
      u = z == 0.f ? 0.f : __fdiv_rn(u, z);
      all -= n * lanes_sum<L>(g * u);
    }
    __syncwarp();
    if (e >= 0) rows::store_bits<TYPE>(a.dlogits, t * a.E + e, rows::bits_of<TYPE>(a.scale * u * slope * all));
  }
}

// A softmax over all experts: L lanes a token, at least k, a lane the experts 4 (sub + L j) + i, EPL of them; all of
// them write the dense part -c p sum_j g_j p_{e_j}, then lane j slot j over that.
template <int TYPE, int L, int EPL>
__global__ void __launch_bounds__(kThreads) dense_kernel(const Args a) {
  constexpr int kPer = 32 / L;  // tokens of a warp
  const int lane = threadIdx.x & 31, sub = lane % L;
  const int64_t warps = ((int64_t)gridDim.x * kThreads) >> 5;
  const bool vec = (a.E & 3) == 0;
  for (int64_t t0 = (((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5) * kPer; t0 < a.T; t0 += warps * kPer) {
    const int64_t t = t0 + lane / L;
    const bool in = t < a.T;
    int e;
    float g, p[EPL], m = -INFINITY;
    ask_slot(a, t, sub, e, g);
#pragma unroll
    for (int j = 0; j < EPL / 4; ++j) {
      const int at = 4 * (sub + L * j);
      if (vec && in && at < a.E) {
        if constexpr (TYPE == MOE_TYPE_F32) {
          const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + t * a.E + at);
          p[4 * j] = v.x, p[4 * j + 1] = v.y, p[4 * j + 2] = v.z, p[4 * j + 3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + t * a.E + at);
          p[4 * j] = bf16_lo(v.x), p[4 * j + 1] = bf16_hi(v.x), p[4 * j + 2] = bf16_lo(v.y), p[4 * j + 3] = bf16_hi(v.y);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          p[4 * j + i] = in && at + i < a.E ? rows::value<TYPE>(rows::load_bits<TYPE>(a.logits, t * a.E + at + i)) : -INFINITY;
      }
    }
    const float l = slot_logit<TYPE>(a, t, e, g);
#pragma unroll
    for (int j = 0; j < EPL; ++j) m = fmaxf(m, p[j]);
    m = lanes_max<L>(m);
    if (m == -INFINITY) m = 0.f;
    float z = 0.f, all, n;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      p[j] = exponential(p[j] - m);
      z += p[j];
    }
    z = lanes_sum<L>(z);
    const float r = z == 0.f ? 0.f : __fdiv_rn(1.0f, z);
    const float u = exponential(l - m) * r;
    // a token without choices, padding say, has no gradient whatever its logits hold
    const uint32_t own = L == 32 ? 0xffffffffu : ((1u << (L & 31)) - 1u) << (lane - sub);
    const bool none = (__ballot_sync(0xffffffffu, e >= 0) & own) == 0u;
    const float dot = lanes_sum<L>(g * u);
    same_expert<L>(a.k, e, g, all, n);
    if (in) {
      const float by = -a.scale * r * dot;
#pragma unroll
      for (int j = 0; j < EPL / 4; ++j) {
        const int at = 4 * (sub + L * j);
        float o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = none ? 0.f : by * p[4 * j + i];
        if (vec && at < a.E) {
          if (TYPE == MOE_TYPE_F32)
            *reinterpret_cast<float4*>(static_cast<float*>(a.dlogits) + t * a.E + at) = make_float4(o[0], o[1], o[2], o[3]);
          else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dlogits) + t * a.E + at) =
                make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (at + i < a.E) rows::store_bits<TYPE>(a.dlogits, t * a.E + at + i, rows::bits_of<TYPE>(o[i]));
        }
      }
    }
    __syncwarp();
    if (e >= 0) rows::store_bits<TYPE>(a.dlogits, t * a.E + e, rows::bits_of<TYPE>(a.scale * u * (all - dot)));
  }
}

template <class F>
cudaError_t with_shape(int E, int k, F&& f) {
  using std::integral_constant;
  const int need = std::max(k, (E + 3) / 4);
  if (need <= 2) return f(integral_constant<int, 2>{}, integral_constant<int, 4>{});
  if (need <= 4) return f(integral_constant<int, 4>{}, integral_constant<int, 4>{});
  if (need <= 8) return f(integral_constant<int, 8>{}, integral_constant<int, 4>{});
  if (need <= 16) return f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  if (need <= 32) return f(integral_constant<int, 32>{}, integral_constant<int, 4>{});
  if (E <= 256) return f(integral_constant<int, 32>{}, integral_constant<int, 8>{});
  if (E <= 512) return f(integral_constant<int, 32>{}, integral_constant<int, 16>{});
  return f(integral_constant<int, 32>{}, integral_constant<int, 32>{});
}

}  // namespace rb

cudaError_t launch_route_backward(const RouteBackwardDesc& d, cudaStream_t stream) {
  rb::Args a;
  a.logits = d.logits;
  a.idx = d.topk_idx;
  a.dw = d.dtopk_w;
  a.dlogits = d.dlogits;
  a.T = d.T;
  a.E = d.E;
  a.k = d.k;
  a.renorm = d.renorm;
  a.scale = d.routed_scale;
  auto go = [&](auto kernel, int per_warp) {
    const int64_t blocks = std::min<int64_t>(cdiv(d.T, (rb::kThreads / 32) * per_warp), (int64_t)num_sms() * 64);
    kernel<<<(unsigned)blocks, rb::kThreads, 0, stream>>>(a);
    return cudaGetLastError();
  };
  auto typed = [&](auto T) {
    constexpr int kT = decltype(T)::value;
    if (!d.sigmoid && !d.renorm)
      return rb::with_shape(d.E, d.k, [&](auto Lc, auto Ec) {
        constexpr int L = decltype(Lc)::value;
        return go(rb::dense_kernel<kT, L, decltype(Ec)::value>, 32 / L);
      });
    auto chosen = [&](auto Lc) {
      constexpr int L = decltype(Lc)::value;
      return d.sigmoid ? go(rb::chosen_kernel<kT, true, L>, 32 / L) : go(rb::chosen_kernel<kT, false, L>, 32 / L);
    };
    using std::integral_constant;
    if (d.k <= 2) return chosen(integral_constant<int, 2>{});
    if (d.k <= 4) return chosen(integral_constant<int, 4>{});
    if (d.k <= 8) return chosen(integral_constant<int, 8>{});
    if (d.k <= 16) return chosen(integral_constant<int, 16>{});
    return chosen(integral_constant<int, 32>{});
  };
  return d.bf16 ? typed(std::integral_constant<int, MOE_TYPE_BF16>{}) : typed(std::integral_constant<int, MOE_TYPE_F32>{});
}

}  // namespace moe
