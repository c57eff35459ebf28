// Gradient of the route weights with respect to the router's logits.
//
// With l the logits of a token, e_j its chosen experts, c the routed scale and g_j the gradient of weight j:
//   softmax           w_j = c p_{e_j}, p = softmax of all logits:   dl_e = c p_e (G_e - sum_j g_j p_{e_j})
//   softmax, renorm.  w_j = c u_j, u = softmax of the chosen ones:  dl_{e_j} = c u_j (g_j - sum_i g_i u_i)
//   sigmoid           w_j = c s_j, s = sigmoid(l_{e_j}):            dl_{e_j} = c s_j (1 - s_j) g_j
//   sigmoid, renorm.  w_j = c u_j, u_j = s_j / sum_i s_i:           dl_{e_j} = c u_j (1 - s_j) (g_j - sum_i g_i u_i)
// G_e adds the g_j of the slots that chose e (an expert chosen twice gets both); 0 where nothing is said. The selection and
// its bias carry no gradient. Slots whose index lies outside [0, E) are left out.
//
// fp32. Sigmoids are taken with e^min(l) factored out of their sum, so that a token whose sigmoids all underflow keeps their
// ratios; a token whose chosen logits are all -inf has no weights and a gradient of 0.
//
// A token is held by L lanes, at least k of them: lane j works on slot j, and all of them write the row, zeros or the dense
// part first and the chosen experts' numbers over it (the group's lanes in order: a barrier of the warp lies between). Bound by the
// bytes of dlogits (and of the logits, for a softmax over all).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace moe {
namespace rb {

constexpr int kThreads = 256;

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

// EPL: numbers of a lane, 4 (sub + L j) + i
template <int TYPE, bool SIGMOID, bool DENSE, int L, int EPL>
__global__ void __launch_bounds__(kThreads) kernel(const Args a) {
  constexpr int kPer = 32 / L;  // tokens of a warp
  const int lane = threadIdx.x & 31, sub = lane % L;
  const int64_t warps = ((int64_t)gridDim.x * kThreads) >> 5;
  const bool vec = (a.E & 3) == 0;
  for (int64_t t0 = (((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5) * kPer; t0 < a.T; t0 += warps * kPer) {
    const int64_t t = t0 + lane / L;
    const bool in = t < a.T;
    int e = -1;
    float g = 0.f, l = -INFINITY;
    if (in && sub < a.k) {
      e = a.idx[t * a.k + sub];
      g = a.dw[t * a.k + sub];
      if (e < 0 || e >= a.E) {
        e = -1;
        g = 0.f;
      } else {
        l = rows::value<TYPE>(rows::load_bits<TYPE>(a.logits, t * a.E + e));
      }
    }
    float p[DENSE ? EPL : 1], m = -INFINITY, u, slope = 1.f;
    if (DENSE) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const int at = 4 * (sub + L * (j / 4)) + j % 4;
        p[j] = in && at < a.E ? rows::value<TYPE>(rows::load_bits<TYPE>(a.logits, t * a.E + at)) : -INFINITY;
        m = fmaxf(m, p[j]);
      }
      m = lanes_max<L>(m);
      if (m == -INFINITY) m = 0.f;
      float z = 0.f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        p[j] = expf(p[j] - m);
        z += p[j];
      }
      z = lanes_sum<L>(z);
      const float r = z == 0.f ? 0.f : __fdiv_rn(1.0f, z);
#pragma unroll
      for (int j = 0; j < EPL; ++j) p[j] *= r;
      u = expf(l - m) * r;
    } else if (!SIGMOID) {
      m = lanes_max<L>(l);
      if (m == -INFINITY) m = 0.f;
      u = expf(l - m);
      const float z = lanes_sum<L>(u);
      u = z == 0.f ? 0.f : __fdiv_rn(u, z);
    } else {
      // sigmoid(l) e^-c = 1 / (e^c + e^(c - l)) with c = min(max l, 0)
      float c = 0.f;
      if (a.renorm) {
        m = lanes_max<L>(l);
        c = m == -INFINITY ? 0.f : fminf(m, 0.f);
      }
      u = __fdiv_rn(1.0f, expf(c) + expf(c - l));
      if (e < 0) u = 0.f;
      slope = __fdiv_rn(1.0f, 1.0f + expf(l));
      if (a.renorm) {
        const float z = lanes_sum<L>(u);
        u = z == 0.f ? 0.f : __fdiv_rn(u, z);
      }
    }
    const bool centred = DENSE || !SIGMOID || a.renorm;
    const float dot = centred ? lanes_sum<L>(e >= 0 ? g * u : 0.f) : 0.f;
    // an expert chosen twice: every slot of it writes the same sum
    float all = 0.f, n = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const int ej = __shfl_sync(0xffffffffu, e, j, L);
      const float gj = __shfl_sync(0xffffffffu, g, j, L);
      if (ej == e) {
        all += gj;
        n += 1.f;
      }
    }
    if (DENSE) n = 1.f;
    const float d = a.scale * u * slope * (all - n * dot);
    if (in) {
#pragma unroll
      for (int j = 0; j < EPL / 4; ++j) {
        const int at = 4 * (sub + L * j);
        float o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = DENSE ? -a.scale * p[DENSE ? 4 * j + i : 0] * dot : 0.f;
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
    if (e >= 0) rows::store_bits<TYPE>(a.dlogits, t * a.E + e, rows::bits_of<TYPE>(d));
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
  const bool dense = !d.sigmoid && !d.renorm;
  return rb::with_shape(d.E, d.k, [&](auto Lc, auto Ec) {
    constexpr int L = decltype(Lc)::value, EPL = decltype(Ec)::value;
    const int64_t blocks = std::min<int64_t>(cdiv(d.T, (rb::kThreads / 32) * (32 / L)), (int64_t)num_sms() * 8);
    auto go = [&](auto kernel) {
      kernel<<<(unsigned)blocks, rb::kThreads, 0, stream>>>(a);
      return cudaGetLastError();
    };
    auto typed = [&](auto T) {
      constexpr int kT = decltype(T)::value;
      if (d.sigmoid) return go(rb::kernel<kT, true, false, L, EPL>);
      return dense ? go(rb::kernel<kT, false, true, L, EPL>) : go(rb::kernel<kT, false, false, L, EPL>);
    };
    return d.bf16 ? typed(std::integral_constant<int, MOE_TYPE_BF16>{}) : typed(std::integral_constant<int, MOE_TYPE_F32>{});
  });
}

}  // namespace moe
