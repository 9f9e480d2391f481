// MoE router for gfx950: expert ids and weights of every token from its
// logits, and the gradient of the weights.
//
//   p = softmax(l) or 1 / (1 + exp(-l)),  z = p + bias,
//   (groups: score = sum of a group's two largest z, the best topk_groups stay)
//   ids = the topk largest z, ties to the lowest index,
//   w_j = scale p_j, or scale p_j / sum_i p_i.
//
// One wavefront per token, lane l holding the E consecutive experts from l E
// on (E = 1, 2, 4, 8, 16: up to 1024 experts), so that the lowest lane of a
// tie has the lowest index. Scores are float64: whether an expert is chosen is
// a comparison of two nearly equal numbers, and its answer should be that of
// the formula, not of the rounding.
#include "common.hpp"
#include <type_traits>

#include "wave.hpp"

namespace fp8q {

constexpr int kRouteWaves = 4;  // tokens per workgroup

struct RouteArgs {
  const void* logits;
  const float* bias;
  int T, G, topk, n_groups, topk_groups;
  int sigmoid, renorm;
  float scale;
  int32_t* ids;
  float* w;
};

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// 64-bit key ordered like the double; 0 (below every finite value's key) marks
// an expert that may not be chosen.
__device__ __forceinline__ uint64_t order_key(double z) {
  if (!(z > -__builtin_huge_val())) return 0;
  const uint64_t u = (uint64_t)__double_as_longlong(z + 0.0);  // -0 counts as +0
  return (u >> 63) ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ double key_value(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? k & ~(1ull << 63) : ~k));
}

// Largest key of the wavefront and its lowest lane; 0 when there is none. The
// upper halves are compared first; only if several lanes share the largest
// (wave-uniform, rare) are the lower halves.
__device__ __forceinline__ uint64_t wave_best(uint64_t k, int& lane) {
  const uint32_t hi = (uint32_t)(k >> 32), lo = (uint32_t)k;
  const uint32_t mhi = wave_max_u32(hi);
  uint64_t at = __ballot(hi == mhi);
  if (__popcll(at) > 1) {
    const uint32_t mlo = wave_max_u32(hi == mhi ? lo : 0u);
    at = __ballot(hi == mhi && lo == mlo);
  }
  lane = __builtin_ctzll(at);
  return ((uint64_t)mhi << 32) | lane_u32(lo, lane);
}

// Probability of expert l E + i for a lane's E logits; masked ones have 0.
template <int E>
__device__ __forceinline__ void route_scores(const float (&x)[E], bool sigmoid, double (&p)[E]) {
  constexpr float kNegInf = -__builtin_huge_valf();
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < E; ++i) p[i] = x[i] > kNegInf ? 1.0 / (1.0 + exp(-(double)x[i])) : 0.0;
    return;
  }
  // order the floats as integers: the maximum over the wavefront is exact
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const uint32_t u = __float_as_uint(x[i]);
    if (x[i] > kNegInf) m = max(m, (u >> 31) ? ~u : u | 0x80000000u);
  }
  m = wave_max_u32(m);
  const double top = m ? (double)__uint_as_float((m >> 31) ? m & 0x7FFFFFFFu : ~m) : 0.0;
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    p[i] = x[i] > kNegInf ? exp((double)x[i] - top) : 0.0;
    sum += p[i];
  }
  sum = wave_sum_f64(sum);
#pragma unroll
  for (int i = 0; i < E; ++i) p[i] = sum > 0.0 ? p[i] / sum : 0.0;
}

template <int E, typename Tin>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs a) {
  __shared__ uint64_t group_keys[kRouteWaves][64 * E];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * kRouteWaves + wave;
  if (t >= a.T) return;
  const Tin* row = (const Tin*)a.logits + (int64_t)t * a.G;
  float x[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int e = lane * E + i;
    x[i] = e < a.G ? load_logit(row + e) : -__builtin_huge_valf();
  }
  double p[E];
  route_scores<E>(x, a.sigmoid, p);
  uint64_t key[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int e = lane * E + i;
    const double z = (a.bias && e < a.G) ? p[i] + (double)a.bias[e] : p[i];
    key[i] = x[i] > -__builtin_huge_valf() ? order_key(z) : 0;
  }

  if (a.n_groups > 1) {
    // a group's two largest keys, found by the lane of its number
    uint64_t* k = group_keys[wave];
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (lane * E + i < a.G) k[lane * E + i] = key[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int gs = a.G / a.n_groups;
    uint64_t g1 = 0, g2 = 0;
    if (lane < a.n_groups) {
      for (int i = 0; i < gs; ++i) {
        const uint64_t v = k[lane * gs + i];
        g2 = max(g2, min(g1, v));
        g1 = max(g1, v);
      }
    }
    const double gz = g1 ? key_value(g1) + (g2 ? key_value(g2) : 0.0) : -__builtin_huge_val();
    uint64_t gk = order_key(gz);
    uint64_t open = 0;  // bit g: group g may be used (wave-uniform)
    for (int j = 0; j < a.topk_groups; ++j) {
      int at;
      if (!wave_best(gk, at)) break;
      open |= 1ull << at;
      if (lane == at) gk = 0;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int e = lane * E + i;
      if (e < a.G && !((open >> (e / gs)) & 1)) key[i] = 0;
    }
  }

  int my_id = -1;     // lane j: choice j
  double my_p = 0.0;
  for (int j = 0; j < a.topk; ++j) {
    uint64_t bk = key[0];
    int bi = 0;
    double bp = p[0];
#pragma unroll
    for (int i = 1; i < E; ++i)
      if (key[i] > bk) bk = key[i], bi = i, bp = p[i];
    int at;
    if (!wave_best(bk, at)) break;  // nothing left to choose
    const int id = at * E + __builtin_amdgcn_readlane(bi, at);
    const double pj = lane_f64(bp, at);
    if (lane == j) my_id = id, my_p = pj;
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (lane == at && i == bi) key[i] = 0;
  }
  double w = my_p;
  if (a.renorm) {
    const double sum = wave_sum_f64(my_p);
    w = sum > 0.0 ? my_p / sum : 0.0;
  }
  if (lane < a.topk) {
    a.ids[(int64_t)t * a.topk + lane] = my_id;
    a.w[(int64_t)t * a.topk + lane] = (float)((double)a.scale * w);
  }
}

// Gradient. Lane j < topk holds choice j. With q_j the renormalized
// probability and g_j = scale dweights_j:
//   softmax, renorm   dl_e = sum_{j: id_j = e} q_j (g_j - sum_i g_i q_i), since
//                     the weights are the softmax over the chosen logits alone
//   softmax           dl_e = p_e (sum_{j: id_j = e} g_j - sum_j g_j p_j)
//   sigmoid           dl_e = sum_{j: id_j = e} dp_j p_j (1 - p_j), dp_j = g_j or
//                     (g_j - sum_i g_i q_i) / sum_i p_i
// so only the plain softmax needs every probability of the row.
struct RouteBwdArgs {
  const void* logits;
  const int32_t* ids;
  const float* dw;
  int T, G, topk;
  int sigmoid, renorm;
  float scale;
  void* dlogits;
};

__device__ __forceinline__ void store_logit(float* p, double v) { *p = (float)v; }
__device__ __forceinline__ void store_logit(uint16_t* p, double v) {
  const __bf16 b = (__bf16)(float)v;
  *p = __builtin_bit_cast(uint16_t, b);
}

template <int E, typename Tin>
__global__ __launch_bounds__(64 * kRouteWaves) void route_bwd_kernel(RouteBwdArgs a) {
  constexpr float kNegInf = -__builtin_huge_valf();
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * kRouteWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= a.T) return;
  const Tin* row = (const Tin*)a.logits + (int64_t)t * a.G;
  Tin* drow = (Tin*)a.dlogits + (int64_t)t * a.G;
  int id = -1;
  double g = 0.0;
  if (lane < a.topk) {
    id = a.ids[(int64_t)t * a.topk + lane];
    g = (double)a.scale * (double)a.dw[(int64_t)t * a.topk + lane];
  }
  const bool on = id >= 0 && id < a.G;
  if (!on) id = -1, g = 0.0;
  const float xj = on ? load_logit(row + id) : kNegInf;
  const bool dense = !a.sigmoid && !a.renorm;

  double v;  // this choice's share of dl[id]
  double p[E];
  double mean = 0.0;
  if (dense) {
    // lane l holds the experts l + 64 i here: dlogits are stored in rows of 64
    float x[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int e = i * 64 + lane;
      x[i] = e < a.G ? load_logit(row + e) : kNegInf;
    }
    route_scores<E>(x, false, p);
    v = g;
  } else if (a.sigmoid) {
    const bool live = xj > kNegInf;
    const double pj = live ? 1.0 / (1.0 + exp(-(double)xj)) : 0.0;
    const double rest = live ? 1.0 / (1.0 + exp((double)xj)) : 0.0;  // 1 - pj, without cancellation
    double dp = g;
    if (a.renorm) {
      const double sum = wave_sum_f64(pj);
      const double gp = wave_sum_f64(g * pj);
      dp = (on && sum > 0.0) ? (g - gp / sum) / sum : 0.0;
    }
    v = dp * pj * rest;
  } else {
    const float one[1] = {xj};
    double q[1];
    route_scores<1>(one, false, q);
    const double gq = wave_sum_f64(g * q[0]);
    v = on ? q[0] * (g - gq) : 0.0;
  }

  double d[E];
#pragma unroll
  for (int i = 0; i < E; ++i) d[i] = 0.0;
  for (int j = 0; j < a.topk; ++j) {
    const int ej = __builtin_amdgcn_readlane(id, j);
    const double vj = lane_f64(v, j);
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (ej == i * 64 + lane) d[i] += vj;
  }
  if (dense) {
#pragma unroll
    for (int i = 0; i < E; ++i) mean += d[i] * p[i];
    mean = wave_sum_f64(mean);
#pragma unroll
    for (int i = 0; i < E; ++i) d[i] = p[i] * (d[i] - mean);
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (i * 64 + lane < a.G) store_logit(drow + i * 64 + lane, d[i]);
}

template <typename Args, typename Launch>
static void by_experts(const Args& a, Launch&& launch) {
  if (a.G <= 64) launch(std::integral_constant<int, 1>{});
  else if (a.G <= 128) launch(std::integral_constant<int, 2>{});
  else if (a.G <= 256) launch(std::integral_constant<int, 4>{});
  else if (a.G <= 512) launch(std::integral_constant<int, 8>{});
  else launch(std::integral_constant<int, 16>{});
}

hipError_t launch_route(const void* logits, bool bf16, const float* bias, int64_t T, int64_t G,
                        int64_t topk, int64_t n_groups, int64_t topk_groups, bool sigmoid,
                        bool renorm, float scale, int32_t* ids, float* w, hipStream_t stream) {
  const RouteArgs a{logits, bias, (int)T, (int)G, (int)topk, (int)n_groups, (int)topk_groups,
                    sigmoid, renorm, scale, ids, w};
  const dim3 grid((unsigned)((T + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
  by_experts(a, [&](auto e) {
    constexpr int E = decltype(e)::value;
    if (bf16)
      hipLaunchKernelGGL((route_kernel<E, uint16_t>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((route_kernel<E, float>), grid, block, 0, stream, a);
  });
  return hipGetLastError();
}

hipError_t launch_route_bwd(const void* logits, bool bf16, const int32_t* ids, const float* dw,
                            int64_t T, int64_t G, int64_t topk, bool sigmoid, bool renorm,
                            float scale, void* dlogits, hipStream_t stream) {
  const RouteBwdArgs a{logits, ids, dw, (int)T, (int)G, (int)topk, sigmoid, renorm, scale, dlogits};
  const dim3 grid((unsigned)((T + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
  by_experts(a, [&](auto e) {
    constexpr int E = decltype(e)::value;
    if (bf16)
      hipLaunchKernelGGL((route_bwd_kernel<E, uint16_t>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((route_bwd_kernel<E, float>), grid, block, 0, stream, a);
  });
  return hipGetLastError();
}

}  // namespace fp8q
