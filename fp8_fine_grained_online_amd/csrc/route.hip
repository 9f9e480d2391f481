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
// tie has the lowest index. A lane sorts its keys once; each choice is then one
// maximum over the wavefront, and the winner's next key moves up. Scores are
// float64: whether an expert is chosen is a comparison of two nearly equal
// numbers, and its answer should be that of the formula, not of the rounding.
//
// Few bytes move (at most 17 MB below, 3.5 us): what the time goes into are
// instructions. For few tokens it is one wavefront's chain (a load, the scores in
// float64, its choices, 0.15 us each) on top of a launch (1.8 us for an empty
// kernel); for batches the vector ALUs are busy 70 to 80% of the time. MI355X, us,
// in a captured graph: 16 tokens of 256 experts in 8 groups, top-8, sigmoid 5.7;
// 8192 of 64, top-6 6.0; 8192 of 256 in 8 groups 14.1; 4096 of 512, top-10 10.2;
// 100 of 1024, top-64 21.2 (41.6 with the places of a lane's experts moved up one by
// one); gradient, 8192 of 256, sigmoid 5.4, softmax 7.6. (With every choice searched
// through all keys, the library's exponential, and gradient shares passed from lane
// to lane the first took 8.8 and the gradient 8.3.)
#include <type_traits>

#include "common.hpp"
#include "wave.hpp"

namespace fp8q {

constexpr int kRouteWaves = 4;  // tokens per workgroup

struct RouteArgs {
  const void* logits;
  const float* bias;
  int T, G, topk, n_groups, topk_groups;
  int gs;  // experts of a group
  int sigmoid, renorm;
  int whole;  // a lane's experts are all in the row or all past it, and aligned
  float scale;
  int32_t* ids;
  float* w;
};

__device__ __forceinline__ float as_logit(float v) { return v; }
__device__ __forceinline__ float as_logit(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// The E consecutive logits from `at` on; masked (-inf) past the row's G. With
// `whole` (uniform) every lane's E are inside or outside the row, and aligned.
template <int E, typename Tin>
__device__ __forceinline__ void load_logits(const Tin* row, int at, int G, bool whole, float (&x)[E]) {
  typedef Tin vec __attribute__((ext_vector_type(E > 1 ? E : 2), aligned(E * sizeof(Tin) < 16 ? E * sizeof(Tin) : 16)));
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = -__builtin_huge_valf();
  if (E > 1 && whole) {
    if (at < G) {
      const vec v = *(const vec*)(row + at);
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = as_logit((Tin)v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (at + i < G) x[i] = as_logit(row[at + i]);
  }
}

// e^x for x <= 710 to about one unit in the last place: x = k ln 2 + r with ln 2
// in two parts, the Taylor series of e^r to r^13 (|r| <= 0.347: the next term is
// below 5e-18), and the power of two put back.
__device__ __forceinline__ double exp64(double x) {
  x = __builtin_fmax(x, -746.0);  // e^-746 rounds to 0
  const double k = __builtin_rint(x * 0x1.71547652b82fep+0);
  double r = __builtin_fma(k, -0x1.62e42fefa3p-1, x);  // the first 41 bits of ln 2: exact
  r = __builtin_fma(k, -0x1.3de6af278ece6p-42, r);     // and the next 53
  constexpr double c[14] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040, 1.0 / 40320,
                            1.0 / 362880, 1.0 / 3628800, 1.0 / 39916800, 1.0 / 479001600, 1.0 / 6227020800};
  double s = c[13];
#pragma unroll
  for (int i = 12; i >= 0; --i) s = __builtin_fma(s, r, c[i]);
  return __builtin_ldexp(s, (int)k);
}

// 1 / d for 1 <= d < 2^1023: two Newton steps from the hardware's estimate
__device__ __forceinline__ double recip64(double d) {
  double r = __builtin_amdgcn_rcp(d);
  r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
  return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}

__device__ __forceinline__ double sigmoid64(float x) {
  // e^709 + 1 still has a reciprocal; before that, 1 + e^x is 1 in float64
  const bool far = x < -700.0f;
  const double e = exp64(far ? (double)x : -(double)x);
  return far ? e : recip64(1.0 + e);
}

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

// The lane of the wavefront's largest key, the lowest if several have it. The
// upper halves are compared first; only if several lanes share the largest
// (wave-uniform, rare) are the lower halves. Returns the upper half: 0 when every
// key is 0 (a finite value's is not).
__device__ __forceinline__ uint32_t wave_best(uint64_t k, int& lane) {
  const uint32_t hi = (uint32_t)(k >> 32), lo = (uint32_t)k;
  const uint32_t mhi = wave_max_u32(hi);
  uint64_t at = __ballot(hi == mhi);
  if (at & (at - 1)) {
    const uint32_t mlo = wave_max_u32(hi == mhi ? lo : 0u);
    at = __ballot(hi == mhi && lo == mlo);
  }
  lane = __builtin_ctzll(at);
  return mhi;
}

// A lane's E keys, largest first, with their places in the lane; equal keys by
// place (Batcher's odd-even merging network).
template <int E>
__device__ __forceinline__ void sort_lane(uint64_t (&k)[E], int (&at)[E]) {
#pragma unroll
  for (int p = 1; p < E; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < E; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i) {
          const int u = i + j, v = i + j + q;
          if (v < E && u / (2 * p) == v / (2 * p)) {
            const bool swap = k[v] > k[u] || (k[v] == k[u] && at[v] < at[u]);
            const uint64_t ku = k[u];
            const int au = at[u];
            k[u] = swap ? k[v] : ku, at[u] = swap ? at[v] : au;
            k[v] = swap ? ku : k[v], at[v] = swap ? au : at[v];
          }
        }
}

// The two largest of the pairs (k0 >= k1) of neighbouring lanes, folded over
// runs of `lanes` (a power of two); every lane of a run gets the result.
__device__ __forceinline__ void merge_two(uint64_t& k0, uint64_t& k1, uint64_t o0, uint64_t o1) {
  const uint64_t low = min(k0, o0);
  k0 = max(k0, o0);
  k1 = max(low, max(k1, o1));
}
template <int kCtrl>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v) {
  return ((uint64_t)dpp_u32<kCtrl>((uint32_t)(v >> 32)) << 32) | dpp_u32<kCtrl>((uint32_t)v);
}
__device__ __forceinline__ void fold_two(uint64_t& k0, uint64_t& k1, int lanes) {
  if (lanes >= 2) merge_two(k0, k1, dpp_u64<0xB1>(k0), dpp_u64<0xB1>(k1));
  if (lanes >= 4) merge_two(k0, k1, dpp_u64<0x4E>(k0), dpp_u64<0x4E>(k1));
  if (lanes >= 8) merge_two(k0, k1, dpp_u64<0x141>(k0), dpp_u64<0x141>(k1));
  if (lanes >= 16) merge_two(k0, k1, dpp_u64<0x140>(k0), dpp_u64<0x140>(k1));
  for (int d = 16; d < lanes; d *= 2) {
    const uint64_t o0 = __shfl_xor((unsigned long long)k0, d), o1 = __shfl_xor((unsigned long long)k1, d);
    merge_two(k0, k1, o0, o1);
  }
}

// The wavefront's largest logit (0 when all are masked): the floats are ordered
// as integers, so the maximum is exact.
template <int E>
__device__ __forceinline__ double wave_top(const float (&x)[E]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const uint32_t u = __float_as_uint(x[i]);
    if (x[i] > -__builtin_huge_valf()) m = max(m, (u >> 31) ? ~u : u | 0x80000000u);
  }
  m = wave_max_u32(m);
  return m ? (double)__uint_as_float((m >> 31) ? m & 0x7FFFFFFFu : ~m) : 0.0;
}

// Renormalized weights are ratios p_j / sum_i p_i of the chosen. Probabilities below
// this have lost bits to underflow, or are about to; their ratios are formed from
// shifted_score instead.
constexpr double kSmallScore = 0x1p-960;

// The chosen logits' probabilities, one per lane (masked: 0), without a factor that
// all share: e^top / sum of the softmax; e^top of sigmoids where the largest chosen
// logit, top, is negative.
__device__ __forceinline__ double shifted_score(float x, bool sigmoid) {
  const float one[1] = {x};
  const double top = wave_top<1>(one), v = (double)x;
  double s = exp64(sigmoid ? __builtin_fmin(v, 0.0) - __builtin_fmin(top, 0.0) : v - top);
  if (sigmoid) s *= recip64(1.0 + exp64(-__builtin_fabs(v)));
  return x > -__builtin_huge_valf() ? s : 0.0;
}

// Numerators of the softmax (all over `sum`), or sigmoids; masked logits have 0.
template <int E>
__device__ __forceinline__ double softmax_terms(const float (&x)[E], double (&p)[E]) {
  constexpr float kNegInf = -__builtin_huge_valf();
  const double top = wave_top<E>(x);
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    p[i] = x[i] > kNegInf ? exp64((double)x[i] - top) : 0.0;
    sum += p[i];
  }
  return wave_sum_f64(sum);
}

template <int E, typename Tin>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs a) {
  // scores by expert: the probabilities of the chosen are looked up at the end,
  // and group scores that do not fall on whole lanes are formed here
  __shared__ uint64_t table[kRouteWaves][64 * E];
  __shared__ int chosen[kRouteWaves][64];  // ids of the choices
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * kRouteWaves + wave;
  if (t >= a.T) return;
  uint64_t* const tab = table[wave];
  float x[E];
  load_logits<E>((const Tin*)a.logits + (int64_t)t * a.G, lane * E, a.G, a.whole, x);
  float bias[E];  // loaded with the logits: later it would be a second wait for memory
#pragma unroll
  for (int i = 0; i < E; ++i) bias[i] = a.bias && lane * E + i < a.G ? a.bias[lane * E + i] : 0.0f;
  double p[E];
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < E; ++i) p[i] = x[i] > -__builtin_huge_valf() ? sigmoid64(x[i]) : 0.0;
  } else {
    const double sum = softmax_terms<E>(x, p);
    const double inv = sum > 0.0 ? recip64(sum) : 0.0;  // 1 <= sum <= G; no logit but masked ones: 0
#pragma unroll
    for (int i = 0; i < E; ++i) p[i] *= inv;
  }
  uint64_t key[E];
  int place[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const double z = p[i] + (double)bias[i];
    key[i] = x[i] > -__builtin_huge_valf() ? order_key(z) : 0;
    place[i] = i;
  }

  const int gs = a.gs;
  const int lanes = gs / E;  // of a group, if groups fall on whole lanes
  const bool by_lanes = gs % E == 0 && (lanes & (lanes - 1)) == 0;
  if (a.n_groups > 1 && !by_lanes) {
    // the two largest keys of group g, by lane g; experts of closed groups lose theirs
#pragma unroll
    for (int i = 0; i < E; ++i) tab[lane * E + i] = key[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    uint64_t g1 = 0, g2 = 0;
    if (lane < a.n_groups) {
      for (int i = 0; i < gs; ++i) {
        const uint64_t v = tab[lane * gs + i];
        g2 = max(g2, min(g1, v));
        g1 = max(g1, v);
      }
    }
    uint64_t gk = g1 ? order_key(key_value(g1) + (g2 ? key_value(g2) : 0.0)) : 0;
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
    __builtin_amdgcn_wave_barrier();
  }
  sort_lane<E>(key, place);
  if (a.n_groups > 1 && by_lanes) {
    uint64_t g1 = key[0], g2 = E > 1 ? key[E > 1 ? 1 : 0] : 0;
    fold_two(g1, g2, lanes);
    uint64_t gk = g1 ? order_key(key_value(g1) + (g2 ? key_value(g2) : 0.0)) : 0;
    bool open = false;
    for (int j = 0; j < a.topk_groups; ++j) {
      int at;
      if (!wave_best(gk, at)) break;
      if ((lane & -lanes) == (at & -lanes)) open = true, gk = 0;  // the winner's run of lanes
    }
#pragma unroll
    for (int i = 0; i < E; ++i) key[i] = open ? key[i] : 0;
  }

#pragma unroll
  for (int i = 0; i < E; ++i) tab[lane * E + i] = (uint64_t)__double_as_longlong(p[i]);
  typedef std::conditional_t<(E > 8), uint64_t, uint32_t> Places;  // 4 bits each, the first lowest
  Places places = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) places |= (Places)place[i] << (4 * i);
  int* const ids = chosen[wave];
  ids[lane] = -1;
  for (int j = 0; j < a.topk; ++j) {
    int at;
    if (!wave_best(key[0], at)) break;  // nothing left to choose
    if (lane == at) {
      // the winner notes its expert, and its next key moves up
      ids[j] = lane * E + (int)(places & 15);
#pragma unroll
      for (int i = 0; i + 1 < E; ++i) key[i] = key[i + 1];
      key[E - 1] = 0;
      places >>= 4;
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const int my_id = ids[lane];  // lane j: choice j
  double w = my_id >= 0 ? __longlong_as_double((long long)tab[my_id]) : 0.0;
  if (a.renorm) {
    if (__ballot(my_id >= 0 && w < kSmallScore))  // rare: the logits are read again
      w = shifted_score(my_id >= 0 ? as_logit(((const Tin*)a.logits)[(int64_t)t * a.G + my_id]) : -__builtin_huge_valf(),
                        a.sigmoid);
    const double sum = wave_sum_f64(w);
    w = sum > 0.0 ? w / sum : 0.0;
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
//   sigmoid, renorm   dl_e = sum_{j: id_j = e} q_j (g_j - sum_i g_i q_i) (1 - p_j)
//   sigmoid           dl_e = sum_{j: id_j = e} g_j p_j (1 - p_j)
// so only the plain softmax needs every probability of the row.
//
// The row is put together in LDS: zeros, then the choices' shares at their
// experts. Should an expert be listed twice, which shows when a lane does not
// read back the number it wrote there, the shares are added one by one.
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
  // By way of binary32, whose own rounding shows only if it lands in the middle
  // between two bfloat16 numbers (one value in 2^16): then v tells the side.
  uint32_t u = __float_as_uint((float)v);
  if ((u & 0xFFFF) == 0x8000) {
    const double mid = __builtin_fabs((double)__uint_as_float(u));
    if (mid < __builtin_fabs(v)) u += 1;
    else if (mid > __builtin_fabs(v)) u -= 1;
  }
  const __bf16 b = (__bf16)__uint_as_float(u);
  *p = __builtin_bit_cast(uint16_t, b);
}

template <int E, typename Tin>
__global__ __launch_bounds__(64 * kRouteWaves) void route_bwd_kernel(RouteBwdArgs a) {
  constexpr float kNegInf = -__builtin_huge_valf();
  __shared__ double shares[kRouteWaves][64 * E];
  __shared__ int owners[kRouteWaves][64 * E];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * kRouteWaves + wave;
  if (t >= a.T) return;
  double* const share = shares[wave];
  int* const owner = owners[wave];
  const Tin* row = (const Tin*)a.logits + (int64_t)t * a.G;
  Tin* drow = (Tin*)a.dlogits + (int64_t)t * a.G;
  const bool dense = !a.sigmoid && !a.renorm;
  float x[E];  // lane l holds the experts l + 64 i: dlogits are stored in runs of 64
  if (dense) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int e = i * 64 + lane;
      x[i] = e < a.G ? as_logit(row[e]) : kNegInf;
    }
  }
  int id = -1;
  double g = 0.0;
  if (lane < a.topk) {
    id = a.ids[(int64_t)t * a.topk + lane];
    g = (double)a.scale * (double)a.dw[(int64_t)t * a.topk + lane];
  }
  const bool on = id >= 0 && id < a.G;
  if (!on) id = -1, g = 0.0;
  const float xj = on ? as_logit(row[id]) : kNegInf;
  if (on) owner[id] = lane;
#pragma unroll
  for (int i = 0; i < E; ++i) share[i * 64 + lane] = 0.0;

  double v = g;  // this choice's share of dl[id]; of the dense form, of dp[id]
  if (a.sigmoid) {
    const bool live = xj > kNegInf;
    // p and 1 - p, the smaller one without cancellation
    const double ex = live ? exp64(-__builtin_fabs((double)xj)) : 0.0;
    const double big = recip64(1.0 + ex), small = ex * big;
    const double pj = !live ? 0.0 : xj >= 0.0f ? big : small;
    const double rest = !live ? 0.0 : xj >= 0.0f ? small : big;
    if (a.renorm) {
      // q and q (g - sum g q) are ordinary numbers; 1 / sum may not be one
      const double part = __ballot(live && pj < kSmallScore) ? shifted_score(xj, true) : pj;
      const double sum = wave_sum_f64(part);
      const double q = sum > 0.0 ? part / sum : 0.0;
      const double gq = wave_sum_f64(g * q);
      v = q * (g - gq) * rest;
    } else {
      v *= pj * rest;
    }
  } else if (!dense) {
    const float one[1] = {xj};
    double q[1];
    const double sum = softmax_terms<1>(one, q);
    q[0] = sum > 0.0 ? q[0] / sum : 0.0;
    const double gq = wave_sum_f64(g * q[0]);
    v = on ? q[0] * (g - gq) : 0.0;
  }

  // (the wave's LDS accesses are in order; the fence keeps the compiler to it)
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const bool alone = !on || owner[id] == lane;
  if (__ballot(!alone) == 0) {
    if (on) share[id] = v;
  } else {
    for (int j = 0; j < a.topk; ++j) {  // wave-uniform; in order
      if (lane == j && on) share[id] += v;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  double d[E];
#pragma unroll
  for (int i = 0; i < E; ++i) d[i] = share[i * 64 + lane];
  if (dense) {
    double p[E], mean = 0.0;
    const double sum = softmax_terms<E>(x, p);
    const double inv = sum > 0.0 ? recip64(sum) : 0.0;
#pragma unroll
    for (int i = 0; i < E; ++i) p[i] *= inv, mean += d[i] * p[i];
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
  RouteArgs a{logits, bias, (int)T, (int)G, (int)topk, (int)n_groups, (int)topk_groups,
              (int)(G / n_groups), sigmoid, renorm, 0, scale, ids, w};
  const dim3 grid((unsigned)((T + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
  by_experts(a, [&](auto e) {
    constexpr int E = decltype(e)::value;
    const int bytes = E * (bf16 ? 2 : 4);
    a.whole = G % E == 0 && (uintptr_t)logits % (bytes < 16 ? bytes : 16) == 0 && G % (bytes < 16 ? E : 16 / (bf16 ? 2 : 4)) == 0;
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
