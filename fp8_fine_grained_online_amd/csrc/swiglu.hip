// The gated activation between an MLP's two products, to rows of bfloat16 or
// binary32 or straight to 1x128 FP8 tiles, and its gradient, for gfx950.
//
//   gu = [gate | up] (M x 2I),  s = 1 / (1 + exp(-gate)),  y = gate s up
//   dgate = dy up s (1 + gate (1 - s)),  dup = dy gate s
//
// A chunk of eight values per thread, and nothing kept in between: every value is read
// once and written once. Memory bounds them (MI355X: gradient of 16384 x 2048 51 us, 6.6
// TB/s; FP8 form of 65536 x 2048 in 32 experts' blocks 118 us, 5.9 TB/s), the FP8 form
// nearly as much as the vector ALU: with 42 operations a value, a transcendental one
// counted as four, it took 142 us, so its arithmetic is the least that keeps the
// accuracy. Two, four or eight chunks per thread were 0 to 30% slower, workgroups that
// stay and walk along the rows 3 to 10%.
//
// With t = exp(-gate) the pair s, 1 - s is {1, t} / (1 + t). t is kept within
// e^-87 .. e^87, so that none of it over- or underflows. Gates below -87, which ordinary
// data does not have, put their wavefront on a way of its own with a factor exp(gate + 87).
#include <type_traits>

#include "common.hpp"
#include "rows.hpp"

namespace fp8q {

constexpr int kSwigluThreads = 256;

constexpr float kFar = 87.0f;  // beyond, a sigmoid or what it lacks to 1 is below 2^-125

struct Gate {
  float s, c, y;  // sigmoid, 1 - sigmoid, gate sigmoid
  float f;        // s and y are to be multiplied by it, last
};

// t = exp(-x), |x| <= 87, to about two units in the last place: 2^p by the hardware's
// instruction for a p next to -x log2(e), and the exponential's first-order term of the
// difference. A bfloat16 x times the 16 leading bits of log2(e) is exact, which leaves x
// times the others (their square is below 2^-23 of t); for any x the rounded product is
// taken, and what it lacks found with a fused multiply-add.
constexpr double kLog2e = 1.44269504088896340736, kLn2 = 0.69314718055994530942;
template <typename X>
__device__ __forceinline__ float exp_neg(float x) {
  float p, rest;
  if constexpr (sizeof(X) == 2) {
    constexpr float kLead = 47274.0f / 32768.0f;
    p = x * -kLead;
    rest = x * (float)((kLead - kLog2e) * kLn2);
  } else {
    constexpr float kHi = (float)kLog2e;
    p = x * -kHi;
    rest = __builtin_fmaf(__builtin_fmaf(x, -kHi, -p), (float)kLn2, x * (float)(((double)kHi - kLog2e) * kLn2));
  }
  const float e = __builtin_amdgcn_exp2f(p);
  return __builtin_fmaf(e, rest, e);
}

// The reciprocal is the hardware's, to one unit: a correction would be two operations
// of the FP8 form's budget. kBelow: some gate of the wavefront may be below -87. Such a one
// counts as -87 in the sigmoid, and f is what its exponential lacks: none of the others'
// factors is subnormal, so the products lose nothing before the last. (From -200 on f is 0; the
// maximum is the one that keeps a NaN.)
template <typename X, bool kBelow>
__device__ __forceinline__ Gate gate_of(float g) {
  const float low = kBelow ? __builtin_elementwise_maximum(g, -kFar) : g;
  const float t = exp_neg<X>(fminf(low, kFar));
  const float s = __builtin_amdgcn_rcpf(1.0f + t);
  if constexpr (!kBelow) return {s, t * s, g * s, 1.0f};
  const float v = __builtin_elementwise_maximum(g, -200.0f);
  return {s, t * s, v * s, v < -kFar ? exp_neg<float>(-kFar - v) : 1.0f};
}

// f(false), or f(true) where some gate of the wavefront is below -87: as bits, negative values order behind
// all others, the farther from zero the later
template <typename F>
__device__ __forceinline__ void for_gates(const float (&g)[8], F&& f) {
  uint32_t most = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) most = umax(most, __float_as_uint(g[e]));
  if (__any(most > 0xC2AE0000u)) f(std::true_type{});  // -87
  else f(std::false_type{});
}

// u becomes gate sigmoid(gate) u
template <typename X>
__device__ __forceinline__ void activate(const float (&g)[8], float (&u)[8]) {
  for_gates(g, [&](auto below) {
    constexpr bool kBelow = decltype(below)::value;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const Gate k = gate_of<X, kBelow>(g[e]);
      u[e] *= k.y;
      if (kBelow) u[e] *= k.f;
    }
  });
}

// n / d for n below 2^31, by a multiplication: m = floor(2^k / d) + 1 for the k = 31 +
// ceil(log2 d) that makes it exact
struct Division {
  uint32_t m, k;
  explicit Division(uint32_t d) {
    k = 31;
    while ((uint64_t(1) << (k - 31)) < d) ++k;
    m = (uint32_t)((uint64_t(1) << k) / d + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (uint32_t)((uint64_t)n * m >> k); }
};

struct SwigluArgs {
  const void *gu, *dy;
  void* out;  // rows of y, codes, or of dgu
  float* sa;
  const int32_t* last;  // m_offsets + G: the rows that exist, or NULL for all
  int64_t ld, ldy;
  int M, I;
  bool nt;  // more is read than stays cached
  Division chunks;  // by the chunks of a row
};

// This thread's row and chunk of the I columns; false past the last row. Chunks
// are numbered along the rows, kSwigluThreads of them per workgroup: less than 2^31.
__device__ __forceinline__ bool my_chunk(const SwigluArgs& p, int64_t& m, int& c) {
  const uint32_t n = blockIdx.x * kSwigluThreads + threadIdx.x;
  const uint32_t row = p.chunks(n);
  m = (int64_t)row;
  c = (int)(n - row * ((uint32_t)(p.I + 7) / 8));
  return (int)row < (p.last ? min(max(*p.last, 0), p.M) : p.M);
}

template <typename X, typename Y>
__global__ __launch_bounds__(kSwigluThreads) void swiglu_kernel(SwigluArgs p) {
  int64_t m;
  int c;
  if (!my_chunk(p, m, c)) return;
  const int at = 8 * c, have = min(p.I - at, 8);
  const X* const row = (const X*)p.gu + m * p.ld + at;
  Chunk<X> rg, ru;
  if (p.nt) rg = load_chunk<true>(row, have), ru = load_chunk<true>(row + p.I, have);
  else rg = load_chunk(row, have), ru = load_chunk(row + p.I, have);
  float g[8], u[8];
  values(rg, g);
  values(ru, u);
  activate<X>(g, u);
  Chunk<Y> out;
  to_chunk(u, out);
  store_chunk((Y*)p.out + m * (int64_t)p.I + at, out, have);
}

// I is a multiple of 128: a tile is 16 chunks, the 16 lanes of a DPP row
template <typename X>
__global__ __launch_bounds__(kSwigluThreads) void swiglu_quant_kernel(SwigluArgs p) {
  int64_t m;
  int c;
  if (!my_chunk(p, m, c)) return;  // whole tiles
  const X* const row = (const X*)p.gu + m * p.ld + 8 * c;
  Chunk<X> rg, ru;
  if (p.nt) rg = load_whole<true>(row), ru = load_whole<true>(row + p.I);
  else rg = load_whole(row), ru = load_whole(row + p.I);
  float g[8], u[8];
  values(rg, g);
  values(ru, u);
  activate<X>(g, u);
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(u[e]));
  const float amax = __uint_as_float(row16_max_u32(__float_as_uint(top)));
  float s;
  uint2 codes;
  // (as bits, which order like the values: 2^-64 to the largest finite one)
  if (__any(__float_as_uint(amax) - 0x1F800000u >= 0x7F800000u - 0x1F800000u)) {
    // tiles of nothing, or of so little that quotients have to be scaled and may pass 448; and those with a
    // product that overflowed, whose codes then do not depend on the tiles beside them
    s = tile_scale(amax);
    const TileDivisor d = make_divisor(s, amax);
    codes.x = pack4_e4m3(quotient(u[0], d), quotient(u[1], d), quotient(u[2], d), quotient(u[3], d));
    codes.y = pack4_e4m3(quotient(u[4], d), quotient(u[5], d), quotient(u[6], d), quotient(u[7], d));
  } else {
    // the same without what such tiles need: |u| <= amax, so a quotient rounds to at most 448
    s = tile_scale(amax);
    const float r = recip_rn(s);
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float q0 = u[e] * r;
      q[e] = __builtin_fmaf(__builtin_fmaf(-q0, s, u[e]), r, q0);
      q[e] = __uint_as_float((__float_as_uint(q[e]) & 0x7FFFFFFFu) | (__float_as_uint(u[e]) & 0x80000000u));
    }
    codes.x = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false), true);
    codes.y = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false), true);
  }
  *(uint2*)((uint8_t*)p.out + m * (int64_t)p.I + 8 * c) = codes;
  if ((c & 15) == 0) p.sa[m * (int64_t)(p.I / kGroup) + c / 16] = s;
}

template <typename X, typename D>
__global__ __launch_bounds__(kSwigluThreads) void swiglu_bwd_kernel(SwigluArgs p) {
  int64_t m;
  int c;
  if (!my_chunk(p, m, c)) return;
  const int at = 8 * c, have = min(p.I - at, 8);
  const X* const row = (const X*)p.gu + m * p.ld + at;
  const D* const dy = (const D*)p.dy + m * p.ldy + at;
  Chunk<X> rg, ru;
  Chunk<D> rd;
  if (p.nt) rg = load_chunk<true>(row, have), ru = load_chunk<true>(row + p.I, have), rd = load_chunk<true>(dy, have);
  else rg = load_chunk(row, have), ru = load_chunk(row + p.I, have), rd = load_chunk(dy, have);
  float g[8], u[8], d[8];
  values(rg, g);
  values(ru, u);
  values(rd, d);
  for_gates(g, [&](auto below) {
    constexpr bool kBelow = decltype(below)::value;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const Gate k = gate_of<X, kBelow>(g[e]);
      // s (1 + gate (1 - s)) = s + (gate s) (1 - s); above 87 it is 1, whatever the gate
      const float slope = g[e] > kFar ? k.s : __builtin_fmaf(k.y, k.c, k.s);
      // (where d u overflows both are above 1, and the slope, never subnormal, is taken to one of them first)
      const float du = d[e] * u[e], f = kBelow ? k.f : 1.0f;
      g[e] = fabsf(du) <= 3.402823466e38f ? du * slope * f : (d[e] * slope) * (u[e] * f);
      u[e] = d[e] * k.y * f;
    }
  });
  X* const out = (X*)p.out + m * (int64_t)(2 * p.I) + at;
  Chunk<X> o;
  to_chunk(g, o);
  store_chunk(out, o, have);
  to_chunk(u, o);
  store_chunk(out + p.I, o, have);
}

// Reads that pass the caches by from 96 MiB on, which neither leaves nor finds them
// there whole: gradient of 16384 x 2048 58.8 -> 56.2 us, activation of 67584 x 2048
// 139.9 -> 135.5; but of 4096 x 1024 8.4 -> 9.1.
static bool beyond_cache(int64_t bytes) { return bytes > (int64_t(96) << 20); }

static dim3 chunk_grid(const SwigluArgs& a) {
  const int64_t chunks = (int64_t)a.M * ((a.I + 7) / 8);
  return dim3((unsigned)((chunks + kSwigluThreads - 1) / kSwigluThreads));
}

hipError_t launch_swiglu(const void* gu, bool gu_bf16, int64_t ld, const int32_t* last, int64_t M, int64_t I, void* y,
                         bool y_bf16, hipStream_t stream) {
  const SwigluArgs a{gu, nullptr, y, nullptr, last, ld, 0, (int)M, (int)I, beyond_cache(M * I * (gu_bf16 ? 4 : 8)), Division((uint32_t)(I + 7) / 8)};
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, chunk_grid(a), dim3(kSwigluThreads), 0, stream, a); };
  if (gu_bf16) y_bf16 ? go(swiglu_kernel<bf16_t, bf16_t>) : go(swiglu_kernel<bf16_t, float>);
  else y_bf16 ? go(swiglu_kernel<float, bf16_t>) : go(swiglu_kernel<float, float>);
  return hipGetLastError();
}

hipError_t launch_swiglu_quant(const void* gu, bool gu_bf16, int64_t ld, const int32_t* last, int64_t M, int64_t I,
                               uint8_t* q, float* sa, hipStream_t stream) {
  const SwigluArgs a{gu, nullptr, q, sa, last, ld, 0, (int)M, (int)I, beyond_cache(M * I * (gu_bf16 ? 4 : 8)), Division((uint32_t)(I + 7) / 8)};
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, chunk_grid(a), dim3(kSwigluThreads), 0, stream, a); };
  gu_bf16 ? go(swiglu_quant_kernel<bf16_t>) : go(swiglu_quant_kernel<float>);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const void* dy, bool dy_bf16, int64_t ldy, const void* gu, bool gu_bf16, int64_t ld,
                             const int32_t* last, int64_t M, int64_t I, void* dgu, hipStream_t stream) {
  const SwigluArgs a{gu, dy, dgu, nullptr, last, ld, ldy, (int)M, (int)I,
                     beyond_cache(M * I * ((gu_bf16 ? 4 : 8) + (dy_bf16 ? 2 : 4))), Division((uint32_t)(I + 7) / 8)};
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, chunk_grid(a), dim3(kSwigluThreads), 0, stream, a); };
  if (gu_bf16) dy_bf16 ? go(swiglu_bwd_kernel<bf16_t, bf16_t>) : go(swiglu_bwd_kernel<bf16_t, float>);
  else dy_bf16 ? go(swiglu_bwd_kernel<float, bf16_t>) : go(swiglu_bwd_kernel<float, float>);
  return hipGetLastError();
}

}  // namespace fp8q
