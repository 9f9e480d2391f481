// The gated activation between an MLP's two products, to rows of bfloat16 or
// binary32 or straight to 1x128 FP8 tiles, and its gradient, for gfx950.
//
//   gu = [gate | up] (M x 2I),  s = 1 / (1 + exp(-gate)),  y = gate s up
//   dgate = dy up s (1 + gate (1 - s)),  dup = dy gate s
//
// All three are bound by memory: every value is read once and written once, eight
// per thread and row part, and nothing is kept in between. With t = exp(-|gate|)
// the pair s, 1 - s is {1, t} / (1 + t), in that order or the other: no overflow
// at either end, and no cancellation in 1 - s.
#include "common.hpp"
#include "rows.hpp"

namespace fp8q {

constexpr int kSwigluThreads = 256;

// exp(-a) for a >= 0, to about two units in the last place: a log2(e) as a
// rounded product and what it lacks, the power of two of the first by the
// hardware's instruction, and the rest as the exponential's first-order term.
__device__ __forceinline__ float exp_neg(float a) {
  constexpr float kLog2e = 1.44269504088896340736f;                      // RN(log2 e)
  constexpr float kRest = (float)(1.44269504088896340736 - (double)kLog2e);
  constexpr float kLn2 = 0.69314718055994530942f;
  const float p = a * kLog2e;
  const float rest = __builtin_fmaf(a, kRest, __builtin_fmaf(a, kLog2e, -p));
  const float e = __builtin_amdgcn_exp2f(-p);
  // past the smallest normal number nothing is left worth correcting (and for an
  // infinite a there is no rest)
  return a < 87.0f ? __builtin_fmaf(-e, rest * kLn2, e) : a == a ? 0.0f : a;
}

struct Gate {
  float s, c;  // sigmoid and 1 - sigmoid
};
__device__ __forceinline__ Gate sigmoid(float g) {
  const float t = exp_neg(fabsf(g));
  const float r = recip_rn(1.0f + t);  // 1 + t in [1, 2]
  const float q = t * r;
  return g >= 0.0f ? Gate{r, q} : Gate{q, r};
}

// gate sigmoid(gate); 0 for a gate of -infinity
__device__ __forceinline__ float silu(float g, float s) { return g < -1e38f ? -0.0f : g * s; }

struct SwigluArgs {
  const void *gu, *dy;
  void* out;  // rows of y, codes, or of dgu
  float* sa;
  const int32_t* last;  // m_offsets + G: the rows that exist, or NULL for all
  int64_t ld, ldy;
  int M, I;
};

// This thread's row and chunk of the I columns; false past the last row. Chunks
// are numbered along the rows, kSwigluThreads of them per workgroup.
__device__ __forceinline__ bool my_chunk(const SwigluArgs& p, int64_t& m, int& c) {
  const uint32_t chunks = (uint32_t)(p.I + 7) / 8;
  const uint64_t first = (uint64_t)blockIdx.x * kSwigluThreads;
  const uint64_t row0 = first / chunks;  // scalar
  const uint32_t local = (uint32_t)(first - row0 * chunks) + threadIdx.x;
  const uint32_t down = local / chunks;
  m = (int64_t)(row0 + down);
  c = (int)(local - down * chunks);
  const int rows = p.last ? min(max(*p.last, 0), p.M) : p.M;
  return m < rows;
}

template <typename X, typename Y>
__global__ __launch_bounds__(kSwigluThreads) void swiglu_kernel(SwigluArgs p) {
  int64_t m;
  int c;
  if (!my_chunk(p, m, c)) return;
  const int at = 8 * c, have = min(p.I - at, 8);
  const X* const row = (const X*)p.gu + m * p.ld + at;
  const Chunk<X> rg = load_chunk(row, have), ru = load_chunk(row + p.I, have);
  float g[8], u[8];
  values(rg, g);
  values(ru, u);
#pragma unroll
  for (int e = 0; e < 8; ++e) u[e] *= silu(g[e], sigmoid(g[e]).s);
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
  const Chunk<X> rg = load_chunk(row, 8), ru = load_chunk(row + p.I, 8);
  float g[8], u[8];
  values(rg, g);
  values(ru, u);
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    u[e] *= silu(g[e], sigmoid(g[e]).s);
    top = fmaxf(top, fabsf(u[e]));
  }
  const float amax = __uint_as_float(row16_max_u32(__float_as_uint(top)));
  const float s = tile_scale(amax);
  const TileDivisor d = make_divisor(s, amax);
  uint2 codes;
  codes.x = pack4_e4m3(quotient(u[0], d), quotient(u[1], d), quotient(u[2], d), quotient(u[3], d));
  codes.y = pack4_e4m3(quotient(u[4], d), quotient(u[5], d), quotient(u[6], d), quotient(u[7], d));
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
  const Chunk<X> rg = load_chunk(row, have), ru = load_chunk(row + p.I, have);
  const Chunk<D> rd = load_chunk((const D*)p.dy + m * p.ldy + at, have);
  float g[8], u[8], d[8];
  values(rg, g);
  values(ru, u);
  values(rd, d);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const Gate k = sigmoid(g[e]);
    const float y = silu(g[e], k.s);
    // s (1 + gate (1 - s)) = s + (gate s) (1 - s); an infinite gate's slope is 0 or 1
    const float slope = k.c == 0.0f ? k.s : __builtin_fmaf(y, k.c, k.s);
    g[e] = d[e] * u[e] * slope;
    u[e] = d[e] * y;
  }
  X* const out = (X*)p.out + m * (int64_t)(2 * p.I) + at;
  Chunk<X> o;
  to_chunk(g, o);
  store_chunk(out, o, have);
  to_chunk(u, o);
  store_chunk(out + p.I, o, have);
}

static dim3 chunk_grid(const SwigluArgs& a) {
  const int64_t chunks = (int64_t)a.M * ((a.I + 7) / 8);
  return dim3((unsigned)((chunks + kSwigluThreads - 1) / kSwigluThreads));
}

hipError_t launch_swiglu(const void* gu, bool gu_bf16, int64_t ld, const int32_t* last, int64_t M, int64_t I, void* y,
                         bool y_bf16, hipStream_t stream) {
  const SwigluArgs a{gu, nullptr, y, nullptr, last, ld, 0, (int)M, (int)I};
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, chunk_grid(a), dim3(kSwigluThreads), 0, stream, a); };
  if (gu_bf16) y_bf16 ? go(swiglu_kernel<bf16_t, bf16_t>) : go(swiglu_kernel<bf16_t, float>);
  else y_bf16 ? go(swiglu_kernel<float, bf16_t>) : go(swiglu_kernel<float, float>);
  return hipGetLastError();
}

hipError_t launch_swiglu_quant(const void* gu, bool gu_bf16, int64_t ld, const int32_t* last, int64_t M, int64_t I,
                               uint8_t* q, float* sa, hipStream_t stream) {
  const SwigluArgs a{gu, nullptr, q, sa, last, ld, 0, (int)M, (int)I};
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, chunk_grid(a), dim3(kSwigluThreads), 0, stream, a); };
  gu_bf16 ? go(swiglu_quant_kernel<bf16_t>) : go(swiglu_quant_kernel<float>);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const void* dy, bool dy_bf16, int64_t ldy, const void* gu, bool gu_bf16, int64_t ld,
                             const int32_t* last, int64_t M, int64_t I, void* dgu, hipStream_t stream) {
  const SwigluArgs a{gu, dy, dgu, nullptr, last, ld, ldy, (int)M, (int)I};
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, chunk_grid(a), dim3(kSwigluThreads), 0, stream, a); };
  if (gu_bf16) dy_bf16 ? go(swiglu_bwd_kernel<bf16_t, bf16_t>) : go(swiglu_bwd_kernel<bf16_t, float>);
  else dy_bf16 ? go(swiglu_bwd_kernel<float, bf16_t>) : go(swiglu_bwd_kernel<float, float>);
  return hipGetLastError();
}

}  // namespace fp8q
