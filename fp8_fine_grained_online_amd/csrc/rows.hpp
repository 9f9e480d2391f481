// Rows of bfloat16 or binary32 in chunks of eight values, at any element alignment.
#pragma once

#include "common.hpp"

namespace fp8q {

struct bf16_t {
  uint16_t bits;
};

// 16 bytes at an address aligned to an element only: gfx950 reads and writes
// them in one instruction whatever the alignment.
typedef uint32_t u32x4_by2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_by4 __attribute__((ext_vector_type(4), aligned(4)));

// Eight values as they lie in memory.
template <typename T>
struct Chunk;
template <>
struct Chunk<bf16_t> {
  u32x4 v;
};
template <>
struct Chunk<float> {
  u32x4 v[2];
};

__device__ __forceinline__ Chunk<bf16_t> zero_chunk(bf16_t) { return {u32x4{0, 0, 0, 0}}; }
__device__ __forceinline__ Chunk<float> zero_chunk(float) { return {{u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}}}; }

// `have` values (1 to 8) at p; those beyond are zero
__device__ __forceinline__ Chunk<bf16_t> load_chunk(const bf16_t* p, int have) {
  Chunk<bf16_t> c = zero_chunk(bf16_t{});
  if (have >= 8) {
    c.v = *(const u32x4_by2*)p;
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < have) c.v[e / 2] |= (uint32_t)p[e].bits << (16 * (e & 1));
  }
  return c;
}
__device__ __forceinline__ Chunk<float> load_chunk(const float* p, int have) {
  Chunk<float> c = zero_chunk(0.0f);
  if (have >= 8) {
    c.v[0] = *(const u32x4_by4*)p;
    c.v[1] = *(const u32x4_by4*)(p + 4);
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < have) c.v[e / 4][e % 4] = __float_as_uint(p[e]);
  }
  return c;
}

__device__ __forceinline__ void values(const Chunk<bf16_t>& c, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(c.v[i]), f[2 * i + 1] = bf16_hi(c.v[i]);
}
__device__ __forceinline__ void values(const Chunk<float>& c, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(c.v[i / 4][i % 4]);
}

// to bfloat16, nearest even (the hardware's conversion; NaN stays NaN)
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
}

// eight values rounded to T
__device__ __forceinline__ void to_chunk(const float (&f)[8], Chunk<bf16_t>& c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c.v[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ void to_chunk(const float (&f)[8], Chunk<float>& c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) c.v[i / 4][i % 4] = __float_as_uint(f[i]);
}

// the first `have` values (1 to 8) to p
__device__ __forceinline__ void store_chunk(bf16_t* p, const Chunk<bf16_t>& c, int have) {
  if (have >= 8) {
    *(u32x4_by2*)p = c.v;
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < have) p[e].bits = (uint16_t)(c.v[e / 2] >> (16 * (e & 1)));
  }
}
__device__ __forceinline__ void store_chunk(float* p, const Chunk<float>& c, int have) {
  if (have >= 8) {
    *(u32x4_by4*)p = c.v[0];
    *(u32x4_by4*)(p + 4) = c.v[1];
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < have) p[e] = __uint_as_float(c.v[e / 4][e % 4]);
  }
}

// eight weights, whose type is known at run time only
__device__ __forceinline__ void load_weights(const void* w, bool bf16, int64_t at, int have, float (&f)[8]) {
  if (bf16) values(load_chunk((const bf16_t*)w + at, have), f);
  else values(load_chunk((const float*)w + at, have), f);
}

}  // namespace fp8q
