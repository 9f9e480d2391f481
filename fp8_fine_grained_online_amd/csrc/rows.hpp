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

// A whole chunk at p; kNt: read once, so it need not stay cached
template <bool kNt = false>
__device__ __forceinline__ Chunk<bf16_t> load_whole(const bf16_t* p) {
  const u32x4_by2* const q = (const u32x4_by2*)p;
  return {kNt ? (u32x4)__builtin_nontemporal_load(q) : (u32x4)*q};
}
template <bool kNt = false>
__device__ __forceinline__ Chunk<float> load_whole(const float* p) {
  const u32x4_by4* const q = (const u32x4_by4*)p;
  if constexpr (kNt) return {{__builtin_nontemporal_load(q), __builtin_nontemporal_load(q + 1)}};
  else return {{q[0], q[1]}};
}

// `have` values (0 to 7) at p, one by one; those beyond are zero
__device__ __forceinline__ Chunk<bf16_t> load_few(const bf16_t* p, int have) {
  Chunk<bf16_t> c = zero_chunk(bf16_t{});
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < have) c.v[e / 2] |= (uint32_t)p[e].bits << (16 * (e & 1));
  return c;
}
__device__ __forceinline__ Chunk<float> load_few(const float* p, int have) {
  Chunk<float> c = zero_chunk(0.0f);
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < have) c.v[e / 4][e % 4] = __float_as_uint(p[e]);
  return c;
}

// `have` values (1 to 8) at p; those beyond are zero
template <bool kNt = false, typename T>
__device__ __forceinline__ Chunk<T> load_chunk(const T* p, int have) {
  return have >= 8 ? load_whole<kNt>(p) : load_few(p, have);
}

// The chunk without its first n values (0 to 7), zeros behind
__device__ __forceinline__ Chunk<bf16_t> shifted(const Chunk<bf16_t>& c, int n) {
  uint64_t lo = (uint64_t)c.v[1] << 32 | c.v[0], hi = (uint64_t)c.v[3] << 32 | c.v[2];
  if (n & 4) lo = hi, hi = 0;
  const int bits = 16 * (n & 3);
  if (bits) lo = lo >> bits | hi << (64 - bits), hi >>= bits;
  return {u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)}};
}
__device__ __forceinline__ Chunk<float> shifted(const Chunk<float>& c, int n) {
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = c.v[e / 4][e % 4];
#pragma unroll
  for (int b = 1; b <= 4; b <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = n & b ? (e + b < 8 ? w[e + b] : 0u) : w[e];
  Chunk<float> o;
#pragma unroll
  for (int e = 0; e < 8; ++e) o.v[e / 4][e % 4] = w[e];
  return o;
}

// Values at .. at + 7 of a row of K >= 8; zeros past its end. The chunk that ends
// past the row is loaded whole all the same, so that it ends with the row, and
// shifted into place.
template <bool kNt = false, typename T>
__device__ __forceinline__ Chunk<T> load_in_row(const T* row, int at, int K) {
  const int past = at + 8 - K;
  Chunk<T> c = load_whole<kNt>(row + (past > 0 ? K - 8 : at));
  if (past > 0) c = shifted(c, past);
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

}  // namespace fp8q
