// 8-bit integer product with one scale per token and per output channel, for
// gfx950 (CDNA4 MFMA), dense and grouped (MoE), and the row quantization that
// feeds it.
//
//   c[m, n] = (sum_k a[m, k] b[n, k]) sa[m] sb[n]
//
// The integer matrix cores (v_mfma_i32_16x16x64_i8, the rate of FP8) add into
// int32 registers, exactly, over the whole of K: nothing is promoted inside
// the loop, and any order or split of K gives the same bits. The two scales
// are applied once, in the epilogue.
#include <type_traits>

#include "common.hpp"
#include "tiles.hpp"
#include "wave.hpp"

namespace fp8q {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// 16 bytes at an address aligned to an element only
typedef uint32_t u32x4_by2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_by4 __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kStepK = 128;  // bytes of K per pipeline step

struct I8Args {
  const uint8_t* a;
  const float* sa;
  const uint8_t* b;
  const float* sb;
  void* c;
  const int32_t* m_offsets;  // grouped only
  int M, N, K, G;
};

__device__ __forceinline__ float scaled(int v, float sa, float sb) {
  return ((float)v * sa) * sb;
}

// ---------------------------------------------------------------------------
// Row quantization. kWaves wavefronts per row; a lane owns chunks of 8 values
// (16 bytes in, 8 bytes of codes out), so that every load and store of a wave
// is one contiguous run. A row of up to kHeld chunks per lane stays in
// registers between its maximum and its codes; longer rows are read twice (the
// second time from the cache). A workgroup per row beats a wavefront per row
// and 16 values per lane: 69632 x 7168 240, 250 and 254 us (6.2 TB/s of reads
// and writes), 8192 x 7168 29.3, 32.4 and 34.4; rows of up to 2048 values
// are too short to share.
//
// The quotient x / s is formed as q0 = x r, q = q0 + (x - q0 s) r with
// r = RN(1 / s). A host comparison over every bfloat16 significand of the
// maximum and of x, down to quotients that give code 0, found q equal to the
// correctly rounded quotient throughout (scaling x and s by powers of two
// changes nothing). Maxima outside [2^-64, 2^100) are scaled into it first, so
// that nothing under- or overflows. Adding 1.5 * 2^23 then rounds q to an
// integer, ties to even, in the low bits of the sum. |x / s| rounds to at most
// 127 (s is within 2^-10 of amax / 127 even where it is subnormal), so no clamp
// is needed. With an IEEE division in its place the kernel was bound by the
// vector ALU (69632 x 7168: 277 us).
// ---------------------------------------------------------------------------
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// largest magnitude bits of the 8 values of a chunk, two halves at once
__device__ __forceinline__ u16x2 absmax_bits(u16x2 m, uint4 a) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, abs2_bits(w[i])));
  return m;
}

struct RowScale {
  float s, r;  // divisor and its reciprocal, both after scaling by p
  float p;     // power of two for x
};

template <bool kScaled>
__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, const RowScale& d) {
  const float x[4] = {bf16_lo(w0), bf16_hi(w0), bf16_lo(w1), bf16_hi(w1)};
  uint32_t t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float xs = kScaled ? x[i] * d.p : x[i];
    const float q0 = xs * d.r;
    const float q = __builtin_fmaf(__builtin_fmaf(-q0, d.s, xs), d.r, q0);
    t[i] = __float_as_uint(q + 12582912.0f);
  }
  const uint32_t lo = __builtin_amdgcn_perm(t[1], t[0], 0x0c0c0400);
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(t[3], t[2], 0x0c0c0400), lo, 0x05040100);
}

template <bool kScaled>
__device__ __forceinline__ u32x2 codes8(uint4 a, const RowScale& d) {
  return u32x2{codes4<kScaled>(a.x, a.y, d), codes4<kScaled>(a.z, a.w, d)};
}

template <int kWaves, int kHeld, bool kNt>
__global__ __launch_bounds__(256) void quant_int8_rows_kernel(const uint4* __restrict__ x, int M,
                                                              int K, u32x2* __restrict__ q,
                                                              float* __restrict__ s_out) {
  constexpr int kThreads = 64 * kWaves;  // per row
  __shared__ uint32_t wave_amax[4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m = (int64_t)blockIdx.x * (4 / kWaves) + wave / kWaves;
  if (m >= M) return;
  const int tid = threadIdx.x % kThreads;
  const int n = K / 8;
  const uint4* xr = x + m * (int64_t)n;
  u32x2* qr = q + m * (int64_t)n;
  const bool held = n <= kHeld * kThreads;
  uint4 v[kHeld];
  u16x2 top = {0, 0};
  if (held) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int c = tid + u * kThreads;
      v[u] = make_uint4(0, 0, 0, 0);
      if (c < n) v[u] = load_nt(xr + c);
    }
#pragma unroll
    for (int u = 0; u < kHeld; ++u) top = absmax_bits(top, v[u]);
  } else {
#pragma unroll 4
    for (int c = tid; c < n; c += kThreads) top = absmax_bits(top, xr[c]);
  }
  // magnitudes of finite values order like their bits
  uint32_t bits = wave_max_u32(umax(top.x, top.y));
  if constexpr (kWaves > 1) {
    if ((threadIdx.x & 63) == 0) wave_amax[wave] = bits;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) bits = umax(bits, wave_amax[w]);
    bits = __builtin_amdgcn_readfirstlane(bits);
  }
  const float amax = __uint_as_float(bits << 16);
  const float s = __fdiv_rn(amax, 127.0f);
  if (tid == 0) s_out[m] = s;
  RowScale d;
  d.p = amax < 0x1p-64f ? 0x1p+64f : amax >= 0x1p+100f ? 0x1p-32f : 1.0f;
  d.s = amax > 0.0f ? s * d.p : 1.0f;  // exact: a power of two
  d.r = __fdiv_rn(1.0f, d.s);
  auto store = [&](int c, u32x2 codes) {
    if constexpr (kNt) __builtin_nontemporal_store(codes, qr + c);
    else qr[c] = codes;
  };
  if (held && d.p == 1.0f) {  // wave-uniform
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int c = tid + u * kThreads;
      if (c < n) store(c, codes8<false>(v[u], d));
    }
  } else {
#pragma unroll 4
    for (int c = tid; c < n; c += kThreads) store(c, codes8<true>(xr[c], d));
  }
}

// ---------------------------------------------------------------------------
// Tiled product. A workgroup of four wavefronts, one per SIMD, computes a
// BM x BN tile, each wave a WM x WN quarter of it. Because nothing but MFMAs
// touches the accumulators they can live in AGPRs, so a wave may hold a
// 128 x 128 part (256 registers) and still has 256 VGPRs: a large part needs
// the fewest operand bytes from LDS per MFMA.
//
// Per step of 128 bytes of K the slabs of A and B go straight from global
// memory to LDS; 16-byte chunk c of row r sits at position c ^ (r % 8), so the
// rows of one operand load fall in distinct banks. A step is multiplied in two
// halves of 64 bytes (one MFMA deep), each from its own set of operand
// registers: while half h multiplies, the other half's operands are read from
// LDS, so an MFMA never waits for a read issued just before it.
//
//   first half of step g   multiplies (g, 0), reads (g, 1), copies A of g + D
//   barrier: every wave has read all of step g's slabs, and step g + 1's have landed
//   second half            multiplies (g, 1), reads (g + 1, 0), copies B of g + D
//
// A's slabs rotate through D + 1 buffers, B's through D (D = 2 and 160 KB in all
// for 256 x 256): a copy has D - 1 steps to land, A's half a step more. Smaller
// tiles multiply a step in less time than a copy takes, and look further ahead.
//
// Operand lanes: lane l supplies row l % 16 of a 16-row block and the 16 bytes
// of K at chunk l / 16 (or 4 + l / 16 for the second half). B is the first
// operand, so a lane holds C[m = l % 16][n = 4 (l / 16) + r], four consecutive
// columns of one row.
//
// Edges: the buffer descriptors cover the tile's valid rows, and in the last
// step the chunks past K get an offset outside them; both read as zeros.
// ---------------------------------------------------------------------------
template <int BM, int BN, int D, int S>
struct I8Tile {
  static constexpr int kThreads = 256;  // of one K group
  static constexpr int kWM = BM / 2, kWN = BN / 2;
  static constexpr int kSlabA = BM * kStepK, kSlabB = BN * kStepK;
  static constexpr int kRing = (D + 1) * kSlabA + D * kSlabB;
  static constexpr int kLds = S * kRing;
  static constexpr int kLoadsA = BM * 8 / kThreads, kLoadsB = BN * 8 / kThreads;
  static_assert(kWM % 16 == 0 && kWN % 16 == 0, "whole MFMA blocks");
  static_assert(BM * 8 % kThreads == 0 && BN * 8 % kThreads == 0, "whole copies");
  static_assert(kLds <= 160 * 1024 && D >= 2, "LDS");
  static_assert((D - 1) * (kLoadsA + kLoadsB) <= 63, "the wait counter holds the copies in flight");
};

constexpr uint32_t kOutside = 0x80000000u;  // past every descriptor: reads as zero

// s_waitcnt immediates: vector-memory count <= n alone; LDS count 0 alone
constexpr int wait_vm(int n) { return 0x0F70 | (n & 15) | ((n >> 4) << 14); }
constexpr int kWaitLds = 0xC07F;

template <int BM, int BN, int D, int S, bool kBf16, bool kGrouped>
__global__ __launch_bounds__(256 * S, S) void gemm_i8_kernel(I8Args p) {
  using Cfg = I8Tile<BM, BN, D, S>;
  constexpr int WM = Cfg::kWM, WN = Cfg::kWN;
  constexpr int SUBM = WM / 16, SUBN = WN / 16;
  constexpr int kMfmas = SUBM * SUBN;
  __shared__ __attribute__((aligned(16))) uint8_t lds_all[Cfg::kLds];
  const int tid = threadIdx.x & 255, lane = tid & 63;
  const int group = S > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) : 0;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint8_t* const lds = lds_all + group * Cfg::kRing;
  const int wm = wave >> 1, wn = wave & 1;
  const int lr = lane & 15, lk = lane >> 4;
  const int n_tiles_n = (p.N + BN - 1) / BN;

  int m0, m_end, tm, tn;
  const uint8_t* bmat = p.b;
  const float* sbv = p.sb;
  if constexpr (kGrouped) {
    // The grid is an upper bound: the host does not know the offsets. Count the
    // real tiles (one expert per lane, 64 a round) and give every XCD its share
    // of those, then find the expert that holds this workgroup's tile.
    // Values found by a lane are read back with readlane into variables of
    // their own: a buffer descriptor built from a vector value becomes a loop.
    int l_lo = 0, l_hi = 0, l_te = 0;
    auto expert = [&](int e) {  // this lane's expert's rows and tiles; tiles up to and with this lane
      l_lo = l_hi = l_te = 0;
      if (e < p.G) {
        l_lo = min(max(p.m_offsets[e], 0), p.M);
        l_hi = min(max(p.m_offsets[e + 1], l_lo), p.M);
        l_te = (l_hi - l_lo + BM - 1) / BM;
      }
      int incl = l_te * n_tiles_n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(incl, d);
        if (lane >= d) incl += v;
      }
      return incl;
    };
    int total = 0;
    for (int e0 = 0; e0 < p.G; e0 += 64) total += __builtin_amdgcn_readlane(expert(e0 + lane), 63);
    if ((int)blockIdx.x >= total) return;
    const int tile = xcd_tile(blockIdx.x, total);
    int e = 0, before = 0, lo = 0, hi = 0, te = 0;
    for (int e0 = 0; e0 < p.G; e0 += 64) {
      const int incl = expert(e0 + lane);
      const uint64_t hit = __ballot(tile < before + incl);
      if (hit) {
        const int L = __builtin_ctzll(hit);
        e = e0 + L;
        lo = __builtin_amdgcn_readlane(l_lo, L);
        hi = __builtin_amdgcn_readlane(l_hi, L);
        te = __builtin_amdgcn_readlane(l_te, L);
        before += __builtin_amdgcn_readlane(incl - l_te * n_tiles_n, L);
        break;
      }
      before += __builtin_amdgcn_readlane(incl, 63);
    }
    const int local = tile - before;
    // (fails only for offsets outside the contract, where the counts overflow)
    if ((uint32_t)local >= (uint32_t)(te * n_tiles_n)) return;
    band_tile<kBandGrouped>(local, te, n_tiles_n, tm, tn);
    m0 = lo + tm * BM;
    m_end = min(m0 + BM, hi);
    bmat += (int64_t)e * p.N * p.K;
    sbv += (int64_t)e * p.N;
  } else {
    band_tile(xcd_tile(blockIdx.x, gridDim.x), (p.M + BM - 1) / BM, n_tiles_n, tm, tn);
    m0 = tm * BM;
    m_end = min(m0 + BM, p.M);
  }
  const int n0 = tn * BN;
  const int rows_a = m_end - m0, rows_b = min(BN, p.N - n0);
  const __amdgpu_buffer_rsrc_t rsrc_a = make_rsrc(p.a + (int64_t)m0 * p.K, (uint32_t)rows_a * (uint32_t)p.K);
  const __amdgpu_buffer_rsrc_t rsrc_b = make_rsrc(bmat + (int64_t)n0 * p.K, (uint32_t)rows_b * (uint32_t)p.K);
  // this group's steps of K: first .. first + steps - 1, those past the last reading zeros
  const int all_steps = (p.K + kStepK - 1) / kStepK;
  const int steps = (all_steps + S - 1) / S;
  const int first = group * steps;
  // The epilogue's scales. Loaded before the loop, they are not one more wait for
  // memory at the end (the largest wave tile has no registers to hold them).
  const int nw = n0 + wn * WN;
  constexpr bool kScalesFirst = SUBM * SUBN < 64;
  float sav[SUBM], sbc[SUBN][4];
  auto load_scales = [&]() {
#pragma unroll
    for (int i = 0; i < SUBM; ++i) {
      const int m = m0 + wm * WM + i * 16 + lr;
      sav[i] = m < m_end && p.K > 0 ? p.sa[m] : 0.0f;  // K == 0: no operand is read
    }
#pragma unroll
    for (int j = 0; j < SUBN; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int n = nw + j * 16 + 4 * lk + r;
        sbc[j][r] = n < p.N && p.K > 0 ? sbv[n] : 0.0f;
      }
  };
  if constexpr (kScalesFirst) load_scales();
  // copy q of thread tid brings row q * 32 + tid / 8, stored chunk tid % 8
  const int row0 = tid >> 3, lc0 = (tid & 7) ^ (row0 & 7);
  constexpr int kRows = Cfg::kLoadsA > Cfg::kLoadsB ? Cfg::kLoadsA : Cfg::kLoadsB;
  uint32_t off[kRows];
#pragma unroll
  for (int q = 0; q < kRows; ++q) off[q] = (uint32_t)(row0 + q * 32) * (uint32_t)p.K + lc0 * 16;
  // From the last step's copies on, a thread whose chunk is past K reads zeros
  // (and every thread, past that step)
  const bool past = (all_steps - 1) * kStepK + lc0 * 16 >= p.K;
  auto enter_step = [&](int g) {
    if (first + g >= all_steps - 1) {
      const bool out = past || first + g >= all_steps;
#pragma unroll
      for (int q = 0; q < kRows; ++q) off[q] = out ? kOutside : off[q];
    }
  };
  // Byte of K where step g of this group starts. The second group may have one step
  // more than K: its offset stays that of the last step, because a load's range check
  // may subtract the scalar offset from the descriptor's size, and past a tile of one
  // row the difference would wrap around and let the load through.
  auto step_k = [&](int g) { return (S > 1 ? min(first + g, all_steps - 1) : first + g) * kStepK; };
  auto copy_a = [&](int q, int k, uint8_t* __restrict__ to) {
    load_lds(rsrc_a, to + (q * 256 + wave * 64) * 16, 16, off[q], k);
  };
  auto copy_b = [&](int q, int k, uint8_t* __restrict__ to) {
    load_lds(rsrc_b, to + (q * 256 + wave * 64) * 16, 16, off[q], k);
  };

  v4i acc[SUBM][SUBN];
#pragma unroll
  for (int i = 0; i < SUBM; ++i)
#pragma unroll
    for (int j = 0; j < SUBN; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  v4i ra[2][SUBM], rb[2][SUBN];  // operands of the two halves
  const int a_off[2] = {(wm * WM + lr) * kStepK + ((lk ^ (lr & 7)) << 4),
                        (wm * WM + lr) * kStepK + (((4 + lk) ^ (lr & 7)) << 4)};
  const int b_off[2] = {a_off[0] + (wn * WN - wm * WM) * kStepK, a_off[1] + (wn * WN - wm * WM) * kStepK};
  // operand number u of half h: B's blocks first, the order the MFMAs want them in
  auto read_operand = [&](int u, int h, const uint8_t* __restrict__ sa, const uint8_t* __restrict__ sb) {
    if (u < SUBN) rb[h][u] = *(const v4i*)(sb + b_off[h] + u * 16 * kStepK);
    else ra[h][u - SUBN] = *(const v4i*)(sa + a_off[h] + (u - SUBN) * 16 * kStepK);
  };
  // MFMAs from one operand read (and from one copy) to the next
  constexpr int kEvery = kMfmas >= 2 * (SUBM + SUBN) ? 2 : 1;
  // Half h of a step: its MFMAs, with the other half's operands read from
  // (sa, sb) and one operand's copies (`issue`) spread between them. Scheduling
  // barriers keep that order.
  auto half = [&](int h, const uint8_t* __restrict__ sa, const uint8_t* __restrict__ sb, int k,
                  uint8_t* __restrict__ to, bool copy_is_a) {
#pragma unroll
    for (int t = 0; t < kMfmas; ++t) {
      const int i = t / SUBN, j = t % SUBN;
      if (t % kEvery == 0 && t / kEvery < SUBM + SUBN) read_operand(t / kEvery, 1 - h, sa, sb);
      if (t % kEvery == kEvery - 1) {
        const int q = t / kEvery;
        if (copy_is_a) { if (q < Cfg::kLoadsA) copy_a(q, k, to); }
        else { if (q < Cfg::kLoadsB) copy_b(q, k, to); }
      }
      acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(rb[h][j], ra[h][i], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  static_assert(kMfmas / kEvery >= SUBM + SUBN && kMfmas / kEvery >= kRows, "reads and copies fit between the MFMAs");

  // a wave whose rows all lie past the tile's valid ones only copies
  const bool idle = wm * WM >= rows_a;
  uint8_t* const lds_b = lds + (D + 1) * Cfg::kSlabA;
  if (steps > 0) {
    enter_step(0);
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int g = min(d, steps - 1);
      if (d > 0) enter_step(g);
      const int k = step_k(g);
#pragma unroll
      for (int q = 0; q < Cfg::kLoadsA; ++q) copy_a(q, k, lds + d * Cfg::kSlabA);
#pragma unroll
      for (int q = 0; q < Cfg::kLoadsB; ++q) copy_b(q, k, lds_b + d * Cfg::kSlabB);
    }
    __builtin_amdgcn_s_waitcnt(wait_vm((D - 1) * (Cfg::kLoadsA + Cfg::kLoadsB)));
    __builtin_amdgcn_s_barrier();
    if (!idle) {
#pragma unroll
      for (int u = 0; u < SUBM + SUBN; ++u) read_operand(u, 0, lds, lds_b);
    }
  }
  // offsets of the buffers of this step's and the next step's slabs, and of the one A is copied to
  int a0 = 0, a1 = Cfg::kSlabA, a2 = D * Cfg::kSlabA;
  int b0 = 0, b1 = D > 1 ? Cfg::kSlabB : 0;
  for (int g = 0; g < steps; ++g) {
    const int gn = min(g + D, steps - 1);  // past the end the last step is copied again, unread
    enter_step(gn);
    const int kn = step_k(gn);
    if (idle) {
#pragma unroll
      for (int q = 0; q < Cfg::kLoadsA; ++q) copy_a(q, kn, lds + a2);
    } else {
      half(0, lds + a0, lds_b + b0, kn, lds + a2, true);
    }
    // this wave has read all of step g, and its copies of step g + 1 have landed
    __builtin_amdgcn_s_waitcnt(kWaitLds);
    __builtin_amdgcn_s_waitcnt(wait_vm((D - 1) * Cfg::kLoadsA + (D - 2) * Cfg::kLoadsB));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (idle) {
#pragma unroll
      for (int q = 0; q < Cfg::kLoadsB; ++q) copy_b(q, kn, lds_b + b0);
    } else {
      half(1, lds + a1, lds_b + b1, kn, lds_b + b0, false);
    }
    a2 = a0, a0 = a1, b0 = b1;
    a1 = a1 == D * Cfg::kSlabA ? 0 : a1 + Cfg::kSlabA;
    b1 = b1 == (D - 1) * Cfg::kSlabB ? 0 : b1 + Cfg::kSlabB;
  }
  // the last copies may still be writing the buffers that are used again below
  __builtin_amdgcn_s_waitcnt(wait_vm(0));
  __syncthreads();
  if constexpr (S > 1) {
    // add the groups' sums: integers, so any order gives the same bits
    static_assert((S - 1) * BM * BN * 4 <= Cfg::kLds, "the other groups' sums fit");
    v4i* const part = (v4i*)lds_all + wave * (kMfmas * 64) + lane;
    if (group > 0) {
#pragma unroll
      for (int t = 0; t < kMfmas; ++t) part[(group - 1) * (4 * kMfmas * 64) + t * 64] = acc[t / SUBN][t % SUBN];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int s = 0; s < S - 1; ++s)
#pragma unroll
      for (int t = 0; t < kMfmas; ++t) acc[t / SUBN][t % SUBN] += part[s * (4 * kMfmas * 64) + t * 64];
    __builtin_amdgcn_s_waitcnt(kWaitLds);
  }

  // ---- epilogue: scale, stage 16 rows of the wave's part in its own LDS, store rows ----
  constexpr int kEl = kBf16 ? 2 : 4;        // bytes per output
  constexpr int kRowBytes = WN * kEl;
  constexpr int kChunks = kRowBytes / 16;
  static_assert((S > 1 ? kMfmas * 64 * 16 : Cfg::kLds / 4) >= 16 * kRowBytes, "staging");
  // (with S > 1 a wave stages where its own part of the other groups' sums was)
  uint8_t* st = lds + wave * (S > 1 ? kMfmas * 64 * 16 : 16 * kRowBytes);
  if constexpr (!kScalesFirst) load_scales();
#pragma unroll
  for (int i = 0; i < SUBM; ++i) {
#pragma unroll
    for (int j = 0; j < SUBN; ++j) {
      float v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = scaled(acc[i][j][r], sav[i], sbc[j][r]);
      const int byte = (j * 16 + 4 * lk) * kEl;
      uint8_t* to = st + lr * kRowBytes + (((byte >> 4) ^ (lr & (kChunks - 1))) << 4) + (byte & 15);
      if constexpr (kBf16) *(bf16x4*)to = bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
      else *(v4f*)to = v4f{v[0], v[1], v[2], v[3]};
    }
    __builtin_amdgcn_s_waitcnt(kWaitLds);  // a wave reads back only its own part
    __builtin_amdgcn_wave_barrier();
    // 16 bytes per lane, neighbouring lanes in a row. Rows of c start at any
    // element, so the stores are not aligned to more than that (narrower, aligned
    // ones where N is odd: 1024 x 4097 x 2048 17.7 -> 21.5 us, bfloat16).
    using Out = std::conditional_t<kBf16, u32x4_by2, u32x4_by4>;
    constexpr int kPer = 16 / kEl;
    static_assert(kChunks % 64 == 0 || 64 % kChunks == 0, "whole wave stores");
#pragma unroll
    for (int k = 0; k < kChunks / 4; ++k) {
      const int m = (k * 64 + lane) / kChunks, ch = (k * 64 + lane) % kChunks;
      const int om = m0 + wm * WM + i * 16 + m, n = nw + ch * kPer;
      const v4i v = *(const v4i*)(st + m * kRowBytes + ((ch ^ (m & (kChunks - 1))) << 4));
      if (om >= m_end) continue;
      uint8_t* const to = (uint8_t*)p.c + ((int64_t)om * p.N + n) * kEl;
      if (n + kPer <= p.N) {
        *(Out*)to = __builtin_bit_cast(Out, v);
      } else {  // the row's end
#pragma unroll
        for (int r = 0; r < kPer; ++r) {
          if (n + r >= p.N) break;
          if constexpr (kBf16) ((uint16_t*)to)[r] = (uint16_t)(v[r / 2] >> (r % 2 * 16));
          else ((int*)to)[r] = v[r];
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// ---------------------------------------------------------------------------
// Small products: a workgroup owns 16 MB x 16 NB outputs and its W waves split
// K between them in pieces of 64 bytes (one MFMA deep), each streaming its
// fragments straight from global memory to registers, kAhead pieces ahead; the
// int32 partial blocks are added through LDS. For products too small to give
// every CU a large tile, and for few rows, where B is read once.
//
// kAhead keeps 6 to 8 loads per lane in flight, whatever MB and NB. us on MI355X
// for 1, 2, 4, 6 pieces ahead, operands beyond the Infinity Cache:
//   16 x 16  1 x 4096 x 8192    11.09   9.41   8.41   8.67
//            1 x 4096 x 1024     3.27   3.21   3.24   3.31
//   16 x 32  1 x 7168 x 7168    14.17  11.43  13.25  13.21
//            8 x 16384 x 2048    9.74   9.07   9.20   9.24
//   32 x 16  32 x 4096 x 8192   16.22  14.95  15.81  15.85
//   32 x 32  256 x 1024 x 2032   5.85   5.70   5.95   5.96
// ---------------------------------------------------------------------------
constexpr int kPiece = 64;

template <int MB, int NB, int W, bool kBf16>
__global__ __launch_bounds__(64 * W) void gemm_i8_small_kernel(I8Args p) {
  constexpr int kAhead = 8 / (MB + NB);
  __shared__ __attribute__((aligned(16))) v4i part[W][MB * NB][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lk = lane >> 4;
  const int n_blocks = (p.N + 16 * NB - 1) / (16 * NB);
  const int n0 = (blockIdx.x % n_blocks) * 16 * NB;
  const int m0 = (blockIdx.x / n_blocks) * 16 * MB;
  const int pieces = (p.K + kPiece - 1) / kPiece;
  const int g_begin = (int)((int64_t)pieces * wave / W);
  const int g_end = (int)((int64_t)pieces * (wave + 1) / W);
  const int rows_a = min(16 * MB, p.M - m0), rows_b = min(16 * NB, p.N - n0);
  const __amdgpu_buffer_rsrc_t rsrc_a = make_rsrc(p.a + (int64_t)m0 * p.K, (uint32_t)rows_a * (uint32_t)p.K);
  const __amdgpu_buffer_rsrc_t rsrc_b = make_rsrc(p.b + (int64_t)n0 * p.K, (uint32_t)rows_b * (uint32_t)p.K);
  const uint32_t off = (uint32_t)lr * (uint32_t)p.K + lk * 16;
  const uint32_t blk = 16u * (uint32_t)p.K;

  // Wave b finishes block b of the workgroup's outputs; its scales are loaded
  // before the loop, not to be one more wait for memory at the end.
  static_assert(MB * NB <= W, "a wave per block");
  float sa0 = 0.0f, sb0[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (wave < MB * NB && p.K > 0) {  // K == 0: no operand is read
    const int gm = m0 + (wave / NB) * 16 + lr, gn = n0 + (wave % NB) * 16 + 4 * lk;
    if (gm < p.M) sa0 = p.sa[gm];
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (gn + r < p.N) sb0[r] = p.sb[gn + r];
  }

  struct Frags {
    v4i a[MB], b[NB];
  };
  auto load = [&](int g, Frags& f) {
    const uint32_t o = g * kPiece + lk * 16 < p.K ? off : kOutside;  // chunks past K read as zeros
#pragma unroll
    for (int j = 0; j < NB; ++j)
      f.b[j] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rsrc_b, o + j * blk, g * kPiece, 0));
#pragma unroll
    for (int i = 0; i < MB; ++i)
      f.a[i] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rsrc_a, o + i * blk, g * kPiece, 0));
  };
  v4i acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  auto compute = [&](const Frags& f) {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
  };
  Frags f[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (g_begin + u < g_end) load(g_begin + u, f[u]);
  for (int g = g_begin; g < g_end; g += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (g + u < g_end) compute(f[u]);
      if (g + u + kAhead < g_end) load(g + u + kAhead, f[u]);
    }
  }
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) part[wave][i * NB + j][lane] = acc[i][j];
  __syncthreads();
  if (wave < MB * NB) {
    const int b = wave;
    v4i sum = part[0][b][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) sum += part[w][b][lane];
    const int gm = m0 + (b / NB) * 16 + lr;
    const int gn = n0 + (b % NB) * 16 + 4 * lk;
    if (gm >= p.M) return;
    float v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = scaled(sum[r], sa0, sb0[r]);
    const int64_t at = (int64_t)gm * p.N + gn;
    if (gn + 4 <= p.N) {  // (rows of c start at any element)
      typedef __bf16 Out16 __attribute__((ext_vector_type(4), aligned(2)));
      typedef float Out32 __attribute__((ext_vector_type(4), aligned(4)));
      if constexpr (kBf16) *(Out16*)((__bf16*)p.c + at) = Out16{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
      else *(Out32*)((float*)p.c + at) = Out32{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (gn + r >= p.N) break;
        if constexpr (kBf16) ((__bf16*)p.c)[at + r] = (__bf16)v[r];
        else ((float*)p.c)[at + r] = v[r];
      }
    }
  }
}

hipError_t launch_quant_int8_rows(const void* x, int64_t M, int64_t K, int8_t* q, float* s,
                                  hipStream_t stream) {
  auto go = [&](auto kernel, int rows) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((M + rows - 1) / rows)), dim3(256), 0, stream,
                       (const uint4*)x, (int)M, (int)K, (u32x2*)q, s);
  };
  // codes larger than the 256 MB Infinity Cache cannot stay there for their reader
  const bool nt = M * K > (int64_t(256) << 20);
  if (K <= 2048)
    nt ? go(quant_int8_rows_kernel<1, 4, true>, 4) : go(quant_int8_rows_kernel<1, 4, false>, 4);
  else if (K <= 8192)
    nt ? go(quant_int8_rows_kernel<4, 4, true>, 1) : go(quant_int8_rows_kernel<4, 4, false>, 1);
  else
    nt ? go(quant_int8_rows_kernel<4, 8, true>, 1) : go(quant_int8_rows_kernel<4, 8, false>, 1);
  return hipGetLastError();
}

template <int BM, int BN, int D, int S, bool kGrouped>
static hipError_t launch_tiles(const I8Args& a, bool bf16, int64_t m_tiles, hipStream_t stream) {
  const dim3 grid((unsigned)(m_tiles * ((a.N + BN - 1) / BN))), block(256 * S);
  if (bf16)
    hipLaunchKernelGGL((gemm_i8_kernel<BM, BN, D, S, true, kGrouped>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((gemm_i8_kernel<BM, BN, D, S, false, kGrouped>), grid, block, 0, stream, a);
  return hipGetLastError();
}

template <int MB, int NB, int W>
static hipError_t launch_small(const I8Args& a, bool bf16, hipStream_t stream) {
  const int64_t wgs = (int64_t)((a.M + 16 * MB - 1) / (16 * MB)) * ((a.N + 16 * NB - 1) / (16 * NB));
  if (bf16)
    hipLaunchKernelGGL((gemm_i8_small_kernel<MB, NB, W, true>), dim3((unsigned)wgs), dim3(64 * W), 0, stream, a);
  else
    hipLaunchKernelGGL((gemm_i8_small_kernel<MB, NB, W, false>), dim3((unsigned)wgs), dim3(64 * W), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_int8_gemm(const int8_t* a, const float* sa, const int8_t* b, const float* sb,
                            void* c, bool bf16, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  const I8Args p{(const uint8_t*)a, sa, (const uint8_t*)b, sb, c, nullptr, (int)M, (int)N, (int)K, 1};
  // Workgroups of bm x bn outputs
  auto wgs = [&](int64_t bm, int64_t bn) { return (M + bm - 1) / bm * ((N + bn - 1) / bn); };
  // The smallest tile that still gives every CU at most one workgroup: below
  // that, CUs idle while others load twice the operand bytes (a CU loads about
  // 90 GB/s whatever its tile); above it, some CUs work twice. Measured on
  // MI355X, us for the chosen tile against its neighbours in size:
  //   64 x 512 x 512         16x16 2.64   32x16 2.81   32x32 3.15
  //   256 x 512 x 2048       32x16 4.87   32x32 5.79   64x64 6.66
  //   256 x 1024 x 512       32x32 3.27   32x16 3.64   64x64 4.03
  //   333 x 2050 x 2064      64x64 8.6    64x128 11.0  32x32 14.4
  //   1024 x 2048 x 2048     64x128 9.0   64x64 12.7   128x128 11.3
  //   1024 x 4096 x 4096     128x128 21.2 64x128 24.1  256x256 47.8
  // Long K is better shared through LDS: 32 x 7168 x 7168 takes 12.5 us in
  // 64x64 tiles and 15.5 in 32x32; at K = 2048 they are equal, 6.5 and 6.3.
  if (M <= 16 && wgs(16, 16) > kCus) return launch_small<1, 2, 8>(p, bf16, stream);
  if (wgs(16, 16) <= kCus) return launch_small<1, 1, 8>(p, bf16, stream);
  if (wgs(32, 16) <= kCus) return launch_small<2, 1, 8>(p, bf16, stream);
  if (wgs(32, 32) <= kCus && K < 2048) return launch_small<2, 2, 8>(p, bf16, stream);
  if (wgs(64, 64) <= kCus) {
    // Two groups of waves that share K have half the steps each but their sums to
    // add, and twice the loads in flight. That pays from K = 2048 on where rows
    // start at whole 128-byte lines; else every copy touches two lines, the cache is
    // what is waited for, and it pays from about 8192 on. us, one group with 5
    // buffers / two groups with 3 (4 buffers: the same), MI355X:
    //     K    200 x 4096     333 x 2050     500 x 1000     1024 x 1024
    //   1536   6.15 /  6.06   6.37 /  6.42   5.98 /  5.76   6.62 /  6.71
    //   1792   6.65 /  6.53   6.91 /  6.91   6.39 /  6.03   7.03 /  7.11
    //   2048   7.31 /  6.95   7.45 /  7.29   6.88 /  6.47   7.50 /  7.38
    //   8192  17.95 / 14.83  17.54 / 15.29  17.94 / 14.64  17.54 / 15.48
    //   2064   8.33 /  8.43   8.55 /  8.79   7.23 /  6.87   8.81 /  9.10
    //   4112  12.86 / 12.85  13.06 / 13.21  12.36 / 12.32  13.13 / 13.55
    //   6208  14.88 / 15.04  14.90 / 15.57  14.94 / 14.60  14.96 / 15.85
    //   8208  21.76 / 21.03  21.92 / 21.78  21.04 / 20.57  22.01 / 22.24
    //  16400  38.31 / 36.41  39.42 / 37.43  37.36 / 34.88  39.33 / 38.63
    if (K < (K % kStepK == 0 ? 2048 : 8192)) return launch_tiles<64, 64, 5, 1, false>(p, bf16, (M + 63) / 64, stream);
    return launch_tiles<64, 64, 3, 2, false>(p, bf16, (M + 63) / 64, stream);
  }
  if (wgs(64, 128) <= kCus) return launch_tiles<64, 128, 3, 1, false>(p, bf16, (M + 63) / 64, stream);
  if (wgs(128, 128) <= kCus) return launch_tiles<128, 128, 3, 1, false>(p, bf16, (M + 127) / 128, stream);
  // Large products: 256 x 256 tiles, one per CU, against 128 x 128, two at a time
  // per CU. In rounds of 256 tiles of the large kind: its last, partly filled
  // round costs about 0.8 of a full one. A round of 512 small tiles costs 0.51 at
  // K = 1024 and more with K (the large tile's loads and LDS reads per MFMA are
  // half as many), its last one at least half. us, 256 x 256 / 128 x 128, MI355X:
  //   4096 x 4096 x 4096 55.8 / 61.1    8192 x 8192 x 8192 378 / 472
  //   8192 x 7168 x 2048  125 / 116     2500 x 7168 x 7168 152 / 118
  //   6000 x 4096 x 4096  102 / 88.7    4500 x 4096 x 4096 95.5 / 73.6
  // (Workgroups that stay and take tile after tile, the next tile's copies begun
  // under the last one's output, were 2-15% slower: the CUs write their outputs
  // at the same time either way, and the loop with the next tile's lookup in it
  // spills registers.)
  const double r256 = (double)wgs(256, 256) / kCus, r128 = (double)wgs(128, 128) / (2 * kCus);
  const double part256 = r256 - (int64_t)r256, part128 = r128 - (int64_t)r128;
  const double cost256 = (int64_t)r256 + (part256 > 0 ? 0.8 : 0);
  const double cost128 = ((int64_t)r128 + (part128 > 0.5 ? part128 : part128 > 0 ? 0.5 : 0)) * (0.5 + 0.011 * K / 1024);
  if (cost128 < cost256) return launch_tiles<128, 128, 2, 1, false>(p, bf16, (M + 127) / 128, stream);
  return launch_tiles<256, 256, 2, 1, false>(p, bf16, (M + 255) / 256, stream);
}

hipError_t launch_int8_gemm_grouped(const int8_t* a, const float* sa, const int8_t* b,
                                    const float* sb, void* c, bool bf16, const int32_t* m_offsets,
                                    int64_t G, int64_t M_total, int64_t N, int64_t K,
                                    hipStream_t stream) {
  const I8Args p{(const uint8_t*)a, sa, (const uint8_t*)b, sb, c, m_offsets, (int)M_total, (int)N, (int)K, (int)G};
  // Rows per expert decide (M_total bounds them: the offsets stay on the GPU).
  // us with 256 x 256 / 128 x 128 tiles, MI355X: 32 experts x 384 rows x 4096 x
  // 2048 140 / 146, 8 x 512 x 4096 x 4096 59 / 81, 8 x 2048 x 4096 x 2048 139 /
  // 186; but with one block of 128 rows each, half of a 256-row tile, 32 x 128 x
  // 4096 x 7168 206 / 200 and 256 x 128 x 2048 x 2048 300 / 272. Where even 64 x
  // 128 tiles leave CUs free they are used: 8 x 128 x 2048 x 2048 11.5 (128 x
  // 128: 14.5).
  const int64_t m128 = M_total / 128;
  if (2 * m128 * ((N + 127) / 128) <= kCus) return launch_tiles<64, 128, 3, 1, true>(p, bf16, 2 * m128, stream);
  if (M_total < 256 * G) return launch_tiles<128, 128, 2, 1, true>(p, bf16, m128, stream);
  // upper bound on sum_e ceil(rows_e / 256) for rows_e multiples of 128
  return launch_tiles<256, 256, 2, 1, true>(p, bf16, (m128 + G + 1) / 2, stream);
}

}  // namespace fp8q
