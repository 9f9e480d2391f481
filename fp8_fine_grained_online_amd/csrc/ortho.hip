// Newton-Schulz orthogonalization of weight gradients' updates, for gfx950.
//
//   X_0 = G / |G| (Frobenius),  A = X X^T,  B = b A + c A^2,  X <- a X + B X
//
// run `steps` times over m x n matrices, m <= n (a tall G is transposed on the way
// in and out), as three matrix products a step on the FP16 matrix cores:
//
//   gram    A = X X^T         symmetric: tiles on and below the diagonal only
//   square  B = b A + c A A   symmetric, and A A = A A^T
//   update  X = a X + B X     the columns of X are the rows of X^T, kept beside it
//
// so that every operand is read along its rows. The products' epilogues do the
// rest: a tile goes out in both orientations where both are read next.
//
// Numbers. X, A and B are kept as FP16 times a power of two that puts their
// entries in FP16's normal range (the singular values of X stay below 3, checked
// on the host). Each is the sum of two such numbers, high and low (kSplit): 22 bits,
// and a product is high high + high low + low high in one binary32 accumulator:
// the result is as near the definition as one formed in binary32 (2e-6 to 4e-5,
// growing with the spread of the singular values), whatever its own type.
//
// Where the caller asks for it, a bfloat16 result comes from the high parts' product
// alone (X keeps its low part, and the term a X loses nothing that matters): a third of
// the MFMAs. It is off by 7e-4 to 2e-3, where values vary, and by up to 1e-2 where they
// share a few magnitudes (a constant matrix, the identity, equal blocks), whose roundings
// go the same way and add up; no form of one FP16 number a value is nearer there. Two
// precautions against such errors of the diagonal:
//
//  * what FP16 cuts off the diagonals of A and B is kept in binary32 vectors and
//    put back in the next epilogue (D A + A D in the square, D X in the update);
//  * in the last two steps, where all singular values are near 1 and b A + c A A
//    would cancel most of a, A is taken about its mean eigenvalue alpha = |X|^2 / m:
//    with A = alpha I + A',  B' = (b + 2 c alpha) A' + c A' A'  and
//    X <- (a + b alpha + c alpha^2) X + B' X. Exact for any alpha. (In earlier steps
//    most eigenvalues are near 0, not near their mean, and the rounding of X in B' X
//    would cost more than it saves.)
//
// Zero rows and columns pad m and n to multiples of 64; they stay zero.
#include <type_traits>

#include "common.hpp"
#include "rows.hpp"
#include "tiles.hpp"
#include "wave.hpp"

namespace fp8q {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr float kScaleX = 8192.0f, kScaleA = 4096.0f;  // X, and A and B, as they are stored
constexpr int kPad = 64;                               // rows and columns are padded to
constexpr int kOrthoStep = 128;                        // bytes of K per pipeline step: 64 values
constexpr int kNormParts = 512;                        // partial sums of |G|^2 per matrix

// Where value (row, col) of a plane lies: blocks of 16 rows x 32 values, the operand of one
// MFMA, one after the other along the rows; in a block, eight values of each of its 16 rows at a time.
// A fragment is 1 KB in one piece whatever the pitch, where rows of 2^k bytes would all
// come from the same few channels of the L2.
__device__ __forceinline__ int64_t plane_at(int row, int col, int ld) {
  return (int64_t)(row >> 4) * 16 * ld + (col >> 5) * 512 + ((col >> 3) & 3) * 128 + (row & 15) * 8 + (col & 7);
}

enum class Product { kGram, kSquare, kUpdate };

struct OrthoArgs {
  // planes of all matrices, one after the other; *_lo: low parts (of A, B and X^T for kSplit only)
  _Float16 *x, *x_lo;          // m x n
  const _Float16 *xt, *xt_lo;  // n x m, as read
  _Float16 *xt_new, *xt_lo_new;
  _Float16 *am, *am_lo, *bm, *bm_lo;  // m x m
  float *da, *db;                     // what FP16 cut off their diagonals, m
  float* alpha;                       // one per matrix
  float* squares;                     // sums of X^2, parts per matrix; written by the update, read by the gram
  void* out;                          // the result, from the last step
  int m, n, m_true, n_true;           // padded and true sizes
  int parts;
  int count;    // tiles per matrix
  int splits;   // runs of K that a gram's blocks are formed in
  v4f* partial;  // their sums, of a block one after the other
  float a, b, c, scale;
  int pivot;    // this step takes A about its mean eigenvalue
  int low_in, low_out;  // X's low part is there, and is kept
  int tall;     // the result is transposed
};

template <int BM, int BN, int D, bool kSplit>
struct OrthoTile {
  static constexpr int kWM = BM / 2, kWN = BN / 2;
  static constexpr int kSlabA = BM * kOrthoStep, kSlabB = BN * kOrthoStep;
  static constexpr int kRing = (D + 1) * kSlabA + D * kSlabB;
  // a wave's staging of its part on the way out: 16 rows (16-byte chunk c of row r at
  // c ^ r), and all of it transposed (rows a chunk apart)
  static constexpr int kPitchR = kWN * 2, kPitchC = kWM * 2 + 16;
  static constexpr int kStageR = 16 * kPitchR, kStageC = kWN * kPitchC;
  static constexpr int kStage = 4 * (kStageR + (kSplit ? 2 : 1) * kStageC);
  static constexpr int kLds = kRing > kStage ? kRing : kStage;
  static constexpr int kLoadsA = BM * 8 / 256, kLoadsB = BN * 8 / 256;
  static_assert(kWM % 16 == 0 && kWN % 16 == 0, "whole MFMA blocks");
  static_assert(BM * 8 % 256 == 0 && BN * 8 % 256 == 0, "whole copies");
  static_assert(kLds <= 160 * 1024 && D >= 2, "LDS");
  static_assert((D - 1) * (kLoadsA + kLoadsB) <= 63, "the wait counter holds the copies in flight");
};

constexpr int ortho_wait_vm(int n) { return 0x0F70 | (n & 15) | ((n >> 4) << 14); }
constexpr int kOrthoWaitLds = 0xC07F;

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
}

// Where chunk c of a staged row r lies, of n: another place in each of the rows that
// are written at once, also where n is no power of two
__device__ __forceinline__ int swz_chunk(int r, int c, int n) { return (n & (n - 1)) ? (c + r) % n : c ^ (r & (n - 1)); }

enum class Result { kPlanes, kBf16, kF32 };

// One value of a product's result, scaled as it is stored: from the product, and what
// the result's place held before (high and low part of X or A; the diagonal's cuts of its
// row and column).
template <Product kWhat, bool kSplit>
__device__ __forceinline__ float ortho_value(const OrthoArgs& p, float acc, float hi, float lo, float cut_m, float cut_n,
                                             bool diagonal, float alpha) {
  if constexpr (kWhat == Product::kGram) {
    const float v = acc * (kScaleA / (kScaleX * kScaleX));
    return diagonal ? v - kScaleA * alpha : v;
  } else if constexpr (kWhat == Product::kSquare) {
    const float whole = hi + (kSplit ? lo : diagonal ? cut_m : 0.0f);
    const float sq = __builtin_fmaf(kSplit ? 0.0f : cut_m + cut_n, hi, acc) * (1.0f / kScaleA);
    return __builtin_fmaf(p.c, sq, (p.b + 2.0f * p.c * alpha) * whole);
  } else {
    const float q = p.a + alpha * (p.b + alpha * p.c) + cut_m * (1.0f / kScaleA);
    return __builtin_fmaf(q, hi + lo, acc * (1.0f / kScaleA));
  }
}

// t-th of the tiles on and below the diagonal, row by row
__device__ __forceinline__ void triangle_tile(int t, int& tm, int& tn) {
  tm = (int)((__builtin_sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
  while (tm * (tm + 1) / 2 > t) --tm;
  while ((tm + 1) * (tm + 2) / 2 <= t) ++tm;
  tn = t - tm * (tm + 1) / 2;
}

// Operands and result of a product for matrix `mat`: rows m0.. of a, rows n0.. of b, K values each
struct OrthoOperands {
  const _Float16 *a_hi, *a_lo, *b_hi, *b_lo;
  int K, rows;  // `rows`: of b
  int64_t mm, mn;
};
template <Product kWhat>
__device__ __forceinline__ OrthoOperands ortho_operands(const OrthoArgs& p, int64_t mat) {
  OrthoOperands o;
  o.mm = mat * p.m * p.m, o.mn = mat * (int64_t)p.m * p.n;
  if constexpr (kWhat == Product::kGram) o.a_hi = o.b_hi = p.x + o.mn, o.a_lo = o.b_lo = p.x_lo + o.mn, o.K = p.n, o.rows = p.m;
  if constexpr (kWhat == Product::kSquare) o.a_hi = o.b_hi = p.am + o.mm, o.a_lo = o.b_lo = p.am_lo + o.mm, o.K = p.m, o.rows = p.m;
  if constexpr (kWhat == Product::kUpdate)
    o.a_hi = p.bm + o.mm, o.a_lo = p.bm_lo + o.mm, o.b_hi = p.xt + o.mn, o.b_lo = p.xt_lo + o.mn, o.K = p.m, o.rows = p.n;
  return o;
}

// Where a result goes: rows of it, and columns (transposed); NULL for neither
struct OrthoPlaces {
  uint16_t *r, *r_lo, *c, *c_lo;
  int64_t ld_r, ld_c;
  int end_m, end_n;
};
template <Product kWhat, Result kOut>
__device__ __forceinline__ OrthoPlaces ortho_places(const OrthoArgs& p, const OrthoOperands& o, int64_t mat, bool on_diagonal) {
  OrthoPlaces w{nullptr, nullptr, nullptr, nullptr, 0, 0, p.m, o.rows};
  if constexpr (kWhat != Product::kUpdate) {
    w.r = (uint16_t*)((kWhat == Product::kGram ? p.am : p.bm) + o.mm);
    w.r_lo = (uint16_t*)((kWhat == Product::kGram ? p.am_lo : p.bm_lo) + o.mm);
    if (!on_diagonal) w.c = w.r, w.c_lo = w.r_lo;
    w.ld_r = w.ld_c = p.m;
  } else if constexpr (kOut == Result::kPlanes) {
    w.r = (uint16_t*)(p.x + o.mn), w.r_lo = (uint16_t*)(p.x_lo + o.mn);
    w.c = (uint16_t*)(p.xt_new + o.mn), w.c_lo = (uint16_t*)(p.xt_lo_new + o.mn);
    w.ld_r = p.n, w.ld_c = p.m;
  } else {
    w.end_m = p.m_true, w.end_n = p.n_true;
    if constexpr (kOut == Result::kBf16) (p.tall ? w.c : w.r) = (uint16_t*)p.out + mat * (int64_t)p.m_true * p.n_true;
    w.ld_r = p.n_true, w.ld_c = p.m_true;
  }
  return w;
}

// alpha = |X|^2 / m from the last update's partial sums, by a whole workgroup
__device__ __forceinline__ float ortho_alpha(const OrthoArgs& p, int64_t mat, float* sums, int threads) {
  float s = 0.0f;
  for (int i = threadIdx.x; i < p.parts; i += threads) s += p.squares[mat * p.parts + i];
  s = wave_sum_f32(s);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = s;
  __syncthreads();
  s = sums[0];
  for (int w = 1; w < threads / 64; ++w) s += sums[w];
  __syncthreads();
  return s / (float)p.m_true;
}

// Neighbouring lanes (l ^ 1) hold four columns of neighbouring rows, packed in two
// numbers of two: the even lane gets both rows' first two columns, the odd one the
// others, each as a pair along the column.
struct Turned {
  uint32_t first, second;  // of columns 2 odd, 2 odd + 1
};
__device__ __forceinline__ Turned turn_pairs(bool odd, uint32_t p0, uint32_t p1) {
  const uint32_t own = odd ? p1 : p0, got = dpp_u32<0xB1>(odd ? p0 : p1);
  // bytes 0 to 3 are own's, 4 to 7 got's; the even lane's row comes first
  return {__builtin_amdgcn_perm(got, own, odd ? 0x01000504u : 0x05040100u), __builtin_amdgcn_perm(got, own, odd ? 0x03020706u : 0x07060302u)};
}

// ---------------------------------------------------------------------------
// One tile of one product. Four wavefronts, each a quarter of the tile; per step
// of 64 values of K the slabs of both operands go straight from global memory to
// LDS as they lie there, fragment by fragment, and each step is
// multiplied in two halves, the one's operands read from LDS while the other
// multiplies; A's slabs rotate through D + 1 buffers, B's through D. Lane l
// supplies row l % 16 of a 16-row block and 8 values of K at 8 (l / 16); B is the
// first operand, so a lane holds C[l % 16][4 (l / 16) + r].
// Its own chain bounds it: of 4096 x 4096 the MFMAs are busy 54% of the gram's time (273 us) and the
// square's (277) and 61% of the update's (381), in 128 x 128 tiles that copy six slabs per 64 values of K where
// four hold both parts of both operands; with one number a value 64% (70), 60% (74) and 56% (133), the rest being
// a tile's first copies and the epilogue's bursts (X, its low part and X^T, 101 MB), which nothing hides.
// ---------------------------------------------------------------------------
template <Product kWhat, Result kOut, bool kSplit, int BM, int BN, int D>
__global__ __launch_bounds__(256, 1) void ortho_product_kernel(OrthoArgs p) {
  using Cfg = OrthoTile<BM, BN, D, kSplit>;
  constexpr int WM = Cfg::kWM, WN = Cfg::kWN, SUBM = WM / 16, SUBN = WN / 16, kMfmas = SUBM * SUBN;
  constexpr bool kSymmetric = kWhat != Product::kUpdate;
  __shared__ __attribute__((aligned(16))) uint8_t lds[Cfg::kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int lr = lane & 15, lk = lane >> 4;

  // tiles of all matrices in one run, shared out to the XCDs
  const int task = xcd_tile(blockIdx.x, gridDim.x);
  const int64_t mat = task / p.count;
  const int t = task % p.count;
  int tm, tn;
  if constexpr (kSymmetric) {
    static_assert(!kSymmetric || BM == BN, "square tiles");
    triangle_tile(t, tm, tn);
  } else {
    band_tile(t, (p.m + BM - 1) / BM, (p.n + BN - 1) / BN, tm, tn);
  }
  const int m0 = tm * BM, n0 = tn * BN;
  const OrthoOperands o = ortho_operands<kWhat>(p, mat);
  const int64_t mm = o.mm, mn = o.mn;
  const _Float16 *const a_hi = o.a_hi, *const a_lo = o.a_lo, *const b_hi = o.b_hi, *const b_lo = o.b_lo;
  const int K = o.K, rows_total = o.rows;
  const int pitch = K * 2;  // bytes
  const uint32_t bytes_a = (uint32_t)min(BM, p.m - m0) * (uint32_t)pitch;
  const uint32_t bytes_b = (uint32_t)min(BN, rows_total - n0) * (uint32_t)pitch;
  const int64_t at_a = (int64_t)m0 * K, at_b = (int64_t)n0 * K;
  const int ksteps = pitch / kOrthoStep;
  const int steps = kSplit ? 3 * ksteps : ksteps;
  auto rsrc_a = [&](int seg, bool any = true) { return make_rsrc((kSplit && seg == 2 ? a_lo : a_hi) + at_a, any ? bytes_a : 0u); };
  auto rsrc_b = [&](int seg, bool any = true) { return make_rsrc((kSplit && seg == 1 ? b_lo : b_hi) + at_b, any ? bytes_b : 0u); };

  // copy q of wavefront w brings fragment 4 q + w of the slab: half w % 2 of row block 2 q + w / 2
  const uint32_t first = (uint32_t)(wave >> 1) * 16 * (uint32_t)pitch + (wave & 1) * 1024 + lane * 16;
  constexpr int kRows = Cfg::kLoadsA > Cfg::kLoadsB ? Cfg::kLoadsA : Cfg::kLoadsB;
  uint32_t off[kRows];
#pragma unroll
  for (int q = 0; q < kRows; ++q) off[q] = first + (uint32_t)(q * 32) * (uint32_t)pitch;
  auto copy_a = [&](int q, __amdgpu_buffer_rsrc_t r, int k, uint8_t* __restrict__ to) {
    load_lds(r, to + (q * 256 + wave * 64) * 16, 16, off[q], k);
  };
  auto copy_b = copy_a;

  v4f acc[SUBM][SUBN];
#pragma unroll
  for (int i = 0; i < SUBM; ++i)
#pragma unroll
    for (int j = 0; j < SUBN; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  f16x8 ra[2][SUBM], rb[2][SUBN];
  const int a_off = wm * WM * kOrthoStep + lane * 16, b_off = wn * WN * kOrthoStep + lane * 16;
  auto read_operand = [&](int u, int h, const uint8_t* __restrict__ sa, const uint8_t* __restrict__ sb) {
    if (u < SUBN) rb[h][u] = *(const f16x8*)(sb + b_off + u * 2048 + h * 1024);
    else ra[h][u - SUBN] = *(const f16x8*)(sa + a_off + (u - SUBN) * 2048 + h * 1024);
  };
  constexpr int kEvery = kMfmas >= 2 * (SUBM + SUBN) ? 2 : 1;
  // Half h of a step: its MFMAs, and between them the other half's operands from (sa, sb)
  // and one operand's copies. Scheduling barriers keep that order.
  auto half = [&](int h, const uint8_t* __restrict__ sa, const uint8_t* __restrict__ sb, __amdgpu_buffer_rsrc_t r, int k,
                  uint8_t* __restrict__ to, bool copy_is_a) {
#pragma unroll
    for (int u = 0; u < kMfmas; ++u) {
      const int i = u / SUBN, j = u % SUBN;
      if (u % kEvery == 0 && u / kEvery < SUBM + SUBN) read_operand(u / kEvery, 1 - h, sa, sb);
      if (u % kEvery == kEvery - 1) {
        const int q = u / kEvery;
        if (copy_is_a) { if (q < Cfg::kLoadsA) copy_a(q, r, k, to); }
        else { if (q < Cfg::kLoadsB) copy_b(q, r, k, to); }
      }
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(rb[h][j], ra[h][i], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  static_assert(kMfmas / kEvery >= SUBM + SUBN && kMfmas / kEvery >= kRows, "reads and copies fit between the MFMAs");

  // step g: byte of K and, for kSplit, which parts are multiplied
  auto seg_of = [&](int g) { return !kSplit || g < ksteps ? 0 : g < 2 * ksteps ? 1 : 2; };
  auto k_of = [&](int g) { return (g - seg_of(g) * ksteps) * (16 * kOrthoStep); };
  uint8_t* const lds_b = lds + (D + 1) * Cfg::kSlabA;
#pragma unroll
  for (int d = 0; d < D; ++d) {
    const int g = min(d, steps - 1);
#pragma unroll
    for (int q = 0; q < Cfg::kLoadsA; ++q) copy_a(q, rsrc_a(seg_of(g)), k_of(g), lds + d * Cfg::kSlabA);
#pragma unroll
    for (int q = 0; q < Cfg::kLoadsB; ++q) copy_b(q, rsrc_b(seg_of(g)), k_of(g), lds_b + d * Cfg::kSlabB);
  }
  __builtin_amdgcn_s_waitcnt(ortho_wait_vm((D - 1) * (Cfg::kLoadsA + Cfg::kLoadsB)));
  __builtin_amdgcn_s_barrier();
#pragma unroll
  for (int u = 0; u < SUBM + SUBN; ++u) read_operand(u, 0, lds, lds_b);
  int a0 = 0, a1 = Cfg::kSlabA, a2 = D * Cfg::kSlabA;
  int b0 = 0, b1 = Cfg::kSlabB;
  const int mw = m0 + wm * WM, nw = n0 + wn * WN;  // this wave's part
  // What the epilogue reads of row block i: the tile's values of X or A, and what
  // FP16 cut off the diagonal there. Loaded a row block ahead of its use, the first under
  // the last step's products.
  struct Before {
    f16x4 hi[SUBN], lo[SUBN];
    float cut;
  };
  constexpr bool kLowBefore = kWhat == Product::kUpdate || (kWhat == Product::kSquare && kSplit);
  auto read_before = [&](int i, Before& f) {
    if constexpr (kWhat == Product::kGram) {
      f = Before{};
      return;
    }
    const int gm = mw + i * 16 + lr;
    f.cut = !kSplit && gm < p.m ? (kWhat == Product::kSquare ? p.da : p.db)[mat * p.m + gm] : 0.0f;
    const _Float16* const hi = (kWhat == Product::kSquare ? p.am + mm : p.x + mn);
    const _Float16* const lo = (kWhat == Product::kSquare ? p.am_lo + mm : p.x_lo + mn);
#pragma unroll
    for (int j = 0; j < SUBN; ++j) {
      const bool inside = gm < p.m && nw + j * 16 + 4 * lk < rows_total;
      const f16x4 none = {0, 0, 0, 0};
      const int64_t at = plane_at(gm, nw + j * 16 + 4 * lk, rows_total);
      f.hi[j] = inside ? *(const f16x4*)(hi + at) : none;
      f.lo[j] = kLowBefore && inside && (kSplit || p.low_in) ? *(const f16x4*)(lo + at) : none;
    }
  };
  constexpr bool kCutN = kWhat == Product::kSquare && !kSplit;
  float cut_n[kCutN ? SUBN : 1][4] = {};  // of the columns' diagonals
  if constexpr (kCutN) {
#pragma unroll
    for (int j = 0; j < SUBN; ++j) {
      const int gn = nw + j * 16 + 4 * lk;
      const v4f d = gn < p.m ? *(const v4f*)(p.da + mat * p.m + gn) : v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int r = 0; r < 4; ++r) cut_n[j][r] = d[r];
    }
  }
  Before before[2];
  for (int g = 0; g < steps; ++g) {
    // past the end the copies read nothing: an empty descriptor gives zeros, unread
    const bool more = g + D < steps;
    const int gn = more ? g + D : 0, seg = seg_of(gn), kn = k_of(gn);
    half(0, lds + a0, lds_b + b0, rsrc_a(seg, more), kn, lds + a2, true);
    // this wave has read all of step g, and its copies of step g + 1 have landed
    __builtin_amdgcn_s_waitcnt(kOrthoWaitLds);
    __builtin_amdgcn_s_waitcnt(ortho_wait_vm((D - 1) * Cfg::kLoadsA + (D - 2) * Cfg::kLoadsB));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (!kSplit && g == steps - 1) read_before(0, before[0]);
    half(1, lds + a1, lds_b + b1, rsrc_b(seg, more), kn, lds_b + b0, false);
    a2 = a0, a0 = a1, b0 = b1;
    a1 = a1 == D * Cfg::kSlabA ? 0 : a1 + Cfg::kSlabA;
    b1 = b1 == (D - 1) * Cfg::kSlabB ? 0 : b1 + Cfg::kSlabB;
  }
  if constexpr (kSplit) read_before(0, before[0]);  // (three times as many steps: its loop is the faster without)
  // the last copies may still be writing the LDS that is used again below
  __builtin_amdgcn_s_waitcnt(ortho_wait_vm(0));
  __syncthreads();

  // ---- the tile's values ----
  const bool on_diagonal = kSymmetric && tm == tn;
  float alpha = 0.0f;
  if (kWhat == Product::kGram && p.pivot && on_diagonal) {
    alpha = ortho_alpha(p, mat, (float*)lds, 256);
    if (t == 0 && tid == 0) p.alpha[mat] = alpha;
  }
  if (kWhat != Product::kGram && p.pivot) alpha = p.alpha[mat];

  constexpr int kPitchR = Cfg::kPitchR, kPitchC = Cfg::kPitchC;
  uint8_t* const st_r = lds + wave * (Cfg::kStage / 4);
  uint8_t* const st_c = st_r + Cfg::kStageR;
  uint8_t* const st_c_lo = st_c + Cfg::kStageC;  // kSplit
  // `kR` rows of `kC` 16-bit values from the wave's LDS to `to` (ld apart), up to the ends of its rows and columns
  auto flush = [&](auto r_c, auto c_c, const uint8_t* st, uint16_t* to, int64_t ld, int row, int col, int row_end,
                   int col_end) {
    constexpr int kR = decltype(r_c)::value, kCh = decltype(c_c)::value / 8;
    constexpr bool kSwizzled = kR == 16;
    constexpr int kPitch = kCh * 16 + (kSwizzled ? 0 : 16);
    static_assert(kR * kCh % 64 == 0, "whole wave stores");
    __builtin_amdgcn_s_waitcnt(kOrthoWaitLds);  // a wave reads back only its own part
    __builtin_amdgcn_wave_barrier();
#pragma unroll 4
    for (int k = 0; k < kR * kCh / 64; ++k) {
      // (planes: 16 rows of a chunk are one piece)
      const int u = k * 64 + lane;
      const int r = kOut == Result::kPlanes ? u / (16 * kCh) * 16 + u % 16 : u / kCh, ch = kOut == Result::kPlanes ? u / 16 % kCh : u % kCh;
      const u32x4 v = *(const u32x4*)(st + r * kPitch + (kSwizzled ? swz_chunk(r, ch, kCh) : ch) * 16);
      if (row + r < row_end && col + ch * 8 < col_end) {
        if constexpr (kOut == Result::kPlanes) *(u32x4*)(to + plane_at(row + r, col + ch * 8, (int)ld)) = v;  // padded to whole chunks
        else store_chunk((bf16_t*)(to + (row + r) * ld + col + ch * 8), {v}, col_end - col - ch * 8);
      }
    }
    __builtin_amdgcn_wave_barrier();
  };
  using std::integral_constant;
  constexpr integral_constant<int, 16> k16{};
  constexpr integral_constant<int, WM> kWMc{};
  constexpr integral_constant<int, WN> kWNc{};
  auto put_row = [&](int j, uint32_t p0, uint32_t p1) {  // block j's four values of this lane's row
    *(uint2*)(st_r + lr * kPitchR + swz_chunk(lr, 2 * j + (lk >> 1), WN / 8) * 16 + (lk & 1) * 8) = make_uint2(p0, p1);
  };
  // transposed: neighbouring lanes hold neighbouring rows; the even one writes the first two columns of both, the odd one the others
  auto put_col = [&](uint8_t* st, int i, int j, uint32_t p0, uint32_t p1) {
    const bool odd = lr & 1;
    const Turned w = turn_pairs(odd, p0, p1);
    uint8_t* const to = st + (j * 16 + 4 * lk + (odd ? 2 : 0)) * kPitchC + (i * 16 + (lr & ~1)) * 2;
    *(uint32_t*)to = w.first;
    *(uint32_t*)(to + kPitchC) = w.second;
  };

  const OrthoPlaces w = ortho_places<kWhat, kOut>(p, o, mat, on_diagonal);
  uint16_t *const to_r = w.r, *const to_r_lo = w.r_lo, *const to_c = w.c, *const to_c_lo = w.c_lo;
  const int64_t ld_r = w.ld_r, ld_c = w.ld_c;
  const int end_m = w.end_m, end_n = w.end_n;
  constexpr bool kLowRows = kSplit || kWhat == Product::kUpdate;  // low parts are kept of X always
  float* const cut = (kWhat == Product::kGram ? p.da : p.db) + mat * p.m;

  float square = 0.0f;
#pragma unroll
  for (int i = 0; i < SUBM; ++i) {
    const int gm = mw + i * 16 + lr;
    const Before& f = before[i % 2];
    if (i + 1 < SUBM) read_before(i + 1, before[(i + 1) % 2]);
    __builtin_amdgcn_sched_barrier(0);
    float val[SUBN][4];
#pragma unroll
    for (int j = 0; j < SUBN; ++j) {
      const int gn = nw + j * 16 + 4 * lk;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        val[j][r] = ortho_value<kWhat, kSplit>(p, acc[i][j][r], (float)f.hi[j][r], (float)f.lo[j][r], f.cut,
                                               cut_n[kCutN ? j : 0][r], kSymmetric && gm == gn + r, alpha);
        if constexpr (kWhat == Product::kUpdate) square = __builtin_fmaf(val[j][r], val[j][r], square);
      }
    }
    if constexpr (!kSplit && kSymmetric) {
      if (on_diagonal && wm == wn && i < SUBN) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (4 * lk + r == lr && gm < p.m) cut[gm] = val[i][r] - (float)(_Float16)val[i][r];
      }
    }
    if constexpr (kOut == Result::kF32) {
      float* const to = (float*)p.out + mat * (int64_t)p.m_true * p.n_true;
#pragma unroll
      for (int j = 0; j < SUBN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int gn = nw + j * 16 + 4 * lk + r;
          if (gm < end_m && gn < end_n)
            to[p.tall ? (int64_t)gn * p.m_true + gm : (int64_t)gm * p.n_true + gn] = val[j][r] * (p.scale * (1.0f / kScaleX));
        }
    } else {
      uint32_t lo[SUBN][2];
#pragma unroll
      for (int j = 0; j < SUBN; ++j) {
        uint32_t hi[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float u = val[j][2 * h], v = val[j][2 * h + 1];
          if constexpr (kOut == Result::kBf16) {
            const float f = p.scale * (1.0f / kScaleX);
            hi[h] = pack_bf16(u * f, v * f);
          } else {
            hi[h] = pack_f16(u, v);
            lo[j][h] = pack_f16(u - (float)(_Float16)u, v - (float)(_Float16)v);
          }
        }
        if (to_r) put_row(j, hi[0], hi[1]);
        if (to_c) {
          put_col(st_c, i, j, hi[0], hi[1]);
          if constexpr (kSplit && kOut == Result::kPlanes) put_col(st_c_lo, i, j, lo[j][0], lo[j][1]);
        }
      }
      if (to_r) flush(k16, kWNc, st_r, to_r, ld_r, mw + i * 16, nw, end_m, end_n);
      if constexpr (kLowRows && kOut == Result::kPlanes) {
        if (kSplit || p.low_out) {
#pragma unroll
          for (int j = 0; j < SUBN; ++j) put_row(j, lo[j][0], lo[j][1]);
          flush(k16, kWNc, st_r, to_r_lo, ld_r, mw + i * 16, nw, end_m, end_n);
        }
      }
    }
    // one row block at a time: with more of their loads ahead the registers do not hold
    __builtin_amdgcn_sched_barrier(0);
  }
  if constexpr (kOut != Result::kF32) {
    if (to_c) {
      flush(kWNc, kWMc, st_c, to_c, ld_c, nw, mw, end_n, end_m);
      if constexpr (kSplit && kOut == Result::kPlanes) flush(kWNc, kWMc, st_c_lo, to_c_lo, ld_c, nw, mw, end_n, end_m);
    }
  }
  if constexpr (kWhat == Product::kUpdate && kOut == Result::kPlanes && !kSplit) {
    square = wave_sum_f32(square) * (1.0f / (kScaleX * kScaleX));
    if (lane == 0) p.squares[mat * p.parts + t * 4 + wave] = square;
  }
}

// Four values of row gm from column gn on, from a lane of a 16 x 16 block's wavefront, to where a product's
// result goes.
template <Product kWhat, Result kOut, bool kSplit>
__device__ __forceinline__ void ortho_put(const OrthoArgs& p, const OrthoOperands& o, int64_t mat, bool on_diagonal, int gm, int gn,
                                          const float (&val)[4]) {
  const float scale = p.scale * (1.0f / kScaleX);
  if constexpr (kOut == Result::kPlanes) {
    const OrthoPlaces to = ortho_places<kWhat, kOut>(p, o, mat, on_diagonal);
    auto put = [&](uint16_t* rows, uint16_t* cols, uint32_t p0, uint32_t p1) {
      if (rows) *(uint2*)(rows + plane_at(gm, gn, (int)to.ld_r)) = make_uint2(p0, p1);
      if (cols) {
        const bool odd = gm & 1;
        const Turned v = turn_pairs(odd, p0, p1);
        uint16_t* const at = cols + plane_at(gn + (odd ? 2 : 0), gm & ~1, (int)to.ld_c);
        *(uint32_t*)at = v.first;
        *(uint32_t*)(at + 8) = v.second;
      }
    };
    auto low = [](float v) { return v - (float)(_Float16)v; };
    put(to.r, to.c, pack_f16(val[0], val[1]), pack_f16(val[2], val[3]));
    if (kSplit || (kWhat == Product::kUpdate && p.low_out))
      put(to.r_lo, kSplit ? to.c_lo : nullptr, pack_f16(low(val[0]), low(val[1])), pack_f16(low(val[2]), low(val[3])));
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (gm >= p.m_true || gn + r >= p.n_true) continue;
      const int64_t at = mat * (int64_t)p.m_true * p.n_true +
                         (p.tall ? (int64_t)(gn + r) * p.m_true + gm : (int64_t)gm * p.n_true + gn + r);
      if constexpr (kOut == Result::kBf16) ((__bf16*)p.out)[at] = (__bf16)(val[r] * scale);
      else ((float*)p.out)[at] = val[r] * scale;
    }
  }
}

// ---------------------------------------------------------------------------
// Small products: a workgroup owns 16 S x 16 S values and its W wavefronts split K
// between them in pieces of 32 values (one MFMA deep), each streaming its fragments
// straight from global memory to registers, kAhead pieces ahead; the partial
// blocks are added through LDS, in the wavefronts' order. What the epilogue reads is
// loaded before the loop. For products whose tiles would leave most CUs without
// work, where a tile's own chain of copies, barriers and short runs of MFMAs is what is
// waited for. A product of 256 x 1024 takes 3.5 to 4.8 us, an empty kernel 2 to 3.
// ---------------------------------------------------------------------------
// kRuns: a block's K is shared out to p.splits workgroups too, whose sums go to p.partial.
template <Product kWhat, Result kOut, bool kSplit, int S, int W, bool kRuns = false>
__global__ __launch_bounds__(64 * W) void ortho_small_kernel(OrthoArgs p) {
  constexpr bool kSymmetric = kWhat != Product::kUpdate;
  static_assert(!kRuns || (kWhat == Product::kGram && kSplit && S == 1), "as they are joined");
  constexpr int kAhead = 2;
  static_assert(S * S <= W, "a wave per block");
  __shared__ __attribute__((aligned(16))) v4f part[W][S * S][64];
  const int lane = threadIdx.x & 63, lr = lane & 15, lk = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int runs = kRuns ? p.splits : 1;
  const int64_t mat = blockIdx.x / runs / p.count;
  const int t = blockIdx.x / runs % p.count;
  int tm, tn;
  if constexpr (kSymmetric) {
    triangle_tile(t, tm, tn);
  } else {
    const int across = p.n / (16 * S);
    tm = t / across, tn = t % across;
  }
  const int m0 = tm * 16 * S, n0 = tn * 16 * S;
  const bool on_diagonal = kSymmetric && tm == tn;
  const OrthoOperands o = ortho_operands<kWhat>(p, mat);
  const int pieces = o.K / 32;
  const int share = blockIdx.x % runs * W + wave, shares = runs * W;
  const int g_begin = pieces * share / shares, g_end = pieces * (share + 1) / shares;
  struct Frags {
    f16x8 a[S], b[S], a_lo[kSplit ? S : 1], b_lo[kSplit ? S : 1];
  };
  const int64_t at_a = (int64_t)m0 * o.K + lane * 8, at_b = (int64_t)n0 * o.K + lane * 8;
  auto load = [&](int g, Frags& f) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int64_t off = (int64_t)i * 16 * o.K + g * 512;
      f.a[i] = *(const f16x8*)(o.a_hi + at_a + off);
      f.b[i] = *(const f16x8*)(o.b_hi + at_b + off);
      if constexpr (kSplit) {
        f.a_lo[i] = *(const f16x8*)(o.a_lo + at_a + off);
        f.b_lo[i] = *(const f16x8*)(o.b_lo + at_b + off);
      }
    }
  };
  v4f acc[S][S];
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int j = 0; j < S; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  auto compute = [&](const Frags& f) {
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int j = 0; j < S; ++j) {
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
        if constexpr (kSplit) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.b_lo[j], f.a[i], acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.b[j], f.a_lo[i], acc[i][j], 0, 0, 0);
        }
      }
  };
  Frags f[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (g_begin + u < g_end) load(g_begin + u, f[u]);

  // wave b finishes block b: what its places held before
  const int bi = wave / S, bj = wave % S;
  const int gm = m0 + bi * 16 + lr, gn = n0 + bj * 16 + 4 * lk;
  const bool finishes = wave < S * S;
  f16x4 hi = {0, 0, 0, 0}, lo = {0, 0, 0, 0};
  float cut_m = 0.0f, alpha = 0.0f;
  v4f cut_n = {0.0f, 0.0f, 0.0f, 0.0f};
  if (finishes) {
    if constexpr (kWhat == Product::kSquare) {
      const int64_t at = o.mm + plane_at(gm, gn, p.m);
      hi = *(const f16x4*)(p.am + at);
      if constexpr (kSplit) lo = *(const f16x4*)(p.am_lo + at);
      else cut_m = p.da[mat * p.m + gm], cut_n = *(const v4f*)(p.da + mat * p.m + gn);
    }
    if constexpr (kWhat == Product::kUpdate) {
      const int64_t at = o.mn + plane_at(gm, gn, p.n);
      hi = *(const f16x4*)(p.x + at);
      if (kSplit || p.low_in) lo = *(const f16x4*)(p.x_lo + at);
      if constexpr (!kSplit) cut_m = p.db[mat * p.m + gm];
    }
    if (kWhat != Product::kGram && p.pivot) alpha = p.alpha[mat];
  }

  for (int g = g_begin; g < g_end; g += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (g + u < g_end) compute(f[u]);
      if (g + u + kAhead < g_end) load(g + u + kAhead, f[u]);
    }
  }
  if (kWhat == Product::kGram && p.pivot && on_diagonal) {
    alpha = ortho_alpha(p, mat, (float*)part, 64 * W);
    if (t == 0 && threadIdx.x == 0) p.alpha[mat] = alpha;
  }
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int j = 0; j < S; ++j) part[wave][i * S + j][lane] = acc[i][j];
  __syncthreads();
  if (!finishes) return;
  v4f sum = part[0][wave][lane];
#pragma unroll
  for (int w = 1; w < W; ++w) sum += part[w][wave][lane];
  if constexpr (kRuns) {
    p.partial[(int64_t)blockIdx.x * 64 + lane] = sum;
    return;
  }

  float val[4], square = 0.0f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    val[r] = ortho_value<kWhat, kSplit>(p, sum[r], (float)hi[r], (float)lo[r], cut_m, cut_n[r], kSymmetric && gm == gn + r, alpha);
    square = __builtin_fmaf(val[r], val[r], square);
  }
  if constexpr (!kSplit && kSymmetric) {
    float* const cut = (kWhat == Product::kGram ? p.da : p.db) + mat * p.m;
    if (on_diagonal && bi == bj) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (4 * lk + r == lr) cut[gm] = val[r] - (float)(_Float16)val[r];
    }
  }
  if constexpr (kWhat == Product::kUpdate && kOut == Result::kPlanes && !kSplit) {
    square = wave_sum_f32(square) * (1.0f / (kScaleX * kScaleX));
    if (lane == 0) p.squares[mat * p.parts + t * (S * S) + wave] = square;
  }
  ortho_put<kWhat, kOut, kSplit>(p, o, mat, on_diagonal, gm, gn, val);
}

// The runs of K of a gram's 16 x 16 blocks, joined in their order; a wavefront per block. (Only kSplit's
// matrices have so few rows.)
__global__ __launch_bounds__(64) void ortho_join_kernel(OrthoArgs p) {
  const int lane = threadIdx.x;
  const int64_t mat = blockIdx.x / p.count;
  int tm, tn;
  triangle_tile(blockIdx.x % p.count, tm, tn);
  const v4f* const from = p.partial + (int64_t)blockIdx.x * p.splits * 64 + lane;
  v4f sum = from[0];
#pragma unroll 4
  for (int z = 1; z < p.splits; ++z) sum += from[z * 64];
  float val[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) val[r] = ortho_value<Product::kGram, true>(p, sum[r], 0.0f, 0.0f, 0.0f, 0.0f, false, 0.0f);
  ortho_put<Product::kGram, Result::kPlanes, true>(p, ortho_operands<Product::kGram>(p, mat), mat, tm == tn, tm * 16 + (lane & 15),
                                                   tn * 16 + 4 * (lane >> 4), val);
}

// ---------------------------------------------------------------------------
// Square and update in one, for few rows: B X = A (b X + c A X), so that a workgroup
// needs no other one's part of B. It owns 16 columns of X, and each of its wavefronts 16
// rows, whose part of A (32 P columns, all of it) it keeps in registers for both products;
// the columns, and between the products W = b X + c A X, go through LDS. That is m^2 n products more
// in place of m^3, but a launch less a step, and either launch takes about 4 us whatever it multiplies.
// W is two FP16 numbers, times 2^9: its singular values |s (b + c s^2)|, and about a mean
// eigenvalue at most |c| alpha s more, stay below a third of what that leaves, 128, for
// every polynomial that passes the checks. (Its rounding to one would not be small beside what
// b A + c A A cancels: 3e-3 for a matrix of rank one.)
// ---------------------------------------------------------------------------
template <Result kOut, bool kSplit, int P>
__global__ __launch_bounds__(128 * P) void ortho_columns_kernel(OrthoArgs p) {
  constexpr int kWaves = 2 * P, kParts = kSplit ? 2 : 1;
  constexpr float kScaleW = 512.0f;
  __shared__ __attribute__((aligned(16))) _Float16 columns[2][2 * P * 512];
  const int lane = threadIdx.x & 63, lr = lane & 15, lk = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t mat = blockIdx.x / p.count;
  const int t = blockIdx.x % p.count;
  const OrthoOperands o = ortho_operands<Product::kUpdate>(p, mat);
  f16x8 a[P], a_lo[kSplit ? P : 1];
#pragma unroll
  for (int g = 0; g < P; ++g) {
    const int64_t at = o.mm + (int64_t)wave * 16 * p.m + g * 512 + lane * 8;
    a[g] = *(const f16x8*)(p.am + at);
    if constexpr (kSplit) a_lo[g] = *(const f16x8*)(p.am_lo + at);
  }
  for (int g = wave; g < kParts * P; g += kWaves) {
    const _Float16* const from = (g < P ? o.b_hi : o.b_lo) + (int64_t)t * 16 * p.m + g % P * 512 + lane * 8;
    *(f16x8*)(columns[0] + g * 512 + lane * 8) = *(const f16x8*)from;
  }
  const int gm = wave * 16 + lr, gn = t * 16 + 4 * lk;
  const int64_t at = o.mn + plane_at(gm, gn, p.n);
  const f16x4 hi = *(const f16x4*)(p.x + at), lo = kSplit || p.low_in ? *(const f16x4*)(p.x_lo + at) : f16x4{0, 0, 0, 0};
  const float cut = kSplit ? 0.0f : p.da[mat * p.m + gm] * (1.0f / kScaleA);
  const float alpha = p.pivot ? p.alpha[mat] : 0.0f;
  __syncthreads();
  auto multiply = [&](const _Float16* v, auto low) {
    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int g = 0; g < P; ++g) {
      const f16x8 b = *(const f16x8*)(v + g * 512 + lane * 8);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, a[g], acc, 0, 0, 0);
      if constexpr (decltype(low)::value)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(*(const f16x8*)(v + (P + g) * 512 + lane * 8), a[g], acc, 0, 0, 0);
      if constexpr (kSplit) acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, a_lo[g], acc, 0, 0, 0);
    }
    return acc;
  };
  v4f acc = multiply(columns[0], std::bool_constant<kSplit>{});
  float w[4];  // as stored
  f16x4 h, l;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float x = (float)hi[r] + (float)lo[r];
    const float y = __builtin_fmaf(cut, x, acc[r] * (1.0f / kScaleA));
    w[r] = __builtin_fmaf(p.c, y, (p.b + 2.0f * p.c * alpha) * x) * (kScaleW / kScaleX);
    h[r] = (_Float16)w[r];
    l[r] = (_Float16)(w[r] - (float)h[r]);
  }
  auto put = [&](_Float16* to, uint2 v) {
    const bool odd = lr & 1;
    const Turned u = turn_pairs(odd, v.x, v.y);
    _Float16* const at = to + plane_at(4 * lk + (odd ? 2 : 0), gm & ~1, 32 * P);
    *(uint32_t*)at = u.first;
    *(uint32_t*)(at + 8) = u.second;
  };
  put(columns[1], __builtin_bit_cast(uint2, h));
  put(columns[1] + P * 512, __builtin_bit_cast(uint2, l));
  __syncthreads();
  acc = multiply(columns[1], std::true_type{});
  const float q = p.a + alpha * (p.b + alpha * p.c);
  float val[4], square = 0.0f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float z = __builtin_fmaf(cut, w[r], acc[r] * (1.0f / kScaleA)) * (kScaleX / kScaleW);
    val[r] = __builtin_fmaf(q, (float)hi[r] + (float)lo[r], z);
    square = __builtin_fmaf(val[r], val[r], square);
  }
  ortho_put<Product::kUpdate, kOut, kSplit>(p, o, mat, false, gm, gn, val);
  if constexpr (kOut == Result::kPlanes && !kSplit) {
    square = wave_sum_f32(square) * (1.0f / (kScaleX * kScaleX));
    if (lane == 0) p.squares[mat * p.parts + t * kWaves + wave] = square;
  }
}

// ---------------------------------------------------------------------------
// The way in. Sums of G's squares, kNormParts per matrix, in float64 (no input's
// squares leave its range), then G / |G| to the planes of X and X^T. Bound by memory: 4 x 4096
// x 7168 (float32) 90 us, 5.2 TB/s, and 206 us, 5.7 TB/s.
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(256) void ortho_squares_kernel(const T* __restrict__ g, int64_t size, double* __restrict__ parts) {
  __shared__ double sums[4];
  const int64_t chunks = (size + 7) / 8;
  const T* const from = g + blockIdx.y * size;
  double s = 0.0;
  for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < chunks; c += kNormParts * 256) {
    float v[8];
    values(load_chunk(from + 8 * c, (int)min(size - 8 * c, (int64_t)8)), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = __builtin_fma((double)v[e], (double)v[e], s);
  }
  s = wave_sum_f64(s);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) parts[blockIdx.y * kNormParts + blockIdx.x] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// A 64 x 64 block of G (M x N) to the planes: X takes it as it lies or, where G is
// tall, transposed, and X^T the other way round.
template <typename T, bool kSplit>
__global__ __launch_bounds__(256) void ortho_spread_kernel(const T* __restrict__ g, const double* __restrict__ parts, int M, int N,
                                                           int tiles_n, int tiles, OrthoArgs p) {
  __shared__ float block[64][65];
  const int mat = blockIdx.x / tiles, t = blockIdx.x % tiles;
  const int r0 = t / tiles_n * 64, c0 = t % tiles_n * 64;
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < kNormParts / 64; ++i) sum += parts[mat * kNormParts + i * 64 + (threadIdx.x & 63)];
  sum = wave_sum_f64(sum);
  const double f = sum > 0.0 ? (double)kScaleX / __dsqrt_rn(sum) : sum;  // (a NaN goes on)
  const T* const from = g + (int64_t)mat * M * N;
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const int ch = threadIdx.x % 8, r = pass * 32 + threadIdx.x / 8, have = r0 + r < M ? N - c0 - ch * 8 : 0;
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (have > 0) values(load_chunk(from + (int64_t)(r0 + r) * N + c0 + ch * 8, have), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) block[r][ch * 8 + e] = (float)((double)v[e] * f);  // (0 f is NaN where f is)
  }
  __syncthreads();
  const int64_t base = (int64_t)mat * p.m * p.n;
  // rows of G as they lie: M by N padded; columns: N by M padded
  const int ld_s = p.tall ? p.m : p.n, ld_t = p.tall ? p.n : p.m;
  auto put = [&](_Float16* hi, _Float16* lo, bool low, int64_t at, const float (&v)[8]) {
    f16x8 h, l;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = (_Float16)v[e], l[e] = (_Float16)(v[e] - (float)h[e]);
    *(f16x8*)(hi + at) = h;
    if (low) *(f16x8*)(lo + at) = l;
  };
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    // a wavefront writes 16 rows x 32 values, one piece of a plane
    const int r = pass * 32 + threadIdx.x / 128 * 16 + threadIdx.x % 16, ch = threadIdx.x / 16 % 8;
    float v[8], w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = block[r][ch * 8 + e], w[e] = block[ch * 8 + e][r];
    put(p.tall ? p.xt_new : p.x, p.tall ? p.xt_lo_new : p.x_lo, kSplit || !p.tall, base + plane_at(r0 + r, c0 + ch * 8, ld_s), v);
    put(p.tall ? p.x : p.xt_new, p.tall ? p.x_lo : p.xt_lo_new, kSplit || p.tall, base + plane_at(c0 + r, r0 + ch * 8, ld_t), w);
  }
}

// ---------------------------------------------------------------------------
// A matrix that fits a CU's LDS: one workgroup of 16 wavefronts takes all the steps of
// one matrix, m and n padded to 32. A wavefront keeps its units of X, of 16 S x 16 S values,
// in registers as binary32; LDS holds X's high and low parts in both orientations, and A's
// and then B's over X's rows, which only the gram reads, one unit to a wavefront. (All units of A
// and B: a SIMD has work for four wavefronts at m = 128 either way, and writing one's mirror costs as
// much as forming it.) The products are as for kSplit. One launch in place of two and three a step, which is
// what small matrices wait for.
// A step takes 1.1 us for 16 x 26, 2.9 us for 64 x 64 and 9.2 us for 128 x 128: there a half the
// MFMAs and half the vector operations that form, split and place the values, in turn.
// S = 1 where m is 32, whose A would be a single 32 x 32 unit.
// ---------------------------------------------------------------------------
constexpr int kWholeWaves = 16, kWholeLds = 160 * 1024, kWholeGap = 8;  // gap: after a row, against bank conflicts
constexpr int64_t whole_lds(int64_t m, int64_t n) { return 4 * (m * (n + kWholeGap) + n * (m + kWholeGap)); }

template <typename T, int S>
__global__ __launch_bounds__(64 * kWholeWaves) void ortho_whole_kernel(const T* __restrict__ g, OrthoArgs p, int steps, bool out_bf16) {
  constexpr int kSide = 16 * S, kOwn = S == 1 ? 5 : 2;  // units of X a wavefront has at most
  __shared__ __attribute__((aligned(16))) _Float16 lds[kWholeLds / 2];
  const int lane = threadIdx.x & 63;
  int lr = lane & 15, lk = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = p.m, n = p.n, pitch_r = n + kWholeGap, pitch_c = m + kWholeGap;
  _Float16 *const xr = lds, *const xr_lo = xr + m * pitch_r, *const xc = xr_lo + m * pitch_r, *const xc_lo = xc + n * pitch_c;
  _Float16 *const am = lds, *const am_lo = am + m * pitch_c;
  const int across = n / kSide, units = m / kSide * across;
  const int across_a = m / kSide, am0 = wave / across_a * kSide, an0 = wave % across_a * kSide;
  const bool has_a = wave < across_a * across_a;
  const int64_t base = blockIdx.x * (int64_t)p.m_true * p.n_true;
  // value r of this lane's four of block (i, j) of unit k: its place in X, and in G and the result
  int row0[kOwn], col0[kOwn];  // of this wavefront's units
#pragma unroll
  for (int k = 0; k < kOwn; ++k)
    row0[k] = (wave + k * kWholeWaves) / across * kSide, col0[k] = (wave + k * kWholeWaves) % across * kSide;
  auto row_of = [&](int k, int i) { return row0[k] + i * 16 + lr; };
  auto col_of = [&](int k, int j) { return col0[k] + j * 16 + 4 * lk; };
  const int ld_row = p.tall ? 1 : p.n_true, ld_col = p.tall ? p.m_true : 1;
  auto place = [&](int row, int col) { return (uint32_t)(row * ld_row + col * ld_col); };

  v4f x[kOwn][S][S];
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < kOwn; ++k)
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int j = 0; j < S; ++j) {
        x[k][i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        if (wave + k * kWholeWaves < units)
#pragma unroll
          for (int r = 0; r < 4; ++r) {  // past the matrix: its last row or column, so that no load waits in a branch
            const T* const from = g + base + place(min(row_of(k, i), p.m_true - 1), min(col_of(k, j) + r, p.n_true - 1));
            if constexpr (sizeof(T) == 2) x[k][i][j][r] = __uint_as_float((uint32_t)from->bits << 16);
            else x[k][i][j][r] = *from;
          }
      }
#pragma unroll
  for (int k = 0; k < kOwn; ++k)
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int j = 0; j < S; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (row_of(k, i) >= p.m_true || col_of(k, j) + r >= p.n_true) x[k][i][j][r] = 0.0f;
          sum = __builtin_fma((double)x[k][i][j][r], (double)x[k][i][j][r], sum);
        }
  sum = wave_sum_f64(sum);
  double* const sums = (double*)lds;
  if (lane == 0) sums[wave] = sum;
  __syncthreads();
  sum = 0.0;
#pragma unroll
  for (int w = 0; w < kWholeWaves; ++w) sum += sums[w];
  const double f = sum > 0.0 ? (double)kScaleX / __dsqrt_rn(sum) : sum;  // (a NaN goes on)
#pragma unroll
  for (int k = 0; k < kOwn; ++k)
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int j = 0; j < S; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) x[k][i][j][r] = (float)((double)x[k][i][j][r] * f);

  // four values of a row to the planes of a matrix, and to those of its transpose
  auto put = [&](_Float16* rows, _Float16* rows_lo, int ld_r, auto turned, _Float16* cols, _Float16* cols_lo, int ld_c, int row, int col,
                 const v4f& v) {
    const bool odd = lr & 1;
    auto part = [&](_Float16* to_r, _Float16* to_c, uint32_t p0, uint32_t p1) {
      *(uint2*)(to_r + row * ld_r + col) = make_uint2(p0, p1);
      if constexpr (!decltype(turned)::value) return;
      const Turned w = turn_pairs(odd, p0, p1);
      _Float16* const at = to_c + (col + (odd ? 2 : 0)) * ld_c + (row & ~1);
      *(uint32_t*)at = w.first;
      *(uint32_t*)(at + ld_c) = w.second;
    };
    const f16x4 hi = {(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
    f16x4 lo;
#pragma unroll
    for (int r = 0; r < 4; ++r) lo[r] = (_Float16)__builtin_fmaf((float)hi[r], -1.0f, v[r]);
    const uint2 h = __builtin_bit_cast(uint2, hi), l = __builtin_bit_cast(uint2, lo);
    part(rows, cols, h.x, h.y);
    part(rows_lo, cols_lo, l.x, l.y);
  };
  // acc = rows a0.. of a times rows b0.. of b, K values each
  auto multiply = [&](const _Float16* a, const _Float16* a_lo, const _Float16* b, const _Float16* b_lo, int ld, int a0, int b0, int K,
                      v4f (&acc)[S][S]) {
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int j = 0; j < S; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int at_a = (a0 + lr) * ld + 8 * lk, at_b = (b0 + lr) * ld + 8 * lk;
    for (int k = 0; k < K; k += 32) {
      f16x8 fa[S], fb[S], fa_lo[S], fb_lo[S];
#pragma unroll
      for (int i = 0; i < S; ++i) {
        fa[i] = *(const f16x8*)(a + at_a + i * 16 * ld + k), fa_lo[i] = *(const f16x8*)(a_lo + at_a + i * 16 * ld + k);
        fb[i] = *(const f16x8*)(b + at_b + i * 16 * ld + k), fb_lo[i] = *(const f16x8*)(b_lo + at_b + i * 16 * ld + k);
      }
      auto add = [&](const f16x8 (&u)[S], const f16x8 (&v)[S]) {
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
          for (int j = 0; j < S; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[j], u[i], acc[i][j], 0, 0, 0);
      };
      add(fa, fb), add(fa, fb_lo), add(fa_lo, fb);
    }
  };
  auto put_a = [&](const v4f (&v)[S][S]) {
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int j = 0; j < S; ++j)
        put(am, am_lo, pitch_c, std::false_type{}, am, am_lo, 0, am0 + i * 16 + lr, an0 + j * 16 + 4 * lk, v[i][j]);
  };

  for (int s = 0; s < steps; ++s) {
    if (S > 1) asm volatile("" : "+v"(lr), "+v"(lk));  // the addresses are formed anew each step: all of them would not fit the registers
    __syncthreads();  // X's and B's readers are done
#pragma unroll
    for (int k = 0; k < kOwn; ++k)
      if (wave + k * kWholeWaves < units)
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
          for (int j = 0; j < S; ++j)
            put(xr, xr_lo, pitch_r, std::true_type{}, xc, xc_lo, pitch_c, row_of(k, i), col_of(k, j), x[k][i][j]);
    __syncthreads();
    v4f v[S][S];
    if (has_a) multiply(xr, xr_lo, xr, xr_lo, pitch_r, am0, an0, n, v);
    __syncthreads();
    if (has_a) {
#pragma unroll
      for (int i = 0; i < S; ++i)
#pragma unroll
        for (int j = 0; j < S; ++j) v[i][j] *= kScaleA / (kScaleX * kScaleX);
      put_a(v);
    }
    __syncthreads();
    v4f acc[S][S];
    if (has_a) multiply(am, am_lo, am, am_lo, pitch_c, am0, an0, m, acc);
    __syncthreads();
    if (has_a) {
#pragma unroll
      for (int i = 0; i < S; ++i)
#pragma unroll
        for (int j = 0; j < S; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            v[i][j][r] = ortho_value<Product::kSquare, true>(p, acc[i][j][r], v[i][j][r], 0.0f, 0.0f, 0.0f, false, 0.0f);
      put_a(v);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kOwn; ++k)
      if (wave + k * kWholeWaves < units) {
        multiply(am, am_lo, xc, xc_lo, pitch_c, row0[k], col0[k], m, acc);
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
          for (int j = 0; j < S; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              x[k][i][j][r] = ortho_value<Product::kUpdate, true>(p, acc[i][j][r], x[k][i][j][r], 0.0f, 0.0f, 0.0f, false, 0.0f);
      }
  }
  const float scale = p.scale * (1.0f / kScaleX);
  auto store = [&](auto* out) {
#pragma unroll
    for (int k = 0; k < kOwn; ++k)
      if (wave + k * kWholeWaves < units)
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
          for (int j = 0; j < S; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int row = row_of(k, i), col = col_of(k, j) + r;
              if (row < p.m_true && col < p.n_true)
                (out + base)[place(row, col)] = (std::remove_pointer_t<decltype(out)>)(x[k][i][j][r] * scale);
            }
  };
  if (out_bf16) store((__bf16*)p.out);
  else store((float*)p.out);
}

// ---------------------------------------------------------------------------
struct OrthoPlan {
  int64_t m, n;  // padded
  bool split, in_lds, columns;  // in_lds: one workgroup a matrix; columns: square and update in one
  int tile_sym, tile;  // of the gram and the square, and of the update
  int64_t symmetric, whole, splits;
  int64_t bytes;
};

// The tile of the least estimated time. A kernel takes about 4 us, and per round of
// its tiles (two at a time on a CU for 64 x 64 and 128 x 128, else one) an epilogue
// and, per 64 values of K, what the chip needs to feed the round: the same for few
// workgroups, then growing with the share p of the round that is filled. Fitted to
// kernels of 1024 to 4096 rows; the tile it picks is the fastest of the four, or within 3% of it, in 28 products of 1000 to
// 4500 rows. us on MI355X, one FP16 number a value,
// for 64 / 128 / 192 / 256 tiles:
//   gram    2048 x 2048 23.0 / 19.4 / 32.3 / 50.2    2048 x 7168 75.6 / 55.9 / 84.0 / 141
//           2900 x 2900 58.2 / 40.4 / 44.5 / 68.8    4096 x 4096 154 / 90.2 / 67.6 / 99.5
//   update  1400 x 1400 15.0 / 19.2 / 34.0 / 52.3    2048 x 2048 34.6 / 26.5 / 42.2 / 62.9
//           2900 x 2900 91.6 / 74.5 / 59.3 / 82.3    4096 x 4096 218 / 132 / 144 / 128
template <typename Count>
static int ortho_tile(int64_t L, Count count, int64_t K, bool symmetric, bool split) {
  struct Kind {
    int side, slots;
    double epilogue, least, base, slope;  // us; per 64 of K: max(least, base + slope p)
  };
  static constexpr Kind kinds[] = {{64, 2 * kCus, 3, 0.21, 0.10, 0.32},
                                   {128, 2 * kCus, 7, 0.35, 0.17, 0.83},
                                   {192, kCus, 12, 0.70, 0.45, 0.50},
                                   {256, kCus, 20, 1.10, 0.60, 1.00}};
  const double steps = (double)(split ? 3 * K : K) / 64;
  int best = 64;
  double least = 0;
  for (const Kind& k : kinds) {
    if (split && k.side > 128) break;
    const double rounds = (double)(L * count(k.side)) / k.slots, whole = (double)(int64_t)rounds;
    auto round = [&](double p) {
      const double feed = k.base + k.slope * p;
      return k.epilogue * (symmetric ? 0.4 : 1.0) + steps * (feed > k.least ? feed : k.least);
    };
    const double us = whole * round(1.0) + (rounds > whole ? round(rounds - whole) : 0);
    if (least == 0 || us < least) least = us, best = k.side;
  }
  return best;
}

static OrthoPlan ortho_plan(int64_t L, int64_t M, int64_t N, bool single) {
  OrthoPlan o{};
  const int64_t lo = M < N ? M : N, hi = M < N ? N : M;
  o.m = (lo + 31) / 32 * 32;
  o.n = (hi + 31) / 32 * 32;
  // A matrix to a workgroup, where it fits (then X has at most 68 16 x 16 or 18 32 x 32 units) and unless few
  // matrices are the larger ones. us for five steps against the products' launches, MI355X, L x m x n:
  //   16 x 26 11 / 36    32 x 540 33 / 39    64 x 64 22 / 40    64 x 200 36 / 40    64 x 256 43 / 39    96 x 96 41 / 40
  //   128 x 128 64 / 40    8 x 96 x 96 42 / 46    8 x 128 x 128 64 / 46    16 x 96 x 192 59 / 59    32 x 96 x 192 59 / 86
  //   32 x 128 x 128 64 / 76    256 x 64 x 64 23 / 111    256 x 128 x 128 68 / 240
  o.in_lds = whole_lds(o.m, o.n) <= kWholeLds && (o.m <= 32 || (o.m <= 64 && o.n <= 224) || L >= 24);
  if (o.in_lds) return o;
  o.m = (lo + kPad - 1) / kPad * kPad;
  o.n = (hi + kPad - 1) / kPad * kPad;
  o.split = !single || lo <= 128;  // (few rows: nothing to gain from one number)
  auto side = [&](int64_t v, int64_t t) { return (v + t - 1) / t; };
  auto sym = [&](int64_t t) { return side(o.m, t) * (side(o.m, t) + 1) / 2; };
  auto all = [&](int64_t t) { return side(o.m, t) * side(o.n, t); };
  // Small products, for few blocks of 16 x 16 or 32 x 32; else tiles. us for five steps, MI355X (here and
  // below with one FP16 number a value above 128 rows, unless float32 is named, which stands for two), with
  // the symmetric products in 16 x 16 blocks / 32 x 32 blocks / 64 x 64 tiles:
  //   256 x 1024 float32 68 / 78 / 133    333 x 1000 70 / 72 / 90    512 x 512 68 / 69 / 84    600 x 600 92 / 89 / 104
  //   800 x 800 118 / 109 / 122    1000 x 1000 135 / 120 / 132    1400 x 1400 242 / 186 / 170    1024 x 4096 - / 253 / 225
  //   8 x 256 x 256 88 / 85 / 79
  // and the update:
  //   256 x 1024 float32 71 / 68 / 87    400 x 400 67 / 66 / 75    333 x 1000 75 / 69 / 78    600 x 600 88 / 83 / 88
  //   700 x 700 98 / 90 / 94    800 x 800 134 / 122 / 122    700 x 2000 148 / 124 / 115    1000 x 1000 float32 283 / 239 / 258
  if (L * all(16) <= 2 * kCus) o.tile = 16;
  else if (L * all(32) <= (o.split ? 4 : 2) * kCus) o.tile = 32;
  else o.tile = ortho_tile(L, all, o.m, false, o.split);
  if (L * sym(16) <= 2 * kCus) o.tile_sym = 16;
  else if (L * sym(32) <= kCus || (L * sym(32) <= 9 * kCus / 4 && o.m >= 512 && o.n <= 2 * o.m)) o.tile_sym = 32;
  else o.tile_sym = ortho_tile(L, sym, o.n, true, o.split);
  // Square and update in one where A's rows fit registers, and up to four rounds of columns. us for five steps,
  // in one / apart: 26 x 1645 46 / 60    128 x 700 float32 48 / 59    128 x 16000 184 / 192    200 x 333 51 / 59
  //   256 x 256 float32 61 / 61    256 x 1024 56 / 62    256 x 1024 float32 68 / 66    256 x 4096 float32 104 / 114
  //   16 x 256 x 1024 136 / 140    333 x 1000 (with two row blocks to a wavefront) 71 / 68
  o.columns = L * o.n <= 16 * 4 * kCus && (o.m <= 192 || (o.m == 256 && (!o.split || o.n >= 2048)));
  o.symmetric = sym(o.tile_sym);
  // A workgroup reads the 32 rows of its block of the gram at about 90 GB/s: from 8192 values of K on (in both parts),
  // where most CUs would have none, runs of K of 16 pieces at least and another launch. us for five steps, with /
  // without: 16 x 8192 60 / 87    100 x 4096 float32 66 / 77    128 x 16000 132 / 186    128 x 2000 (4096) 61 / 58
  //   4 x 128 x 16000 (144 blocks) 330 / 321    256 x 4096 float32 (136) 115 / 104
  o.splits = 1;
  if (o.split && o.tile_sym == 16 && L * o.symmetric <= kCus / 4 && 2 * o.n >= 8192) {
    o.splits = 2 * kCus / (L * o.symmetric);
    if (o.splits > o.n / 512) o.splits = o.n / 512;
    if (o.splits > 16) o.splits = 16;
  }
  o.whole = o.columns ? o.n / 16 : all(o.tile);
  const int64_t mn = L * o.m * o.n * 2, mm = L * o.m * o.m * 2;
  o.bytes = mn * (o.split ? 6 : 4) + mm * (o.split ? 2 : 1) * (o.columns ? 1 : 2);
  o.bytes += L * (kNormParts * 8 + 2 * o.m * 4 + o.whole * (o.columns ? 64 : 16) + 16);
  if (o.splits > 1) o.bytes += L * o.symmetric * o.splits * 1024;
  return o;
}

int64_t ortho_workspace_bytes(int64_t L, int64_t M, int64_t N, bool single) { return ortho_plan(L, M, N, single).bytes; }

template <Product kWhat, Result kOut, bool kSplit>
static void launch_product(const OrthoArgs& a, int64_t L, int tile, hipStream_t stream) {
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)(L * a.count)), dim3(256), 0, stream, a); };
  auto small = [&](auto kernel, int runs) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(L * a.count * runs)), dim3(512), 0, stream, a);
  };
  if constexpr (kWhat == Product::kGram && kSplit)
    if (a.splits > 1) return small(ortho_small_kernel<kWhat, kOut, kSplit, 1, 8, true>, a.splits);
  if (tile == 16) return small(ortho_small_kernel<kWhat, kOut, kSplit, 1, 8>, 1);
  if (tile == 32) return small(ortho_small_kernel<kWhat, kOut, kSplit, 2, 8>, 1);
  // Slabs ahead: 64 x 64 tiles two to a CU beat one with a deeper ring (2048 x 2048 gram 23.5 / 29.8 us), a
  // 128 x 128 one alone on its CU wants the ring (18.4 / 21.3)
  if (tile == 64) return go(ortho_product_kernel<kWhat, kOut, kSplit, 64, 64, 3>);
  if (tile == 128 && L * a.count <= kCus) return go(ortho_product_kernel<kWhat, kOut, kSplit, 128, 128, 3>);
  if (tile == 128) return go(ortho_product_kernel<kWhat, kOut, kSplit, 128, 128, 2>);
  if constexpr (!kSplit) {
    if (tile == 192) return go(ortho_product_kernel<kWhat, kOut, kSplit, 192, 192, 2>);
    go(ortho_product_kernel<kWhat, kOut, kSplit, 256, 256, 2>);
  }
}

template <Result kOut, bool kSplit>
static void launch_columns(const OrthoArgs& a, int64_t L, hipStream_t stream) {
  auto go = [&](auto pieces) {
    constexpr int P = decltype(pieces)::value;
    hipLaunchKernelGGL((ortho_columns_kernel<kOut, kSplit, P>), dim3((unsigned)(L * a.count)), dim3(128 * P), 0, stream, a);
  };
  using std::integral_constant;
  if constexpr (kSplit) {  // (of one number a value, m is more than 128)
    if (a.m == 64) return go(integral_constant<int, 2>{});
    if (a.m == 128) return go(integral_constant<int, 4>{});
  }
  if (a.m == 192) go(integral_constant<int, 6>{});
  else go(integral_constant<int, 8>{});
}

template <bool kSplit>
static hipError_t run_ortho(const void* g, bool g_bf16, int64_t L, int64_t M, int64_t N, int steps, bool bf16,
                            const OrthoPlan& o, OrthoArgs p, double* parts, _Float16* xt[2], _Float16* xt_lo[2], hipStream_t stream) {
  auto both = [&](auto squares, auto spread, auto from) {
    hipLaunchKernelGGL(squares, dim3(kNormParts, (unsigned)L), dim3(256), 0, stream, from, M * N, parts);
    const int64_t tn = (p.tall ? o.m : o.n) / 64, tiles = o.m / 64 * (o.n / 64);
    p.xt_new = xt[0], p.xt_lo_new = xt_lo[0];
    hipLaunchKernelGGL(spread, dim3((unsigned)(L * tiles)), dim3(256), 0, stream, from, (const double*)parts, (int)M, (int)N, (int)tn,
                       (int)tiles, p);
  };
  if (g_bf16) both(ortho_squares_kernel<bf16_t>, ortho_spread_kernel<bf16_t, kSplit>, (const bf16_t*)g);
  else both(ortho_squares_kernel<float>, ortho_spread_kernel<float, kSplit>, (const float*)g);
  for (int k = 0; k < steps; ++k) {
    // (the first step has no sum of squares before it, and alpha = 1 / m there)
    p.pivot = !kSplit && k >= 1 && k >= steps - 2;
    // (X before the last step: its rounding is not amplified any more, high alone adds 0 to 3e-4)
    p.low_in = k == 0 || k < steps - 1, p.low_out = k < steps - 2;
    p.xt = xt[k % 2], p.xt_lo = xt_lo[k % 2];
    p.xt_new = xt[1 - k % 2], p.xt_lo_new = xt_lo[1 - k % 2];
    p.count = (int)o.symmetric;
    launch_product<Product::kGram, Result::kPlanes, kSplit>(p, L, o.tile_sym, stream);
    if constexpr (kSplit)
      if (p.splits > 1) hipLaunchKernelGGL(ortho_join_kernel, dim3((unsigned)(L * p.count)), dim3(64), 0, stream, p);
    if (!o.columns) launch_product<Product::kSquare, Result::kPlanes, kSplit>(p, L, o.tile_sym, stream);
    p.count = (int)o.whole;
    auto update = [&](auto out) {
      constexpr Result kOut = decltype(out)::value;
      if (o.columns) launch_columns<kOut, kSplit>(p, L, stream);
      else launch_product<Product::kUpdate, kOut, kSplit>(p, L, o.tile, stream);
    };
    if (k < steps - 1) update(std::integral_constant<Result, Result::kPlanes>{});
    else if (bf16) update(std::integral_constant<Result, Result::kBf16>{});
    else if constexpr (kSplit) update(std::integral_constant<Result, Result::kF32>{});
  }
  return hipGetLastError();
}

hipError_t launch_orthogonalize(const void* g, bool g_bf16, int64_t L, int64_t M, int64_t N, int steps, float a, float b,
                                float c, float scale, void* out, bool out_bf16, bool single, void* ws, hipStream_t stream) {
  const OrthoPlan o = ortho_plan(L, M, N, single);  // single: of a bfloat16 result only
  OrthoArgs p{};
  p.m = (int)o.m, p.n = (int)o.n;
  p.tall = M > N;
  p.m_true = (int)(p.tall ? N : M), p.n_true = (int)(p.tall ? M : N);
  p.a = a, p.b = b, p.c = c, p.scale = scale, p.out = out;
  if (o.in_lds) {
    auto go = [&](auto kernel, auto from) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)L), dim3(64 * kWholeWaves), 0, stream, from, p, steps, out_bf16);
    };
    auto of = [&](auto s, auto from) {
      constexpr int S = decltype(s)::value;
      go(ortho_whole_kernel<std::remove_const_t<std::remove_pointer_t<decltype(from)>>, S>, from);
    };
    auto sized = [&](auto from) {
      if (o.m == 32) of(std::integral_constant<int, 1>{}, from);
      else of(std::integral_constant<int, 2>{}, from);
    };
    if (g_bf16) sized((const bf16_t*)g);
    else sized((const float*)g);
    return hipGetLastError();
  }
  p.parts = (int)o.whole * (o.columns ? (int)o.m / 16 : o.tile == 16 ? 1 : 4);
  uint8_t* at = (uint8_t*)ws;
  auto take = [&](int64_t bytes) {
    void* r = at;
    at += bytes;
    return r;
  };
  const int64_t mn = L * o.m * o.n * 2, mm = L * o.m * o.m * 2;
  _Float16 *xt[2], *xt_lo[2] = {nullptr, nullptr};
  p.x = (_Float16*)take(mn), p.x_lo = (_Float16*)take(mn);
  for (auto& v : xt) v = (_Float16*)take(mn);
  p.am = (_Float16*)take(mm);
  if (!o.columns) p.bm = (_Float16*)take(mm);
  if (o.split) {
    for (auto& v : xt_lo) v = (_Float16*)take(mn);
    p.am_lo = (_Float16*)take(mm);
    if (!o.columns) p.bm_lo = (_Float16*)take(mm);
  }
  double* const parts = (double*)take(L * kNormParts * 8);
  p.da = (float*)take(L * o.m * 4), p.db = (float*)take(L * o.m * 4);
  p.squares = (float*)take(L * o.whole * (o.columns ? 64 : 16));
  p.alpha = (float*)take(L * 16);
  p.splits = (int)o.splits;
  if (o.splits > 1) p.partial = (v4f*)take(L * o.symmetric * o.splits * 1024);
  return o.split ? run_ortho<true>(g, g_bf16, L, M, N, steps, out_bf16, o, p, parts, xt, xt_lo, stream)
                 : run_ortho<false>(g, g_bf16, L, M, N, steps, out_bf16, o, p, parts, xt, xt_lo, stream);
}

}  // namespace fp8q
