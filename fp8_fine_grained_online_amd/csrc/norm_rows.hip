// Normalization of rows that stay in bfloat16 or binary32, and its gradient with
// the reduction of the weights' gradients, for gfx950.
//
//   h = x + residual (rounded to x's type, where a residual is given), else x
//   centred: mu = sum h / K, var = sum (h - mu)^2 / K;  RMS: mu = 0
//   r = 1 / sqrt(var + eps),  hat = (h - mu) r,  y = hat gamma + beta
//
//   dg = dy gamma
//   dx = r (dg - [centred: sum dg / K] - hat sum(dg hat) / K) + dres
//   dgamma = sum over rows of dy hat,  dbeta = sum over rows of dy
//
// Both are bound by memory: a row is read once, held in registers by one
// wavefront or by a workgroup's, and reduced twice there (the mean, then the
// deviations). The second reduction also sums the deviations themselves, whose
// mean is what the rounded mean is off by: var and hat are put right with it, so
// rows with a mean far larger than their spread lose nothing to the mean's
// rounding. Sums are in binary32; a row whose statistics leave binary32's range
// (squares that overflow, or underflow where eps does not cover them) is done
// again in float64, from the registers.
#include <type_traits>

#include "common.hpp"
#include "rows.hpp"
#include "wave.hpp"

namespace fp8q {

typedef float v4f __attribute__((ext_vector_type(4)));

// kThreads per row (64: a wavefront; else a whole number of them), kChunks of
// eight values per thread: value 8 (t + kThreads i) + e belongs to thread t.
template <int kThreads, int kChunks>
struct RowShape {
  static constexpr int kT = kThreads, kC = kChunks;
  static constexpr int kMaxK = 8 * kThreads * kChunks;
  static constexpr bool kFew = false;
};
// Rows of 1 to 7 values: one thread has them all
struct FewShape : RowShape<64, 1> {
  static constexpr bool kFew = true;
};

template <typename Shape, bool kNt = false, typename T>
__device__ __forceinline__ Chunk<T> load_row_chunk(const T* row, int at, int K) {
  if constexpr (Shape::kFew) return load_few(row + at, K);
  else return load_in_row<kNt>(row, at, K);
}

// Eight weights, whose type is known at run time only
template <typename Shape>
__device__ __forceinline__ void row_weights(const void* w, bool bf16, int at, int K, float (&f)[8]) {
  if (bf16) values(load_row_chunk<Shape>((const bf16_t*)w, at, K), f);
  else values(load_row_chunk<Shape>((const float*)w, at, K), f);
}

// Sums over the threads of a row, the same bits in all of them. `slot`: LDS for
// kN sums of each of the row's wavefronts; a barrier separates two calls' uses of
// one slot.
template <int kThreads, int kN, typename S>
__device__ __forceinline__ void row_sums(S (&v)[kN], S (*slot)[kN]) {
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    if constexpr (sizeof(S) == 8) v[n] = wave_sum_f64(v[n]);
    else v[n] = wave_sum_f32(v[n]);
  }
  if constexpr (kThreads > 64) {
    const int wave = (threadIdx.x % kThreads) >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int n = 0; n < kN; ++n) slot[wave][n] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      S s = slot[0][n];
#pragma unroll
      for (int w = 1; w < kThreads / 64; ++w) s += slot[w][n];
      v[n] = s;
    }
  }
}

// LDS of one row's sums, a slot per reduction so that none waits for another's readers
template <int kThreads>
struct RowLds {
  float one[kThreads / 64][1], two[kThreads / 64][2];
  double wide[2][kThreads / 64][1];
};

struct RowStats {
  float mu, shift, r;  // hat = (h - mu) r - shift, shift = (what mu is off by) r
  float lift;             // 1 / std is r lift: 1, or 2^64 where it may pass binary32 (for the gradient)
  double wide_mu, wide_r;
  bool wide;  // the statistics are in the doubles
};

// An empty asm that "modifies" the values: what was computed from them before, their
// float64 forms above all, cannot be kept in registers for a later pass.
template <int C>
__device__ __forceinline__ void forget(float (&v)[C][8]) {
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) asm volatile("" : "+v"(v[i][e]));
}

// Statistics of the row whose values are in v; absent values are zeros.
// `present(i)`: how many of chunk i's values exist (0 to 8). kTogether: other rows
// of the workgroup meet the same barriers, so one that needs the wide way takes all
// along (who did not need it keeps what it had).
template <typename Shape, bool kCentred, bool kTogether, typename Present>
__device__ __forceinline__ RowStats row_stats(float (&v)[Shape::kC][8], Present present, int K, float eps,
                                              RowLds<Shape::kT>& lds) {
  constexpr int T = Shape::kT, C = Shape::kC;
  RowStats s;
  s.mu = s.shift = 0.0f, s.lift = 1.0f;
  s.wide_mu = 0.0, s.wide_r = 0.0;
  const float inv_k = 1.0f / (float)K;
  float stat[2] = {0.0f, 0.0f};  // sum of squared deviations, of deviations
  if constexpr (kCentred) {
    float sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[0] += v[i][e];
    row_sums<T, 1>(sum, lds.one);
    s.mu = sum[0] * inv_k;
  }
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int have = present(i);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = kCentred ? (e < have ? v[i][e] - s.mu : 0.0f) : v[i][e];
      stat[0] = __builtin_fmaf(d, d, stat[0]);
      if constexpr (kCentred) stat[1] += d;
    }
  }
  row_sums<T, 2>(stat, lds.two);
  const float off = stat[1] * inv_k;  // the true mean is mu + off
  const float raw = stat[0] * inv_k - off * off;  // NaN where both overflow
  s.wide = !(raw <= 1e36f) || (raw < 1e-30f && eps < 1e-25f);
  const float var = fmaxf(raw, 0.0f);
  s.r = (float)(1.0 / __dsqrt_rn((double)var + (double)eps));
  s.shift = off * s.r;
  if (!(kTogether ? __syncthreads_or(s.wide) : s.wide)) return s;
  forget(v);
  if constexpr (kCentred) {
    double sum[1] = {0.0};
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[0] += (double)v[i][e];
    row_sums<T, 1>(sum, lds.wide[0]);
    s.wide_mu = sum[0] / (double)K;
    forget(v);
  }
  double sq[1] = {0.0};
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int have = present(i);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double d = e < have ? (double)v[i][e] - s.wide_mu : 0.0;
      sq[0] = __builtin_fma(d, d, sq[0]);
    }
  }
  row_sums<T, 1>(sq, lds.wide[1]);
  s.wide_r = 1.0 / __dsqrt_rn(sq[0] / (double)K + (double)eps);
  if (s.wide) {
    s.lift = s.wide_r > 0x1p100 ? 0x1p64f : 1.0f;
    s.r = (float)(s.wide_r / (double)s.lift);
  }
  forget(v);
  return s;
}

// v becomes hat. The branch is the row's, so the wavefront's.
template <bool kCentred, int C>
__device__ __forceinline__ void to_hat(float (&v)[C][8], const RowStats& s) {
  if (__builtin_amdgcn_readfirstlane(s.wide)) {
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = (float)(((double)v[i][e] - s.wide_mu) * s.wide_r);
    return;
  }
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = kCentred ? __builtin_fmaf(v[i][e] - s.mu, s.r, -s.shift) : v[i][e] * s.r;
}

// ---------------------------------------------------------------------------
// Forward. One row per kT threads; rows of up to 1024 values take a wavefront
// each, four to a workgroup, longer ones a workgroup.
// 8192 x 7168 with a residual 81 us (5.8 TB/s), 1237 x 2050 (float32) 7.6, one row 3.6: there x, the residual and
// gamma are waited for one after the other. Rows below 512 values leave lanes without work: 64 values 1 TB/s, 256 3.4.
// ---------------------------------------------------------------------------
struct NormArgs {
  const void *x, *res, *gamma, *beta;
  void *y, *h;
  int64_t ldx, ldr;
  int M, K;
  float eps;
  bool weights_bf16;
  bool nt;  // more is read and written than stays cached
};

// Reads that pass the caches by from 96 MiB of reads and writes on, which neither
// leaves nor finds them there whole: 8192 x 7168 with a residual 86.6 -> 83.0 us, its
// gradient 95.5 -> 93.1, 16384 x 1024 25.6 -> 23.9; but 4096 x 2048 12.0 -> 12.4.
static bool beyond_cache(int64_t bytes) { return bytes > (int64_t(96) << 20); }

template <typename Shape>
constexpr int kRowThreads = Shape::kT == 64 ? 256 : Shape::kT;  // of a workgroup

template <typename Shape, typename X, typename Y, bool kCentred>
__global__ __launch_bounds__(kRowThreads<Shape>) void norm_rows_kernel(NormArgs p) {
  constexpr int T = Shape::kT, C = Shape::kC, kRows = kRowThreads<Shape> / T;
  __shared__ RowLds<T> lds[kRows];
  const int tid = threadIdx.x % T, sub = __builtin_amdgcn_readfirstlane(threadIdx.x / T);
  const int64_t m = (int64_t)blockIdx.x * kRows + sub;
  if (m >= p.M) return;  // (kRows > 1: rows are single wavefronts, which meet no barrier)
  const int chunks = (p.K + 7) / 8;
  auto at = [&](int i) { return 8 * (tid + T * i); };
  auto present = [&](int i) { return min(max(p.K - at(i), 0), 8); };
  const X* const x = (const X*)p.x + m * p.ldx;
  Chunk<X> raw[C];
  auto read = [&](const X* row) {
    if (p.nt) {
#pragma unroll
      for (int i = 0; i < C; ++i) raw[i] = tid + T * i < chunks ? load_row_chunk<Shape, true>(row, at(i), p.K) : zero_chunk(X{});
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) raw[i] = tid + T * i < chunks ? load_row_chunk<Shape>(row, at(i), p.K) : zero_chunk(X{});
    }
  };
  read(x);
  float v[C][8];
#pragma unroll
  for (int i = 0; i < C; ++i) values(raw[i], v[i]);
  if (p.res) {
    const X* const res = (const X*)p.res + m * p.ldr;
    X* const h = (X*)p.h + m * (int64_t)p.K;
    read(res);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float r[8];
      values(raw[i], r);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] += r[e];
      to_chunk(v[i], raw[i]);  // what is kept is what is normalized
      values(raw[i], v[i]);
      if (tid + T * i < chunks) store_chunk(h + at(i), raw[i], present(i));
    }
  }
  const RowStats s = row_stats<Shape, kCentred, false>(v, present, p.K, p.eps, lds[sub]);
  to_hat<kCentred>(v, s);
  Y* const y = (Y*)p.y + m * (int64_t)p.K;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if (tid + T * i >= chunks) break;
    const int have = present(i);
    float g[8], b[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    row_weights<Shape>(p.gamma, p.weights_bf16, at(i), p.K, g);
    if (kCentred && p.beta) row_weights<Shape>(p.beta, p.weights_bf16, at(i), p.K, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      g[e] *= v[i][e];
      if (kCentred && p.beta) g[e] += b[e];
    }
    Chunk<Y> out;
    to_chunk(g, out);
    store_chunk(y + at(i), out, have);
  }
}

// ---------------------------------------------------------------------------
// Gradient. A workgroup of kBwdThreads takes rows in turn, 512 / kT at once, the
// next ones' loads on their way while it works on these; gamma stays in LDS. A
// thread's columns are the same in every row, so the weights' gradients are sums
// in its registers, joined at the end over the workgroup's rows in LDS and written
// as one row of partial sums. A second kernel adds those in order: no atomics,
// and the same bits every time. 8192 x 7168 with a residual's gradient 84 us (5.6 TB/s, of
// which the second kernel 5), 333 x 2049 (float32) 12.8: two launches and a row's chain of reductions.
// ---------------------------------------------------------------------------
constexpr int kBwdThreads = 512;  // of a workgroup

struct NormBwdArgs {
  const void *dy, *x, *gamma, *dres;
  void* dx;
  float* partial;  // [workgroups][centred ? 2 : 1][K]
  int64_t ldy, ldx, ldr;
  int M, K;
  float eps;
  bool weights_bf16, nt;
};

template <typename Shape, typename X, typename D, bool kCentred>
__global__ __launch_bounds__(kBwdThreads) void norm_rows_bwd_kernel(NormBwdArgs p) {
  constexpr int kWg = kBwdThreads, T = Shape::kT, C = Shape::kC, kRows = kWg / T;
  constexpr int kSums = kCentred ? 2 : 1;
  struct Slots {
    RowLds<T> row;
    float sums[T / 64][2];
  };
  __shared__ Slots slots[kRows];
  extern __shared__ __attribute__((aligned(16))) float shared[];  // gamma, padded to whole chunks; then sums to join
  const int tid = threadIdx.x % T, sub = __builtin_amdgcn_readfirstlane(threadIdx.x / T);
  const int chunks = (p.K + 7) / 8;
  auto at = [&](int i) { return 8 * (tid + T * i); };
  auto present = [&](int i) { return min(max(p.K - at(i), 0), 8); };
  auto gamma_of = [&](int i, float (&g)[8]) {
    const v4f a = *(const v4f*)(shared + at(i)), b = *(const v4f*)(shared + at(i) + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) g[e] = a[e], g[4 + e] = b[e];
  };
  float dgamma[C][8], dbeta[kCentred ? C : 1][8];
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dgamma[i][e] = 0.0f;
      if constexpr (kCentred) dbeta[i][e] = 0.0f;
    }
  Chunk<X> rx[C], rr[C];
  Chunk<D> rd[C];
  auto read_as = [&](auto nt, int64_t m) {
    constexpr bool kNt = decltype(nt)::value;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const bool have = m < p.M && tid + T * i < chunks;
      rx[i] = have ? load_row_chunk<Shape, kNt>((const X*)p.x + m * p.ldx, at(i), p.K) : zero_chunk(X{});
      rd[i] = have ? load_row_chunk<Shape, kNt>((const D*)p.dy + m * p.ldy, at(i), p.K) : zero_chunk(D{});
      rr[i] = have && p.dres ? load_row_chunk<Shape, kNt>((const X*)p.dres + m * p.ldr, at(i), p.K) : zero_chunk(X{});
    }
  };
  auto read_rows = [&](int64_t m) {  // (longer parts of a row than two chunks leave no registers for both forms)
    if (C <= 2 && p.nt) read_as(std::true_type{}, m);
    else read_as(std::false_type{}, m);
  };
  const float inv_k = 1.0f / (float)p.K;
  read_rows((int64_t)blockIdx.x * kRows + sub);
  for (int c = threadIdx.x; c < chunks; c += kWg) {
    float g[8];
    row_weights<Shape>(p.gamma, p.weights_bf16, 8 * c, p.K, g);  // absent ones are zeros
    *(v4f*)(shared + 8 * c) = v4f{g[0], g[1], g[2], g[3]};
    *(v4f*)(shared + 8 * c + 4) = v4f{g[4], g[5], g[6], g[7]};
  }
  __syncthreads();
  // every thread of the workgroup makes the same number of rounds (barriers inside)
  for (int64_t m0 = (int64_t)blockIdx.x * kRows; m0 < p.M; m0 += (int64_t)gridDim.x * kRows) {
    const int64_t m = m0 + sub;
    float v[C][8];
    Chunk<D> d_now[C];
    Chunk<X> r_now[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      values(rx[i], v[i]);
      d_now[i] = rd[i];
      r_now[i] = rr[i];
    }
    read_rows(m + (int64_t)gridDim.x * kRows);
    const RowStats s = row_stats<Shape, kCentred, (T > 64 && kRows > 1)>(v, present, p.K, p.eps, slots[sub].row);
    to_hat<kCentred>(v, s);
    float sums[2] = {0.0f, 0.0f};  // of dg hat, of dg
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if (tid + T * i >= chunks) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
        continue;
      }
      float d[8], g[8];
      gamma_of(i, g);
      values(d_now[i], d);
      // (dy and gamma are zero past the row's end, and a row that is not there has zeros throughout,
      // but its hat may not be finite)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (m < p.M) dgamma[i][e] = __builtin_fmaf(d[e], v[i][e], dgamma[i][e]);
        if constexpr (kCentred) dbeta[i][e] += d[e];
        const float dg = d[e] * g[e];
        sums[0] = __builtin_fmaf(dg, v[i][e], sums[0]);
        sums[1] += dg;
      }
    }
    row_sums<T, 2>(sums, slots[sub].sums);
    const float c_hat = sums[0] * inv_k, c_one = kCentred ? sums[1] * inv_k : 0.0f;
    const float lift = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(s.lift)));
    if (m < p.M) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        if (tid + T * i >= chunks) break;
        float d[8], g[8], o[8];
        gamma_of(i, g);
        values(d_now[i], d);
        values(r_now[i], o);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float t = __builtin_fmaf(-v[i][e], c_hat, d[e] * g[e] - c_one);
          o[e] = __builtin_fmaf(s.r, t * lift, o[e]);
        }
        Chunk<X> out;
        to_chunk(o, out);
        store_chunk((X*)p.dx + m * (int64_t)p.K + at(i), out, present(i));
      }
    }
    if constexpr (T > 64) __syncthreads();  // the slots are used again
  }
  // join the workgroup's rows, in order
  if constexpr (kRows > 1) {
    float* const join = shared;  // (gamma has been read)
    for (int r = 0; r < kRows; ++r) {
      __syncthreads();
      if (sub == r) {
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float* const to = join + (i * 8 + e) * T + tid;
            dgamma[i][e] = *to = r ? *to + dgamma[i][e] : dgamma[i][e];
            if constexpr (kCentred) dbeta[i][e] = to[8 * T * C] = r ? to[8 * T * C] + dbeta[i][e] : dbeta[i][e];
          }
      }
    }
    if (sub != kRows - 1) return;
  }
  float* const part = p.partial + (int64_t)blockIdx.x * kSums * p.K;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int have = present(i);
    if (!have) continue;
    Chunk<float> c;
    to_chunk(dgamma[i], c);
    store_chunk(part + at(i), c, have);
    if constexpr (kCentred) {
      to_chunk(dbeta[i], c);
      store_chunk(part + p.K + at(i), c, have);
    }
  }
}

// Sums of the partial rows: 32 columns and 32 runs of rows per workgroup.
constexpr int kJoinCols = 32, kJoinRuns = 32;

__global__ __launch_bounds__(kJoinCols* kJoinRuns) void join_partials_kernel(const float* __restrict__ partial, int rows,
                                                                             int cols, int K, float* __restrict__ dgamma,
                                                                             float* __restrict__ dbeta) {
  __shared__ float runs[kJoinRuns][kJoinCols];
  const int c = blockIdx.x * kJoinCols + threadIdx.x % kJoinCols, run = threadIdx.x / kJoinCols;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int r = run; r < rows; r += kJoinRuns) s += partial[(int64_t)r * cols + c];
  }
  runs[run][threadIdx.x % kJoinCols] = s;
  __syncthreads();
  if (run || c >= cols) return;
#pragma unroll
  for (int r = 1; r < kJoinRuns; ++r) s += runs[r][threadIdx.x];
  if (c < K) dgamma[c] = s;
  else dbeta[c - K] = s;
}

// ---------------------------------------------------------------------------
template <typename Shape, typename X, typename Y>
static void launch_fwd(const NormArgs& a, bool centred, hipStream_t stream) {
  constexpr int rows = kRowThreads<Shape> / Shape::kT;
  const dim3 grid((unsigned)((a.M + rows - 1) / rows)), block(kRowThreads<Shape>);
  if (centred) hipLaunchKernelGGL((norm_rows_kernel<Shape, X, Y, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((norm_rows_kernel<Shape, X, Y, false>), grid, block, 0, stream, a);
}

template <typename X, typename Y>
static void launch_fwd_shape(const NormArgs& a, bool centred, hipStream_t stream) {
  // Few chunks per thread: more rows in flight beat longer parts of a row (8192 x 7168 with
  // 512 x 2 / 256 x 4 82.4 / 83.3 us, 333 x 7168 6.2 / 6.7; with 1024 x 2 / 512 x 4 100 x
  // 16384 5.4 / 6.3, but 6000 x 10240 86.7 / 84.3). 512 threads of one chunk beat 256 of two where they
  // are nearly all used: 16384 x 4096 89.2 / 92.8, but 4000 x 2049 (float32) 17.3 / 15.1.
  if (a.K < 8) return launch_fwd<FewShape, X, Y>(a, centred, stream);
  if (a.K <= 512) return launch_fwd<RowShape<64, 1>, X, Y>(a, centred, stream);
  if (a.K <= 1024) return launch_fwd<RowShape<64, 2>, X, Y>(a, centred, stream);
  if (a.K <= 2048) return launch_fwd<RowShape<128, 2>, X, Y>(a, centred, stream);
  if (a.K <= 3584) return launch_fwd<RowShape<256, 2>, X, Y>(a, centred, stream);
  if (a.K <= 4096) return launch_fwd<RowShape<512, 1>, X, Y>(a, centred, stream);
  if (a.K <= 8192) return launch_fwd<RowShape<512, 2>, X, Y>(a, centred, stream);
  if (a.K <= 12288) return launch_fwd<RowShape<512, 4>, X, Y>(a, centred, stream);
  launch_fwd<RowShape<1024, 2>, X, Y>(a, centred, stream);
}

hipError_t launch_norm_rows(const void* x, bool x_bf16, int64_t ldx, const void* res, int64_t ldr, const void* gamma,
                            const void* beta, bool weights_bf16, float eps, bool centred, int64_t M, int64_t K, void* y,
                            bool y_bf16, void* h, hipStream_t stream) {
  const int64_t ex = x_bf16 ? 2 : 4, ey = y_bf16 ? 2 : 4;
  const NormArgs a{x, res, gamma, beta, y, h, ldx, ldr, (int)M, (int)K, eps, weights_bf16,
                   beyond_cache(M * K * (ex * (res ? 3 : 1) + ey))};
  if (x_bf16) {
    if (y_bf16) launch_fwd_shape<bf16_t, bf16_t>(a, centred, stream);
    else launch_fwd_shape<bf16_t, float>(a, centred, stream);
  } else {
    if (y_bf16) launch_fwd_shape<float, bf16_t>(a, centred, stream);
    else launch_fwd_shape<float, float>(a, centred, stream);
  }
  return hipGetLastError();
}

// The gradient's threads per row and per workgroup, and its workgroups: as many as are
// resident, fewer for few rows. us, MI355X, threads x chunks and workgroups against others:
//   8192 x 7168   512 x 2, 512  89.9    256 workgroups 111    256 x 4, 256  94.2
//   16384 x 4096  512 x 1, 512  90.1    256 x 2, 512  90.6    256 x 2, 256  124
//   4096 x 2048   256 x 1, 512  20.2    128 x 2, 512  20.4    64 x 4, 256  over 22
//   16384 x 1024  64 x 2, 512  28.9     64 x 2, 256  31.7     128 x 1, 512  33.4
//   6000 x 10240  512 x 3, 256  98.5    512 x 4, 256  96.8    1024 x 2, 256  109
//   3000 x 10240 (float32)  512 x 3, 256  90.4    512 x 4, 256  174    1024 x 2, 256  260
//   4000 x 16384  512 x 4, 256  110     512 x 4, 512  117     1024 x 2, 256  110
struct BwdPlan {
  int threads;
  int64_t workgroups;
};
static BwdPlan bwd_plan(int64_t M, int64_t K) {
  BwdPlan b;
  b.threads = K <= 1024 ? 64 : K <= 2048 ? 256 : 512;
  const int rows = kBwdThreads / b.threads;
  const int64_t need = (M + rows - 1) / rows, most = K <= 8192 ? 512 : 256;
  b.workgroups = need < most ? need : most;
  return b;
}

int64_t norm_bwd_workspace_bytes(int64_t M, int64_t K, bool centred) {
  return bwd_plan(M, K).workgroups * (centred ? 2 : 1) * K * (int64_t)sizeof(float);
}

template <typename Shape, typename X, typename D>
static void launch_bwd(const NormBwdArgs& a, bool centred, const BwdPlan& b, hipStream_t stream) {
  constexpr int kT = Shape::kT, kWg = kBwdThreads;
  const dim3 grid((unsigned)b.workgroups), block(kWg);
  const size_t gamma = (size_t)(a.K + 7) / 8 * 32, join = kWg > kT ? (size_t)(centred ? 2 : 1) * Shape::kMaxK * 4 : 0;
  const size_t lds = gamma > join ? gamma : join;
  if (centred) hipLaunchKernelGGL((norm_rows_bwd_kernel<Shape, X, D, true>), grid, block, lds, stream, a);
  else hipLaunchKernelGGL((norm_rows_bwd_kernel<Shape, X, D, false>), grid, block, lds, stream, a);
}

template <typename X, typename D>
static void launch_bwd_shape(const NormBwdArgs& a, bool centred, const BwdPlan& b, hipStream_t stream) {
  if (a.K < 8) return launch_bwd<FewShape, X, D>(a, centred, b, stream);
  if (a.K <= 512) return launch_bwd<RowShape<64, 1>, X, D>(a, centred, b, stream);
  if (a.K <= 1024) return launch_bwd<RowShape<64, 2>, X, D>(a, centred, b, stream);
  if (a.K <= 2048) return launch_bwd<RowShape<256, 1>, X, D>(a, centred, b, stream);
  if (a.K <= 4096) return launch_bwd<RowShape<512, 1>, X, D>(a, centred, b, stream);
  if (a.K <= 8192) return launch_bwd<RowShape<512, 2>, X, D>(a, centred, b, stream);
  if (a.K <= 12288) return launch_bwd<RowShape<512, 3>, X, D>(a, centred, b, stream);
  launch_bwd<RowShape<512, 4>, X, D>(a, centred, b, stream);
}

hipError_t launch_norm_rows_bwd(const void* dy, bool dy_bf16, int64_t ldy, const void* x, bool x_bf16, int64_t ldx,
                                const void* gamma, bool weights_bf16, const void* dres, int64_t ldr, float eps,
                                bool centred, int64_t M, int64_t K, void* dx, float* dgamma, float* dbeta, void* ws,
                                hipStream_t stream) {
  const int64_t ex = x_bf16 ? 2 : 4, ed = dy_bf16 ? 2 : 4;
  const NormBwdArgs a{dy, x, gamma, dres, dx, (float*)ws, ldy, ldx, ldr, (int)M, (int)K, eps, weights_bf16,
                      beyond_cache(M * K * (ex * (dres ? 3 : 2) + ed))};
  const BwdPlan b = bwd_plan(M, K);
  if (M > 0) {
    if (x_bf16) {
      if (dy_bf16) launch_bwd_shape<bf16_t, bf16_t>(a, centred, b, stream);
      else launch_bwd_shape<bf16_t, float>(a, centred, b, stream);
    } else {
      if (dy_bf16) launch_bwd_shape<float, bf16_t>(a, centred, b, stream);
      else launch_bwd_shape<float, float>(a, centred, b, stream);
    }
    if (hipError_t e = hipGetLastError()) return e;
  }
  const int cols = (int)K * (centred ? 2 : 1);
  hipLaunchKernelGGL(join_partials_kernel, dim3((unsigned)((cols + kJoinCols - 1) / kJoinCols)),
                     dim3(kJoinCols * kJoinRuns), 0, stream, (const float*)ws, (int)b.workgroups, cols, (int)K,
                     dgamma, dbeta);
  return hipGetLastError();
}

}  // namespace fp8q
