// Rows sorted by expert and back, for gfx950: the copy of the tokens' rows
// into the padded per-expert layout (permute), the weighted sum back to tokens
// (combine) and that sum's gradient (combine_bwd).
//
//   xp[row_of_slot[t, j], :] = x[t, :]
//   y[t, :] = sum_j w[t, j] c[row_of_slot[t, j], :]
//   dc[row_of_slot[t, j], :] = w[t, j] dy[t, :],  dw[t, j] = <dy[t, :], c[row_of_slot[t, j], :]>
//
// All three move rows and do almost no arithmetic: they are bound by HBM.
// Rows are handled in chunks of 8 values, one chunk per lane (16 bytes of
// bfloat16, 32 of float32).
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "wave.hpp"

namespace fp8q {

constexpr int kTokWaves = 4;  // wavefronts per workgroup

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 8 values of a row: kept as loaded (Raw), and as floats
template <typename T>
struct Chunk;
template <>
struct Chunk<uint16_t> {  // bfloat16
  struct Raw { u32x4 v; };
  static constexpr int kBytes = 16;
  static __device__ __forceinline__ Raw load(const void* p) { return {*(const u32x4*)p}; }
  static __device__ __forceinline__ Raw load_nt(const void* p) {
    return {__builtin_nontemporal_load((const u32x4*)p)};
  }
  static __device__ __forceinline__ Raw zero() { return {u32x4{0, 0, 0, 0}}; }
  template <bool kNt>
  static __device__ __forceinline__ void store(void* p, Raw r) {
    if constexpr (kNt) __builtin_nontemporal_store(r.v, (u32x4*)p);
    else *(u32x4*)p = r.v;
  }
  static __device__ __forceinline__ void floats(Raw r, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(r.v[i]), f[2 * i + 1] = bf16_hi(r.v[i]);
  }
  static __device__ __forceinline__ Raw round(const float (&f)[8]) {
    bf16x8 b;
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = (__bf16)f[i];
    return {__builtin_bit_cast(u32x4, b)};
  }
};
template <>
struct Chunk<float> {
  struct Raw { u32x4 v, w; };
  static constexpr int kBytes = 32;
  static __device__ __forceinline__ Raw load(const void* p) {
    return {((const u32x4*)p)[0], ((const u32x4*)p)[1]};
  }
  static __device__ __forceinline__ Raw load_nt(const void* p) {
    return {__builtin_nontemporal_load((const u32x4*)p), __builtin_nontemporal_load((const u32x4*)p + 1)};
  }
  static __device__ __forceinline__ Raw zero() { return {u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}}; }
  template <bool kNt>
  static __device__ __forceinline__ void store(void* p, Raw r) {
    if constexpr (kNt) {
      __builtin_nontemporal_store(r.v, (u32x4*)p);
      __builtin_nontemporal_store(r.w, (u32x4*)p + 1);
    } else {
      ((u32x4*)p)[0] = r.v;
      ((u32x4*)p)[1] = r.w;
    }
  }
  static __device__ __forceinline__ void floats(Raw r, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(r.v[i]), f[4 + i] = __uint_as_float(r.w[i]);
  }
  static __device__ __forceinline__ Raw round(const float (&f)[8]) {
    Raw r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = __float_as_uint(f[i]), r.w[i] = __float_as_uint(f[4 + i]);
    return r;
  }
};

// ---------------------------------------------------------------------------
// permute: one workgroup per token copies its row to the rows of its valid
// slots; further workgroups, up to kPadParts per expert, zero its padding rows
// (at most 127, 32 KB each at least: 512 slots of 1024 experts, K = 256, took
// 29.5 us with 16 parts, a row per part, and 9.3 with 2).
//
// A slot's row is its expert's first row plus the number of earlier slots with
// that expert. Where that comes from (Way):
//   kSort   every workgroup sorts the ids by itself, in LDS: the call is this
//           kernel alone. Up to kSortSlots slots.
//   kCount  a kernel counts blocks of kCountBlock slots and leaves every slot's
//           rank in its block; the workgroups here add the blocks up. Up to
//           kCountBlocks blocks and kCountTokens tokens (each pays for it).
//   kScan   the dispatch's counting and scanning kernels.
// us on MI355X, kSort / kCount / kScan:
//   16 tokens, top-8 of 8, K = 256      4.5 /   - / 10.3
//   1024, top-1 of 64, K = 256          6.2 /   - / 13.6
//   256, top-8 of 8, K = 256           10.4 / 7.7 / 10.7
//   512, top-8 of 32, K = 7168            - / 20.9 / 25.7
//   2048, top-8 of 32, K = 7168           - / 54.1 / 59.9
//   4096, top-1 of 8, K = 256             - / 12.5 / 11.8; K = 7168 29.3 / 31.8
//   8192, top-8 of 32, K = 7168           - / 226 / 215
//
// Rows are written with ordinary stores even where they cannot stay in the
// Infinity Cache: 8192 tokens x top-8 x 7168 took 197 us with them and 210 with
// non-temporal ones (a wavefront per token, its row held in registers: 205 and
// 227).
// ---------------------------------------------------------------------------
constexpr int kPadParts = 16;
constexpr int kSortSlots = 1024;   // most slots a workgroup sorts by itself
constexpr int kCountBlock = 4096;  // slots per block of the counting kernel below
constexpr int kCountBlocks = 16;
constexpr int kCountTokens = 4096;
constexpr int kDispBlock = 256;    // and of the dispatch's
constexpr int kMaxExperts = 1024;

struct PermuteArgs {
  const uint8_t* x;
  const int32_t* ids;
  const int32_t* hist;    // kCount: slots of each (block, expert)
  const int32_t* base;    // kScan: first row of each (block, expert)
  const int32_t* counts;  // kScan: slots of each expert
  int32_t* row_of_slot;
  int32_t* m_offsets;
  uint8_t* xp;
  int n_tok, K, topk, G, pad_parts;
};

enum Way { kSort, kCount, kScan };

// Ranks of the slots of a block among its slots with the same expert (-1: no
// expert), and the block's histogram. 16 wavefronts, each with a histogram of
// its 256 slots so far: lanes with the same expert find each other bit by bit
// of its number.
constexpr int kCountWaves = kCountBlock / 256;

__global__ __launch_bounds__(64 * kCountWaves) void token_count_kernel(const int32_t* __restrict__ ids, int slots,
                                                                      int G, int32_t* __restrict__ hist,
                                                                      int32_t* __restrict__ in_block) {
  __shared__ int32_t of_wave[kCountWaves][kMaxExperts];
  constexpr int kSets = 4;  // of 64 slots per wavefront
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t slot0 = (int64_t)blockIdx.x * kCountBlock + wave * 256 + lane;
  int e[kSets], rank[kSets];
#pragma unroll
  for (int u = 0; u < kSets; ++u) e[u] = slot0 + u * 64 < slots ? ids[slot0 + u * 64] : -1;
  for (int i = lane; i < G; i += 64) of_wave[wave][i] = 0;
  const int bits = G > 1 ? 32 - __builtin_clz(G - 1) : 0;
#pragma unroll
  for (int u = 0; u < kSets; ++u) {
    const bool on = e[u] >= 0 && e[u] < G;
    uint64_t same = __ballot(on);
    for (int b = 0; b < bits; ++b) {
      const bool one = (e[u] >> b) & 1;
      const uint64_t ones = __ballot(one);
      same &= one ? ones : ~ones;
    }
    if (!on) e[u] = -1;
    // (the wave's LDS accesses are in order; the fences keep the compiler to it)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int before = on ? of_wave[wave][e[u]] : 0;
    rank[u] = before + __popcll(same & ((1ull << lane) - 1));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (on && (same >> lane) == 1) of_wave[wave][e[u]] = rank[u] + 1;  // the last of them
  }
  __syncthreads();
  for (int x = tid; x < G; x += 64 * kCountWaves) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kCountWaves; ++w) {
      const int c = of_wave[w][x];
      of_wave[w][x] = sum;
      sum += c;
    }
    hist[(int64_t)blockIdx.x * G + x] = sum;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kSets; ++u)
    if (slot0 + u * 64 < slots) in_block[slot0 + u * 64] = e[u] < 0 ? -1 : rank[u] + of_wave[wave][e[u]];
}

struct ExpertLds {
  int32_t counts[kMaxExperts];
  int32_t offsets[kMaxExperts + 1];  // first row of each expert's block
  int32_t wave_sum[kTokWaves];
};
struct SortLds : ExpertLds {
  int16_t ids[kSortSlots];  // -1: dropped
};
struct CountLds : ExpertLds {
  int32_t before[kMaxExperts];  // slots of each expert in the blocks before the token's
};
struct ScanLds {};

template <Way kWay>
using WayLds = std::conditional_t<kWay == kSort, SortLds, std::conditional_t<kWay == kCount, CountLds, ScanLds>>;

// The ids and every expert's count, by the whole workgroup.
__device__ __forceinline__ void count_experts(SortLds& s, const PermuteArgs& a) {
  constexpr int kThreads = 64 * kTokWaves;
  const int tid = threadIdx.x, slots = a.n_tok * a.topk;
  for (int e = tid; e < a.G; e += kThreads) s.counts[e] = 0;
  __syncthreads();
  for (int i = tid; i < slots; i += kThreads) {
    const int e = a.ids[i];
    const bool on = e >= 0 && e < a.G;
    s.ids[i] = on ? (int16_t)e : (int16_t)-1;
    if (on) atomicAdd(&s.counts[e], 1);  // integers: any order, the same counts
  }
}

// Every expert's count, and that of the blocks before block `own`.
__device__ __forceinline__ void count_experts(CountLds& s, const PermuteArgs& a, int n_blk, int own) {
  for (int e = threadIdx.x; e < a.G; e += 64 * kTokWaves) {
    int h[kCountBlocks], before = 0, sum = 0;
#pragma unroll
    for (int b = 0; b < kCountBlocks; ++b) h[b] = b < n_blk ? a.hist[b * a.G + e] : 0;
#pragma unroll
    for (int b = 0; b < kCountBlocks; ++b) {
      if (b == own) before = sum;
      sum += h[b];
    }
    s.counts[e] = sum;
    s.before[e] = before;
  }
}

// Padded offsets from the counts, by the whole workgroup.
__device__ __forceinline__ void offset_experts(ExpertLds& s, int G) {
  constexpr int kThreads = 64 * kTokWaves;
  constexpr int kEach = kMaxExperts / kThreads;  // consecutive experts per thread
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  __syncthreads();
  int padded[kEach], sum = 0;
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int e = tid * kEach + u;
    padded[u] = e < G ? (s.counts[e] + kGroup - 1) / kGroup * kGroup : 0;
    sum += padded[u];
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 63) s.wave_sum[wave] = incl;
  __syncthreads();
  int at = incl - sum;
  for (int w = 0; w < wave; ++w) at += s.wave_sum[w];
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int e = tid * kEach + u;
    if (e < G) s.offsets[e] = at;
    at += padded[u];
    if (e == G - 1) s.offsets[G] = at;
  }
  __syncthreads();
}

template <typename T, Way kWay>
__global__ __launch_bounds__(64 * kTokWaves) void permute_kernel(PermuteArgs a) {
  using C = Chunk<T>;
  constexpr int kThreads = 64 * kTokWaves;
  constexpr int kHeld = 4;  // chunks of the row a lane holds at a time
  __shared__ WayLds<kWay> experts;
  __shared__ int32_t rows[64];  // of the current 64 choices
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n_chunks = a.K / 8;
  const int64_t row_bytes = (int64_t)n_chunks * C::kBytes;
  const int64_t first_slot = (int64_t)blockIdx.x * a.topk;
  const int own = (int)(first_slot / kCountBlock);  // kCount: the block of the token's first slot
  int rank = -1, mine = -1;                         // choice j0 + lane: rank in its block, and expert
  auto load_choice = [&](int j) {
    rank = mine = -1;
    if (j < a.topk) rank = a.row_of_slot[first_slot + j], mine = a.ids[first_slot + j];
  };
  if constexpr (kWay != kScan) {
    if constexpr (kWay == kSort) {
      count_experts(experts, a);
    } else {
      if ((int)blockIdx.x < a.n_tok && wave == 0) load_choice(lane);
      count_experts(experts, a, (int)(((int64_t)a.n_tok * a.topk + kCountBlock - 1) / kCountBlock), own);
    }
    offset_experts(experts, a.G);
    if (blockIdx.x == 0)
      for (int e = tid; e <= a.G; e += kThreads) a.m_offsets[e] = experts.offsets[e];
  }
  if ((int)blockIdx.x >= a.n_tok) {
    const int pad = blockIdx.x - a.n_tok;
    const int e = pad / a.pad_parts;
    int row, end;
    if constexpr (kWay != kScan) row = experts.offsets[e] + experts.counts[e], end = experts.offsets[e + 1];
    else row = a.m_offsets[e] + a.counts[e], end = a.m_offsets[e + 1];
    const int64_t n = (int64_t)(end - row) * n_chunks;  // contiguous
    for (int64_t i = pad % a.pad_parts * kThreads + tid; i < n; i += a.pad_parts * kThreads)
      C::template store<false>(a.xp + row * row_bytes + i * C::kBytes, C::zero());
    return;
  }
  const uint8_t* xr = a.x + blockIdx.x * row_bytes;
  for (int j0 = 0; j0 < a.topk; j0 += 64) {
    const int n = min(64, a.topk - j0);
    // ---- rows of choices j0 .. j0 + n - 1 ----
    if (j0 > 0) __syncthreads();
    if constexpr (kWay == kSort) {
      // a slot's rank: the earlier slots with its expert
      for (int j = wave; j < n; j += kTokWaves) {
        const int slot = (int)first_slot + j0 + j;
        const int e = experts.ids[slot];
        int rank = 0;
        for (int i0 = 0; i0 < slot; i0 += 64)
          rank += __popcll(__ballot(i0 + lane < slot && experts.ids[i0 + lane] == e));
        if (lane == 0) rows[j] = e < 0 ? -1 : experts.offsets[e] + rank;
      }
    } else if (wave == 0 && lane < n) {
      const int64_t slot = first_slot + j0 + lane;
      if constexpr (kWay == kCount) {
        if (j0 > 0) load_choice(j0 + lane);
        int row = rank;
        if (rank >= 0) {
          row += experts.offsets[mine] + experts.before[mine];
          for (int b = own; b < (int)(slot / kCountBlock); ++b) row += a.hist[b * a.G + mine];
        }
        rows[lane] = row;
      } else {
        const int in_block = a.row_of_slot[slot];
        rows[lane] = in_block < 0 ? -1 : a.base[(slot / kDispBlock) * a.G + a.ids[slot]] + in_block;
      }
    }
    __syncthreads();
    if (wave == 0 && lane < n) a.row_of_slot[first_slot + j0 + lane] = rows[lane];
    const int lane_row = lane < n ? rows[lane] : -1;
    // ---- copies ----
    for (int c0 = tid; c0 < n_chunks; c0 += kThreads * kHeld) {
      typename C::Raw v[kHeld];
#pragma unroll
      for (int u = 0; u < kHeld; ++u)
        if (c0 + kThreads * u < n_chunks) v[u] = C::load_nt(xr + (int64_t)(c0 + kThreads * u) * C::kBytes);
      for (int j = 0; j < n; ++j) {
        const int row = __builtin_amdgcn_readlane(lane_row, j);
        if (row < 0) continue;
#pragma unroll
        for (int u = 0; u < kHeld; ++u)
          if (c0 + kThreads * u < n_chunks)
            C::template store<false>(a.xp + row * row_bytes + (int64_t)(c0 + kThreads * u) * C::kBytes, v[u]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// combine: one wavefront per token and run of 64 chunks. All rows of a batch
// of 8 choices are in flight together. Rows that outgrow the Infinity Cache are
// read non-temporally: 8192 tokens x top-8 x 7168 181 us (5.8 TB/s) against 206;
// smaller ones are not: 1237 x top-6 x 2056 9.1 us against 9.6, 256 x top-8 x
// 7168 7.2 against 7.8. (Two runs per wavefront: 195 and 12.4 us.)
// ---------------------------------------------------------------------------
template <typename Tin, typename Tout, bool kNt>
__global__ __launch_bounds__(64 * kTokWaves) void combine_kernel(
    const uint8_t* __restrict__ c, const int32_t* __restrict__ row_of_slot,
    const float* __restrict__ weights, int n_tok, int K, int topk, int M, int n_runs,
    uint8_t* __restrict__ y) {
  using CI = Chunk<Tin>;
  using CO = Chunk<Tout>;
  const int lane = threadIdx.x & 63;
  const int64_t task = (int64_t)blockIdx.x * kTokWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = task / n_runs;
  if (t >= n_tok) return;
  const int n_chunks = K / 8;
  const int chunk = (int)(task - t * n_runs) * 64 + lane;
  const bool have = chunk < n_chunks;
  const uint8_t* col = c + (int64_t)chunk * CI::kBytes;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  constexpr int kBatch = 8;
  for (int j0 = 0; j0 < topk; j0 += kBatch) {
    int row[kBatch];
    float w[kBatch];
    typename CI::Raw v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      row[u] = -1;
      w[u] = 1.0f;
      if (j0 + u < topk) {
        const int64_t slot = t * topk + j0 + u;
        row[u] = row_of_slot[slot];
        if (weights) w[u] = weights[slot];
        if (row[u] >= M) row[u] = -1;
      }
      if (row[u] >= 0 && have) {
        const uint8_t* at = col + (int64_t)row[u] * n_chunks * CI::kBytes;
        v[u] = kNt ? CI::load_nt(at) : CI::load(at);
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (row[u] < 0) continue;  // wave-uniform
      float f[8];
      CI::floats(v[u], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w[u], f[i], acc[i]);
    }
  }
  if (have) CO::template store<false>(y + (t * n_chunks + chunk) * CO::kBytes, CO::round(acc));
}

// ---------------------------------------------------------------------------
// combine_bwd: one workgroup per token. dy's row is read once per batch of 8
// choices; each choice's row of c is read once, its dot product summed over
// the workgroup in a fixed order, and its row of dc written.
//
// The first pad_parts workgroups of every expert zero the padding rows of its
// block: those past the last row that any slot maps into it, which each finds
// by looking at all slots. They come first in the grid so that this runs beside
// the tokens' copies; as the grid's last workgroups they cost 65 of 429 us at
// 8192 tokens x top-8 of 32 experts, K = 7168. dc is stored non-temporally only
// where it outgrows the Infinity Cache (that case: 364 us against 382; 4096 x
// top-6, K = 2048: 44.8 against 38.7 with ordinary stores).
// ---------------------------------------------------------------------------
template <typename Ty, typename Tc, bool kDw, bool kNt>
__global__ __launch_bounds__(64 * kTokWaves) void combine_bwd_kernel(
    const uint8_t* __restrict__ dy, const uint8_t* __restrict__ c,
    const int32_t* __restrict__ row_of_slot, const float* __restrict__ weights,
    const int32_t* __restrict__ m_offsets, int n_tok, int K, int topk, int M, int n_pad,
    int pad_parts, uint8_t* __restrict__ dc, float* __restrict__ dw) {
  using CY = Chunk<Ty>;
  using CC = Chunk<Tc>;
  constexpr int kThreads = 64 * kTokWaves;
  constexpr int kBatch = 8;
  __shared__ float part[kTokWaves][kBatch];
  __shared__ int last_of_wave[kTokWaves];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n_chunks = K / 8;
  const int64_t rb = (int64_t)n_chunks * CC::kBytes;
  if ((int)blockIdx.x < n_pad) {
    const int e = blockIdx.x / pad_parts;
    const int lo = min(max(m_offsets[e], 0), M);
    const int hi = min(max(m_offsets[e + 1], lo), M);
    if (hi == lo) return;
    int last = lo - 1;
    const int64_t slots = (int64_t)n_tok * topk;
    constexpr int kAtOnce = 8;
    for (int64_t s0 = tid; s0 < slots; s0 += kThreads * kAtOnce) {
      int r[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int64_t s = s0 + u * kThreads;
        r[u] = s < slots ? row_of_slot[s] : -1;
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (r[u] >= lo && r[u] < hi) last = max(last, r[u]);
    }
    last = (int)wave_max_u32((uint32_t)(last + 1)) - 1;
    if (lane == 0) last_of_wave[wave] = last;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTokWaves; ++w) last = max(last, last_of_wave[w]);
    const int64_t n = (int64_t)(hi - 1 - last) * n_chunks;  // contiguous
    for (int64_t i = blockIdx.x % pad_parts * kThreads + tid; i < n; i += pad_parts * kThreads)
      CC::template store<kNt>(dc + (last + 1) * rb + i * CC::kBytes, CC::zero());
    return;
  }
  const int64_t t = blockIdx.x - n_pad;
  for (int j0 = 0; j0 < topk; j0 += kBatch) {
    int row[kBatch];
    float w[kBatch], dot[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      row[u] = -1;
      w[u] = 1.0f;
      dot[u] = 0.0f;
      if (j0 + u < topk) {
        const int64_t slot = t * topk + j0 + u;
        row[u] = row_of_slot[slot];
        if (weights) w[u] = weights[slot];
        if (row[u] >= M) row[u] = -1;
      }
    }
    for (int ch = tid; ch < n_chunks; ch += kThreads) {
      typename CC::Raw v[kBatch];
      if constexpr (kDw) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (row[u] >= 0) v[u] = CC::load_nt(c + (int64_t)row[u] * rb + (int64_t)ch * CC::kBytes);
      }
      float g[8];
      CY::floats(CY::load(dy + (t * n_chunks + ch) * CY::kBytes), g);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (row[u] < 0) continue;  // wave-uniform
        float f[8];
        if constexpr (kDw) {
          CC::floats(v[u], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[u] = __builtin_fmaf(g[i], f[i], dot[u]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = w[u] * g[i];
        CC::template store<kNt>(dc + (int64_t)row[u] * rb + (int64_t)ch * CC::kBytes, CC::round(f));
      }
    }
    if constexpr (kDw) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const float s = wave_sum_f32(dot[u]);
        if (lane == 0) part[wave][u] = s;
      }
      __syncthreads();
      if (tid < kBatch && j0 + tid < topk) {
        float s = part[0][tid];
#pragma unroll
        for (int v = 1; v < kTokWaves; ++v) s += part[v][tid];
        dw[t * topk + j0 + tid] = s;
      }
      __syncthreads();
    }
  }
}

// the dispatch's counting and scanning kernels, and its workspace: histogram,
// first rows, counts
__global__ void dispatch_count_kernel(const int32_t* __restrict__ ids, int S, int G,
                                      int32_t* __restrict__ hist, int32_t* __restrict__ in_block);
__global__ void dispatch_scan_kernel(const int32_t* __restrict__ hist, int n_blk, int G,
                                     int32_t* __restrict__ base, int32_t* __restrict__ counts,
                                     int32_t* __restrict__ m_offsets);
int64_t dispatch_blocks(int64_t slots);

hipError_t launch_moe_permute(const void* x, bool bf16, const int32_t* ids, int64_t T, int64_t K,
                              int64_t topk, int64_t G, void* xp, int32_t* m_offsets,
                              int32_t* row_of_slot, void* workspace, hipStream_t stream) {
  const int64_t slots = T * topk, n_blk = dispatch_blocks(slots);
  int32_t* hist = (int32_t*)workspace;
  int32_t* base = hist + n_blk * G;
  int32_t* counts = base + n_blk * G;
  const Way way = T == 0               ? kScan
                  : slots <= kSortSlots ? kSort
                  : slots <= kCountBlock * kCountBlocks && T <= kCountTokens ? kCount : kScan;
  if (way == kCount) {
    token_count_kernel<<<dim3((unsigned)((slots + kCountBlock - 1) / kCountBlock)), dim3(64 * kCountWaves), 0, stream>>>(
        ids, (int)slots, (int)G, hist, row_of_slot);
  } else if (way == kScan) {
    if (T > 0)
      dispatch_count_kernel<<<dim3((unsigned)n_blk), dim3(kDispBlock), 0, stream>>>(ids, (int)slots, (int)G, hist, row_of_slot);
    dispatch_scan_kernel<<<dim3(1), dim3(kMaxExperts), 0, stream>>>(hist, (int)n_blk, (int)G, base, counts, m_offsets);
    if (T == 0) return hipGetLastError();
  }
  const int64_t parts = std::min<int64_t>(std::max<int64_t>(K * (bf16 ? 2 : 4) / 256, 1), kPadParts);
  const PermuteArgs a{(const uint8_t*)x, ids, hist, base, counts, row_of_slot, m_offsets, (uint8_t*)xp,
                      (int)T, (int)K, (int)topk, (int)G, (int)parts};
  const dim3 grid((unsigned)(T + (K > 0 ? parts * G : 0))), block(64 * kTokWaves);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
  auto by_way = [&](auto t) {
    using E = decltype(t);
    way == kSort    ? go(permute_kernel<E, kSort>)
    : way == kCount ? go(permute_kernel<E, kCount>)
                    : go(permute_kernel<E, kScan>);
  };
  bf16 ? by_way(uint16_t{}) : by_way(float{});
  return hipGetLastError();
}

hipError_t launch_moe_combine(const void* c, bool c_bf16, const int32_t* row_of_slot,
                              const float* weights, int64_t T, int64_t K, int64_t topk, int64_t M,
                              void* y, bool y_bf16, hipStream_t stream) {
  const int64_t n_runs = (K / 8 + 63) / 64;
  const dim3 grid((unsigned)((T * n_runs + kTokWaves - 1) / kTokWaves)), block(64 * kTokWaves);
  const bool nt = T * topk * K * (c_bf16 ? 2 : 4) > (int64_t(256) << 20);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, (const uint8_t*)c, row_of_slot, weights,
                       (int)T, (int)K, (int)topk, (int)M, (int)n_runs, (uint8_t*)y);
  };
  auto by_size = [&](auto tin, auto tout) {
    using Tin = decltype(tin);
    using Tout = decltype(tout);
    nt ? go(combine_kernel<Tin, Tout, true>) : go(combine_kernel<Tin, Tout, false>);
  };
  if (c_bf16) y_bf16 ? by_size(uint16_t{}, uint16_t{}) : by_size(uint16_t{}, float{});
  else y_bf16 ? by_size(float{}, uint16_t{}) : by_size(float{}, float{});
  return hipGetLastError();
}

hipError_t launch_moe_combine_bwd(const void* dy, bool dy_bf16, const void* c, bool c_bf16,
                                  const int32_t* row_of_slot, const float* weights,
                                  const int32_t* m_offsets, int64_t T, int64_t K, int64_t topk,
                                  int64_t G, int64_t M, void* dc, float* dw, hipStream_t stream) {
  // Each padding workgroup reads every slot's row, so many slots get fewer of them
  const int pad_parts = T * topk <= 16384 ? kPadParts : 4;
  const int64_t n_pad = K > 0 && M > 0 ? G * pad_parts : 0;
  if (n_pad + T == 0) return hipSuccess;
  const bool nt = M * K * (c_bf16 ? 2 : 4) > (int64_t(256) << 20);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(n_pad + T)), dim3(64 * kTokWaves), 0, stream,
                       (const uint8_t*)dy, (const uint8_t*)c, row_of_slot, weights, m_offsets, (int)T,
                       (int)K, (int)topk, (int)M, (int)n_pad, pad_parts, (uint8_t*)dc, dw);
  };
  auto by_dw = [&](auto ty, auto tc) {
    using Ty = decltype(ty);
    using Tc = decltype(tc);
    if (dw) nt ? go(combine_bwd_kernel<Ty, Tc, true, true>) : go(combine_bwd_kernel<Ty, Tc, true, false>);
    else nt ? go(combine_bwd_kernel<Ty, Tc, false, true>) : go(combine_bwd_kernel<Ty, Tc, false, false>);
  };
  if (dy_bf16) c_bf16 ? by_dw(uint16_t{}, uint16_t{}) : by_dw(uint16_t{}, float{});
  else c_bf16 ? by_dw(float{}, uint16_t{}) : by_dw(float{}, float{});
  return hipGetLastError();
}

}  // namespace fp8q
