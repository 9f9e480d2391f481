// C ABI of the fp8q library: host-side argument checks, then kernel launches.
// Every check runs before the first HIP call, so a rejected call touches no
// device state and can be exercised without a GPU.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "../../include/fp8q.h"

namespace fp8q {
hipError_t launch_quant_act_1x128(const void* x, int64_t M, int64_t K, uint8_t* q, float* sa,
                                  bool nontemporal, hipStream_t stream);
hipError_t launch_quant_weight_128x128(const void* w, int64_t N, int64_t K, uint8_t* q, float* sb,
                                       hipStream_t stream);
hipError_t launch_gemm_blockscaled(const uint8_t* a, const float* sa, const uint8_t* b,
                                   const float* sb, void* c, bool bf16_out, int64_t M, int64_t N,
                                   int64_t K, hipStream_t stream);
hipError_t launch_gemm_grouped(const uint8_t* a, const float* sa, const uint8_t* b,
                               const float* sb, void* c, bool bf16_out, const int32_t* m_offsets,
                               int64_t G, int64_t M_total, int64_t N, int64_t K,
                               hipStream_t stream);
int64_t splitk_workspace_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm_blockscaled_ws(const uint8_t* a, const float* sa, const uint8_t* b,
                                      const float* sb, void* c, bool bf16_out, int64_t M,
                                      int64_t N, int64_t K, float* ws, hipStream_t stream);
hipError_t launch_gemm_rowscaled(const uint8_t* a, const float* sa, const uint8_t* b,
                                 const float* sb_rows, void* c, bool bf16_out, int64_t M, int64_t N,
                                 int64_t K, hipStream_t stream);
int64_t static_scratch_bytes();
hipError_t launch_gemm_blockscaled_static(const uint8_t* a, const float* sa, const uint8_t* b,
                                          const float* sb, void* c, bool bf16_out, int64_t M,
                                          int64_t N, int64_t K, hipStream_t stream);
hipError_t launch_gemm_quant_a(const void* a, const uint8_t* b, const float* sb, void* c,
                               bool bf16_out, int64_t M, int64_t N, int64_t K, uint8_t* qa,
                               float* sa, hipStream_t stream);
hipError_t launch_quant_act_128x1(const void* x, int64_t M, int64_t K, uint8_t* qt, float* st,
                                  hipStream_t stream);
hipError_t launch_norm_quant_act_1x128(const void* x, const void* gamma, const void* beta,
                                       float eps, bool centred, int64_t M, int64_t K, uint8_t* q,
                                       float* sa, hipStream_t stream);
int64_t dispatch_workspace_bytes(int64_t slots, int64_t G);
hipError_t launch_moe_dispatch(const void* x, const int32_t* ids, int64_t T, int64_t K, int64_t k,
                               int64_t G, uint8_t* q, float* sa, int32_t* m_offsets,
                               int32_t* row_of_slot, void* workspace, hipStream_t stream);
hipError_t launch_quant_act_dual(const void* x, int64_t M, int64_t K, uint8_t* q, float* sa,
                                 uint8_t* qt, float* st, hipStream_t stream);
hipError_t launch_requant_1x128_to_128x1(const uint8_t* q, const float* sa, int64_t M, int64_t K,
                                         uint8_t* qt, float* st, hipStream_t stream);
hipError_t launch_transpose_weight_128x128(const uint8_t* q, const float* sb, int64_t N, int64_t K,
                                           uint8_t* qt, float* sbt, hipStream_t stream);
hipError_t launch_route(const void* logits, bool bf16, const float* bias, int64_t T, int64_t G,
                        int64_t topk, int64_t n_groups, int64_t topk_groups, bool sigmoid,
                        bool renorm, float scale, int32_t* ids, float* w, hipStream_t stream);
hipError_t launch_route_bwd(const void* logits, bool bf16, const int32_t* ids, const float* dw,
                            int64_t T, int64_t G, int64_t topk, bool sigmoid, bool renorm,
                            float scale, void* dlogits, hipStream_t stream);
hipError_t launch_moe_permute(const void* x, bool bf16, const int32_t* ids, int64_t T, int64_t K,
                              int64_t topk, int64_t G, void* xp, int32_t* m_offsets,
                              int32_t* row_of_slot, void* workspace, hipStream_t stream);
hipError_t launch_moe_combine(const void* c, bool c_bf16, const int32_t* row_of_slot,
                              const float* weights, int64_t T, int64_t K, int64_t topk, int64_t M,
                              void* y, bool y_bf16, hipStream_t stream);
hipError_t launch_moe_combine_bwd(const void* dy, bool dy_bf16, const void* c, bool c_bf16,
                                  const int32_t* row_of_slot, const float* weights,
                                  const int32_t* m_offsets, int64_t T, int64_t K, int64_t topk,
                                  int64_t G, int64_t M, void* dc, float* dw, hipStream_t stream);
hipError_t launch_quant_int8_rows(const void* x, int64_t M, int64_t K, int8_t* q, float* s,
                                  hipStream_t stream);
hipError_t launch_int8_gemm(const int8_t* a, const float* sa, const int8_t* b, const float* sb,
                            void* c, bool bf16, int64_t M, int64_t N, int64_t K, hipStream_t stream);
hipError_t launch_int8_gemm_grouped(const int8_t* a, const float* sa, const int8_t* b,
                                    const float* sb, void* c, bool bf16, const int32_t* m_offsets,
                                    int64_t G, int64_t M_total, int64_t N, int64_t K,
                                    hipStream_t stream);
hipError_t launch_norm_rows(const void* x, bool x_bf16, int64_t ldx, const void* res, int64_t ldr,
                            const void* gamma, const void* beta, bool weights_bf16, float eps,
                            bool centred, int64_t M, int64_t K, void* y, bool y_bf16, void* h,
                            hipStream_t stream);
int64_t norm_bwd_workspace_bytes(int64_t M, int64_t K, bool centred);
hipError_t launch_norm_rows_bwd(const void* dy, bool dy_bf16, int64_t ldy, const void* x, bool x_bf16,
                                int64_t ldx, const void* gamma, bool weights_bf16, const void* dres,
                                int64_t ldr, float eps, bool centred, int64_t M, int64_t K, void* dx,
                                float* dgamma, float* dbeta, void* ws, hipStream_t stream);
hipError_t launch_swiglu(const void* gu, bool gu_bf16, int64_t ld, const int32_t* last, int64_t M,
                         int64_t I, void* y, bool y_bf16, hipStream_t stream);
hipError_t launch_swiglu_quant(const void* gu, bool gu_bf16, int64_t ld, const int32_t* last,
                               int64_t M, int64_t I, uint8_t* q, float* sa, hipStream_t stream);
hipError_t launch_swiglu_bwd(const void* dy, bool dy_bf16, int64_t ldy, const void* gu, bool gu_bf16,
                             int64_t ld, const int32_t* last, int64_t M, int64_t I, void* dgu,
                             hipStream_t stream);
int64_t ortho_workspace_bytes(int64_t L, int64_t M, int64_t N, bool single);
hipError_t launch_orthogonalize(const void* g, bool g_bf16, int64_t L, int64_t M, int64_t N, int steps,
                                float a, float b, float c, float scale, void* out, bool out_bf16,
                                bool single, void* ws, hipStream_t stream);
}  // namespace fp8q

namespace {

constexpr int64_t kGroup = 128;
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;  // kernels index rows/cols with int32
// GEMM operand tiles (up to 256 rows of K bytes) are addressed with 32-bit
// offsets through buffer descriptors
constexpr int64_t kMaxK = int64_t(1) << 23;
constexpr int64_t kMaxExperts = 1024;  // dispatch: one scan thread per expert
// the fused normalization keeps a row in one wavefront's registers
constexpr int64_t kNormMaxK = 16384;
constexpr int kMaxDevices = 64;
constexpr int64_t kMaxTopk = 64;    // router: one lane per choice
constexpr int64_t kMaxGroups = 64;  // router: one lane per expert group
// largest K whose int8 sums stay below 2^31 (128 * 128 * K), a multiple of 16
constexpr int64_t kInt8MaxK = 131056;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// 0 = unknown, 1 = gfx950, 2 = other; one slot per device ordinal.
std::atomic<int> g_device_kind[kMaxDevices];

int check_device() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return FP8Q_ERR_NO_DEVICE;
  if (dev >= kMaxDevices) return FP8Q_ERR_NO_DEVICE;
  int kind = g_device_kind[dev].load(std::memory_order_relaxed);
  if (kind == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return FP8Q_ERR_NO_DEVICE;
    kind = (strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    g_device_kind[dev].store(kind, std::memory_order_relaxed);
  }
  return kind == 1 ? FP8Q_OK : FP8Q_ERR_NO_DEVICE;
}

int launched(hipError_t e) { return e == hipSuccess ? FP8Q_OK : FP8Q_ERR_LAUNCH; }

int check_gemm_common(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                      const void* c, int out_dtype, int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0) return FP8Q_ERR_SHAPE;
  if (N % kGroup || K % kGroup) return FP8Q_ERR_SHAPE;
  if (out_dtype != FP8Q_OUT_F32 && out_dtype != FP8Q_OUT_BF16) return FP8Q_ERR_DTYPE;
  if (M > kMaxDim || N > kMaxDim || K > kMaxK) return FP8Q_ERR_TOO_LARGE;
  if ((M + 127) / 128 * (N / 128) > kMaxDim) return FP8Q_ERR_TOO_LARGE;
  if (M == 0 || N == 0) return -1;  // valid no-op
  if (!c) return FP8Q_ERR_NULL;
  if (K > 0 && (!a || !sa || !b || !sb)) return FP8Q_ERR_NULL;  // K == 0 reads no operand
  if (!aligned(c, 16)) return FP8Q_ERR_ALIGN;
  if (K > 0 && (!aligned(a, 16) || !aligned(b, 16) || !aligned(sa, 4) || !aligned(sb, 4)))
    return FP8Q_ERR_ALIGN;
  return FP8Q_OK;
}

// One launch holds less than 2^32 threads.
bool launchable(int64_t workgroups, int64_t threads) { return workgroups * threads < (int64_t(1) << 32); }

bool known_dtype(int d) { return d == FP8Q_OUT_F32 || d == FP8Q_OUT_BF16; }

// Sizes shared by the calls that move rows between tokens and experts.
int check_rows(int64_t T, int64_t K, int64_t topk, int64_t M) {
  if (T < 0 || K < 0 || K % 8 || topk < 1 || M < 0) return FP8Q_ERR_SHAPE;
  if (K > kMaxDim || M > kMaxDim || T > kMaxDim / topk) return FP8Q_ERR_TOO_LARGE;
  return FP8Q_OK;
}

int check_int8(const int8_t* a, const float* sa, const int8_t* b, const float* sb, const void* c,
               int out_dtype, int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0 || K % 16) return FP8Q_ERR_SHAPE;
  if (!known_dtype(out_dtype)) return FP8Q_ERR_DTYPE;
  if (M > kMaxDim || N > kMaxDim || K > kInt8MaxK) return FP8Q_ERR_TOO_LARGE;
  // tiles are numbered with 32 bits; where there are many they are 128 x 128 or
  // larger (16 x 32 for up to 16 rows, by workgroups of 512 threads)
  const int64_t tm = M <= 16 ? 1 : (M + 127) / 128, tn = M <= 16 ? (N + 31) / 32 : (N + 127) / 128;
  if (tm * tn > kMaxDim || !launchable(tm * tn, M <= 16 ? 512 : 256)) return FP8Q_ERR_TOO_LARGE;
  if (M == 0 || N == 0) return -1;  // valid no-op
  if (!c) return FP8Q_ERR_NULL;
  if (K > 0 && (!a || !sa || !b || !sb)) return FP8Q_ERR_NULL;  // K == 0 reads no operand
  if (!aligned(c, 16)) return FP8Q_ERR_ALIGN;
  if (K > 0 && (!aligned(a, 16) || !aligned(b, 16) || !aligned(sa, 4) || !aligned(sb, 4)))
    return FP8Q_ERR_ALIGN;
  return FP8Q_OK;
}

uintptr_t element(int dtype) { return dtype == FP8Q_OUT_BF16 ? 2 : 4; }

// Sizes shared by the normalization's calls.
int check_norm(float eps, int centred, int64_t M, int64_t K) {
  if (M < 0 || K < 0) return FP8Q_ERR_SHAPE;
  if (centred != 0 && centred != 1) return FP8Q_ERR_SHAPE;
  if (!(eps >= 0.0f) || eps > 3.0e38f) return FP8Q_ERR_SHAPE;  // NaN, negative or infinite
  // at most 512 threads per row, or 1024 for the longest (rows of up to 1024 values take 64, but one limit
  // for all of the shorter ones is easier to know)
  if (M > kMaxDim || K > kNormMaxK || !launchable(M, K > 12288 ? 1024 : 512)) return FP8Q_ERR_TOO_LARGE;
  return FP8Q_OK;
}

// Sizes and offsets shared by the gated activation's calls.
int check_swiglu(int gu_dtype, int64_t ld, const int32_t* m_offsets, int64_t G, int64_t M, int64_t I) {
  if (M < 0 || I < 0 || (m_offsets && G < 1)) return FP8Q_ERR_SHAPE;
  if (!known_dtype(gu_dtype)) return FP8Q_ERR_DTYPE;
  if (M > kMaxDim || I > kMaxDim / 2 || (m_offsets && G > kMaxDim)) return FP8Q_ERR_TOO_LARGE;
  if (M * ((I + 7) / 8) > kMaxDim - 256) return FP8Q_ERR_TOO_LARGE;  // chunks of 8, numbered with 31 bits
  if (M == 0 || I == 0) return -1;  // valid no-op
  if (ld < 2 * I) return FP8Q_ERR_SHAPE;
  if (!aligned(m_offsets, 4)) return FP8Q_ERR_ALIGN;
  return FP8Q_OK;
}

// Sizes of the orthogonalization.
int check_ortho(int64_t L, int64_t M, int64_t N) {
  if (L < 0 || M < 0 || N < 0) return FP8Q_ERR_SHAPE;
  if (L > 65535 || M > 65536 || N > 65536) return FP8Q_ERR_TOO_LARGE;
  // one workgroup of 256 threads per 64 x 64 values, padded
  if (!launchable(L * ((M + 63) / 64) * ((N + 63) / 64), 256)) return FP8Q_ERR_TOO_LARGE;
  if (L == 0 || M == 0 || N == 0) return -1;  // valid no-op
  return FP8Q_OK;
}

// Whether s <- a s + b s^3 + c s^5 keeps [0, 1] below 3, and b s^2 + c s^4 within 7.5,
// for `steps` steps: the FP16 planes' scales count on it. The largest |p| over
// [0, top] is at the end or where p' = a + 3 b s^2 + 5 c s^4 is zero, the other's at the
// end or at s^2 = -b / 2c.
bool bounded(int steps, double a, double b, double c) {
  if (!isfinite(a) || !isfinite(b) || !isfinite(c)) return false;
  auto p = [&](double s) { return fabs(s * (a + s * s * (b + s * s * c))); };
  auto q = [&](double t) { return fabs(t * (b + t * c)); };
  double top = 1.0;
  for (int k = 0; k < steps; ++k) {
    const double t1 = top * top;
    double most = p(top), inner = q(t1);
    if (const double t = -b / (2 * c); t > 0 && t < t1) inner = fmax(inner, q(t));
    const double disc = 9 * b * b - 20 * a * c;
    if (disc >= 0) {
      // (5 c and a over the larger root's numerator: nothing cancels, whatever is near zero)
      const double r = -0.5 * (3 * b + copysign(sqrt(disc), b));
      for (double t : {r / (5 * c), a / r})
        if (t > 0 && t < t1) most = fmax(most, p(sqrt(t)));
    }
    if (inner > 7.5 || most > 3.0) return false;
    top = most;
  }
  return true;
}

// Both forms of the orthogonalization; `single`: of one FP16 number a value, for a bfloat16 out.
int orthogonalize(const void* g, int g_dtype, int64_t L, int64_t M, int64_t N, int steps, float a, float b, float c,
                  float scale, void* out, bool bf16, bool single, void* workspace, int64_t workspace_bytes,
                  void* stream) {
  if (!known_dtype(g_dtype)) return FP8Q_ERR_DTYPE;
  if (steps < 1 || steps > 100 || !isfinite(scale) || !bounded(steps, a, b, c)) return FP8Q_ERR_SHAPE;
  int s = check_ortho(L, M, N);
  if (s == -1) return FP8Q_OK;
  if (s) return s;
  const int64_t need = fp8q::ortho_workspace_bytes(L, M, N, single);
  if (!g || !out || (need && !workspace)) return FP8Q_ERR_NULL;
  if (workspace_bytes < need) return FP8Q_ERR_SHAPE;
  if (!aligned(g, element(g_dtype)) || !aligned(out, bf16 ? 2 : 4) || !aligned(workspace, 16)) return FP8Q_ERR_ALIGN;
  if ((s = check_device())) return s;
  return launched(fp8q::launch_orthogonalize(g, g_dtype == FP8Q_OUT_BF16, L, M, N, steps, a, b, c, scale, out, bf16,
                                             single, workspace, (hipStream_t)stream));
}

// worst-case m_offsets[G] of the MoE dispatch (every expert padded by 127
// rows), rounded up to a multiple of 128 so that it is a valid M_total for
// the grouped GEMM
int64_t dispatch_max_rows(int64_t T, int64_t topk, int64_t G) {
  return (T * topk + (kGroup - 1) * G + kGroup - 1) / kGroup * kGroup;
}

// Checks shared by the three 128 x 128 tile re-tiling calls (R x C -> C x R).
int check_retile(const void* in, const float* in_s, bool need_in_s, int64_t R, int64_t C,
                 const uint8_t* out, const float* out_s) {
  if (R < 0 || C < 0 || R % kGroup || C % kGroup) return FP8Q_ERR_SHAPE;
  if (R > kMaxDim || C > kMaxDim || C / kGroup > 65535) return FP8Q_ERR_TOO_LARGE;
  if (R == 0 || C == 0) return -1;  // valid no-op
  if (!in || !out || !out_s || (need_in_s && !in_s)) return FP8Q_ERR_NULL;
  if (!aligned(in, 16) || !aligned(out, 16) || !aligned(out_s, 4)) return FP8Q_ERR_ALIGN;
  if (need_in_s && !aligned(in_s, 4)) return FP8Q_ERR_ALIGN;
  return FP8Q_OK;
}

}  // namespace

extern "C" {

int fp8q_version(void) { return 202; }

const char* fp8q_status_string(int status) {
  switch (status) {
    case FP8Q_OK: return "ok";
    case FP8Q_ERR_NULL: return "a required pointer is NULL";
    case FP8Q_ERR_SHAPE: return "invalid shape (negative size, K or N not a multiple of 128, or G < 1)";
    case FP8Q_ERR_ALIGN: return "misaligned pointer (16 bytes for data, 4 bytes for scales)";
    case FP8Q_ERR_DTYPE: return "unknown output dtype";
    case FP8Q_ERR_LAUNCH: return "kernel launch failed";
    case FP8Q_ERR_NO_DEVICE: return "no gfx950 device is current";
    case FP8Q_ERR_TOO_LARGE: return "size exceeds the kernels' 32-bit indexing";
    case FP8Q_ERR_SCRATCH: return "the split-K partials exceed the library's static scratch (8 MiB)";
    default: return "unknown status";
  }
}

static int quant_act_1x128(const void* x_bf16, int64_t M, int64_t K, uint8_t* q, float* sa,
                           bool nontemporal, void* stream) {
  if (M < 0 || K < 0 || K % kGroup) return FP8Q_ERR_SHAPE;
  if (M > kMaxDim || K > kMaxDim || M * (K / kGroup) > (kMaxDim / 16)) return FP8Q_ERR_TOO_LARGE;
  if (M == 0 || K == 0) return FP8Q_OK;
  if (!x_bf16 || !q || !sa) return FP8Q_ERR_NULL;
  if (!aligned(x_bf16, 16) || !aligned(q, 16) || !aligned(sa, 4)) return FP8Q_ERR_ALIGN;
  if (int s = check_device()) return s;
  return launched(fp8q::launch_quant_act_1x128(x_bf16, M, K, q, sa, nontemporal, (hipStream_t)stream));
}

int fp8q_quant_act_1x128(const void* x_bf16, int64_t M, int64_t K, uint8_t* q, float* sa,
                         void* stream) {
  return quant_act_1x128(x_bf16, M, K, q, sa, false, stream);
}

int fp8q_quant_act_1x128_nt(const void* x_bf16, int64_t M, int64_t K, uint8_t* q, float* sa,
                            void* stream) {
  return quant_act_1x128(x_bf16, M, K, q, sa, true, stream);
}

int fp8q_quant_weight_128x128(const void* w_bf16, int64_t N, int64_t K, uint8_t* q, float* sb,
                              void* stream) {
  if (N < 0 || K < 0 || N % kGroup || K % kGroup) return FP8Q_ERR_SHAPE;
  if (N / kGroup > 65535 || K > kMaxDim) return FP8Q_ERR_TOO_LARGE;
  if (N == 0 || K == 0) return FP8Q_OK;
  if (!w_bf16 || !q || !sb) return FP8Q_ERR_NULL;
  if (!aligned(w_bf16, 16) || !aligned(q, 16) || !aligned(sb, 4)) return FP8Q_ERR_ALIGN;
  if (int s = check_device()) return s;
  return launched(fp8q::launch_quant_weight_128x128(w_bf16, N, K, q, sb, (hipStream_t)stream));
}

int fp8_gemm_blockscaled(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                         void* c, int out_dtype, int64_t M, int64_t N, int64_t K, void* stream) {
  int s = check_gemm_common(a, sa, b, sb, c, out_dtype, M, N, K);
  if (s == -1) return FP8Q_OK;
  if (s) return s;
  if ((s = check_device())) return s;
  return launched(fp8q::launch_gemm_blockscaled(a, sa, b, sb, c, out_dtype == FP8Q_OUT_BF16, M, N,
                                                K, (hipStream_t)stream));
}

int fp8_gemm_blockscaled_bf16a(const void* a, const uint8_t* b, const float* sb, void* c,
                               int out_dtype, int64_t M, int64_t N, int64_t K, uint8_t* qa, float* sa,
                               void* stream) {
  if (M < 0 || N < 0 || K < 0) return FP8Q_ERR_SHAPE;
  if (N % kGroup || K % kGroup) return FP8Q_ERR_SHAPE;
  if (out_dtype != FP8Q_OUT_F32 && out_dtype != FP8Q_OUT_BF16) return FP8Q_ERR_DTYPE;
  if (M > kMaxDim || N > kMaxDim || K > kMaxK) return FP8Q_ERR_TOO_LARGE;
  if ((M + 127) / 128 * ((N + 255) / 256) > kMaxDim) return FP8Q_ERR_TOO_LARGE;
  if (M == 0 || N == 0) return FP8Q_OK;  // valid no-op (no outputs written)
  if (!c) return FP8Q_ERR_NULL;
  if ((qa == nullptr) != (sa == nullptr)) return FP8Q_ERR_NULL;  // both outputs or neither
  if (K > 0 && (!a || !b || !sb)) return FP8Q_ERR_NULL;         // K == 0 reads no operand
  if (!aligned(c, 16)) return FP8Q_ERR_ALIGN;
  if (K > 0 && (!aligned(a, 16) || !aligned(b, 16) || !aligned(sb, 4))) return FP8Q_ERR_ALIGN;
  if (qa && (!aligned(qa, 16) || !aligned(sa, 4))) return FP8Q_ERR_ALIGN;
  int s;
  if ((s = check_device())) return s;
  return launched(fp8q::launch_gemm_quant_a(a, b, sb, c, out_dtype == FP8Q_OUT_BF16, M, N, K,
                                            K > 0 ? qa : nullptr, K > 0 ? sa : nullptr,
                                            (hipStream_t)stream));
}

int64_t fp8_gemm_blockscaled_ws_bytes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0 || N % kGroup || K % kGroup) return -1;
  if (M > kMaxDim || N > kMaxDim || K > kMaxK) return -1;
  return fp8q::splitk_workspace_bytes(M, N, K);
}

int fp8_gemm_blockscaled_ws(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                            void* c, int out_dtype, int64_t M, int64_t N, int64_t K,
                            void* workspace, int64_t workspace_bytes, void* stream) {
  int s = check_gemm_common(a, sa, b, sb, c, out_dtype, M, N, K);
  if (s == -1) return FP8Q_OK;
  if (s) return s;
  const int64_t need = fp8q::splitk_workspace_bytes(M, N, K);
  if (need > 0) {
    if (!workspace) return FP8Q_ERR_NULL;
    if (workspace_bytes < need) return FP8Q_ERR_SHAPE;
    if (!aligned(workspace, 16)) return FP8Q_ERR_ALIGN;
  }
  if ((s = check_device())) return s;
  return launched(fp8q::launch_gemm_blockscaled_ws(a, sa, b, sb, c, out_dtype == FP8Q_OUT_BF16, M, N,
                                                   K, need > 0 ? (float*)workspace : nullptr,
                                                   (hipStream_t)stream));
}

int fp8_gemm_blockscaled_noalloc(const uint8_t* a, const float* sa, const uint8_t* b,
                                 const float* sb, void* c, int out_dtype, int64_t M, int64_t N,
                                 int64_t K, void* stream) {
  int s = check_gemm_common(a, sa, b, sb, c, out_dtype, M, N, K);
  if (s == -1) return FP8Q_OK;
  if (s) return s;
  if (fp8q::splitk_workspace_bytes(M, N, K) > fp8q::static_scratch_bytes()) return FP8Q_ERR_SCRATCH;
  if ((s = check_device())) return s;
  return launched(fp8q::launch_gemm_blockscaled_static(a, sa, b, sb, c, out_dtype == FP8Q_OUT_BF16,
                                                       M, N, K, (hipStream_t)stream));
}

int fp8_gemm_grouped(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                     void* c, int out_dtype, const int32_t* m_offsets, int64_t G, int64_t M_total,
                     int64_t N, int64_t K, void* stream) {
  if (G < 1) return FP8Q_ERR_SHAPE;
  if (M_total % kGroup) return FP8Q_ERR_SHAPE;
  if (G > kMaxDim || G * N > kMaxDim) return FP8Q_ERR_TOO_LARGE;
  int s = check_gemm_common(a, sa, b, sb, c, out_dtype, M_total, N, K);
  if (s == -1) return FP8Q_OK;
  if (s) return s;
  if (!m_offsets) return FP8Q_ERR_NULL;
  if (!aligned(m_offsets, 4)) return FP8Q_ERR_ALIGN;
  if ((s = check_device())) return s;
  return launched(fp8q::launch_gemm_grouped(a, sa, b, sb, c, out_dtype == FP8Q_OUT_BF16,
                                            m_offsets, G, M_total, N, K, (hipStream_t)stream));
}

int fp8q_quant_act_128x1(const void* x_bf16, int64_t M, int64_t K, uint8_t* qt, float* st,
                         void* stream) {
  int s = check_retile(x_bf16, nullptr, false, M, K, qt, st);
  if (s == -1) return FP8Q_OK;
  if (s || (s = check_device())) return s;
  return launched(fp8q::launch_quant_act_128x1(x_bf16, M, K, qt, st, (hipStream_t)stream));
}

int64_t fp8q_moe_dispatch_workspace_bytes(int64_t T, int64_t topk, int64_t G) {
  if (T < 0 || topk < 1 || G < 1 || G > kMaxExperts) return -1;
  if (T > kMaxDim / topk) return -1;
  return fp8q::dispatch_workspace_bytes(T * topk, G);
}

int64_t fp8q_moe_dispatch_max_rows(int64_t T, int64_t topk, int64_t G) {
  if (T < 0 || topk < 1 || G < 1 || G > kMaxExperts) return -1;
  if (T > kMaxDim / topk) return -1;
  return dispatch_max_rows(T, topk, G);
}

int fp8q_moe_dispatch_1x128(const void* x_bf16, const int32_t* topk_ids, int64_t T, int64_t K,
                            int64_t topk, int64_t G, uint8_t* q, float* sa, int64_t M_cap,
                            int32_t* m_offsets, int32_t* row_of_slot, void* workspace,
                            int64_t workspace_bytes, void* stream) {
  if (T < 0 || K < 0 || K % kGroup || topk < 1 || G < 1) return FP8Q_ERR_SHAPE;
  if (G > kMaxExperts || K > kMaxDim || T > kMaxDim / topk) return FP8Q_ERR_TOO_LARGE;
  const int64_t need_rows = dispatch_max_rows(T, topk, G);
  if (need_rows > kMaxDim || T > kMaxDim / 4) return FP8Q_ERR_TOO_LARGE;
  if (M_cap < need_rows) return FP8Q_ERR_SHAPE;  // outputs too small for the worst-case padding
  if (!m_offsets || !workspace) return FP8Q_ERR_NULL;
  if (T > 0 && (!topk_ids || !row_of_slot)) return FP8Q_ERR_NULL;
  if (K > 0 && (!q || !sa || (T > 0 && !x_bf16))) return FP8Q_ERR_NULL;
  if (workspace_bytes < fp8q::dispatch_workspace_bytes(T * topk, G)) return FP8Q_ERR_SHAPE;
  if (!aligned(m_offsets, 4) || !aligned(workspace, 4)) return FP8Q_ERR_ALIGN;
  if (T > 0 && (!aligned(topk_ids, 4) || !aligned(row_of_slot, 4))) return FP8Q_ERR_ALIGN;
  if (K > 0 && (!aligned(q, 16) || !aligned(sa, 4) || (T > 0 && !aligned(x_bf16, 16))))
    return FP8Q_ERR_ALIGN;
  if (int s = check_device()) return s;
  return launched(fp8q::launch_moe_dispatch(x_bf16, topk_ids, T, K, topk, G, q, sa, m_offsets,
                                            row_of_slot, workspace, (hipStream_t)stream));
}

int fp8q_norm_quant_act_1x128(const void* x_bf16, const void* gamma_bf16, const void* beta_bf16,
                              float eps, int centred, int64_t M, int64_t K, uint8_t* q, float* sa,
                              void* stream) {
  if (M < 0 || K < 0 || K % kGroup) return FP8Q_ERR_SHAPE;
  if (centred != 0 && centred != 1) return FP8Q_ERR_SHAPE;
  if (!(eps >= 0.0f) || eps > 3.0e38f) return FP8Q_ERR_SHAPE;  // NaN, negative or infinite
  if (M > kMaxDim || K > kNormMaxK) return FP8Q_ERR_TOO_LARGE;
  if (M == 0 || K == 0) return FP8Q_OK;
  if (!x_bf16 || !gamma_bf16 || !q || !sa || (centred && !beta_bf16)) return FP8Q_ERR_NULL;
  if (!aligned(x_bf16, 16) || !aligned(gamma_bf16, 16) || !aligned(q, 16) || !aligned(sa, 4))
    return FP8Q_ERR_ALIGN;
  if (centred && !aligned(beta_bf16, 16)) return FP8Q_ERR_ALIGN;
  if (int s = check_device()) return s;
  return launched(fp8q::launch_norm_quant_act_1x128(x_bf16, gamma_bf16, beta_bf16, eps,
                                                    centred == 1, M, K, q, sa,
                                                    (hipStream_t)stream));
}

int fp8q_quant_act_1x128_128x1(const void* x_bf16, int64_t M, int64_t K, uint8_t* q, float* sa,
                               uint8_t* qt, float* st, void* stream) {
  int s = check_retile(x_bf16, nullptr, false, M, K, qt, st);
  if (s == -1) return FP8Q_OK;
  if (s) return s;
  if (!q || !sa) return FP8Q_ERR_NULL;
  if (!aligned(q, 16) || !aligned(sa, 4)) return FP8Q_ERR_ALIGN;
  if ((s = check_device())) return s;
  return launched(fp8q::launch_quant_act_dual(x_bf16, M, K, q, sa, qt, st, (hipStream_t)stream));
}

int fp8q_requant_1x128_to_128x1(const uint8_t* q, const float* sa, int64_t M, int64_t K,
                                uint8_t* qt, float* st, void* stream) {
  int s = check_retile(q, sa, true, M, K, qt, st);
  if (s == -1) return FP8Q_OK;
  if (s || (s = check_device())) return s;
  return launched(fp8q::launch_requant_1x128_to_128x1(q, sa, M, K, qt, st, (hipStream_t)stream));
}

int fp8q_transpose_weight_128x128(const uint8_t* q, const float* sb, int64_t N, int64_t K,
                                  uint8_t* qt, float* sbt, void* stream) {
  int s = check_retile(q, sb, true, N, K, qt, sbt);
  if (s == -1) return FP8Q_OK;
  if (s || (s = check_device())) return s;
  return launched(fp8q::launch_transpose_weight_128x128(q, sb, N, K, qt, sbt, (hipStream_t)stream));
}

int fp8_gemm_rowscaled(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                       void* c, int out_dtype, int64_t M, int64_t N, int64_t K, void* stream) {
  int s = check_gemm_common(a, sa, b, sb, c, out_dtype, M, N, K);
  if (s == -1) return FP8Q_OK;
  if (s) return s;
  if ((s = check_device())) return s;
  return launched(fp8q::launch_gemm_rowscaled(a, sa, b, sb, c, out_dtype == FP8Q_OUT_BF16, M, N, K,
                                              (hipStream_t)stream));
}

int fp8q_moe_route(const void* logits, int dtype, const float* bias, int64_t T, int64_t G,
                   int64_t topk, int64_t n_groups, int64_t topk_groups, int score, int renormalize,
                   float scale, int32_t* topk_ids, float* weights, void* stream) {
  if (T < 0 || G < 1 || topk < 1 || n_groups < 1 || topk_groups < 1 || topk_groups > n_groups)
    return FP8Q_ERR_SHAPE;
  if (G > kMaxExperts || topk > kMaxTopk || n_groups > kMaxGroups || T > kMaxDim / topk)
    return FP8Q_ERR_TOO_LARGE;
  if (!launchable((T + 3) / 4, 256)) return FP8Q_ERR_TOO_LARGE;
  if (G % n_groups || topk > topk_groups * (G / n_groups)) return FP8Q_ERR_SHAPE;
  if (score != FP8Q_SCORE_SOFTMAX && score != FP8Q_SCORE_SIGMOID) return FP8Q_ERR_SHAPE;
  if (renormalize != 0 && renormalize != 1) return FP8Q_ERR_SHAPE;
  if (!(scale >= -3.4e38f && scale <= 3.4e38f)) return FP8Q_ERR_SHAPE;  // NaN or infinite
  if (!known_dtype(dtype)) return FP8Q_ERR_DTYPE;
  if (T == 0) return FP8Q_OK;
  if (!logits || !topk_ids || !weights) return FP8Q_ERR_NULL;
  if (!aligned(logits, dtype == FP8Q_OUT_BF16 ? 2 : 4) || !aligned(bias, 4) || !aligned(topk_ids, 4) ||
      !aligned(weights, 4))
    return FP8Q_ERR_ALIGN;
  if (int s = check_device()) return s;
  return launched(fp8q::launch_route(logits, dtype == FP8Q_OUT_BF16, bias, T, G, topk, n_groups,
                                     topk_groups, score == FP8Q_SCORE_SIGMOID, renormalize == 1,
                                     scale, topk_ids, weights, (hipStream_t)stream));
}

int fp8q_moe_route_bwd(const void* logits, int dtype, const int32_t* topk_ids, const float* dweights,
                       int64_t T, int64_t G, int64_t topk, int score, int renormalize, float scale,
                       void* dlogits, void* stream) {
  if (T < 0 || G < 1 || topk < 1) return FP8Q_ERR_SHAPE;
  if (G > kMaxExperts || topk > kMaxTopk || T > kMaxDim / topk) return FP8Q_ERR_TOO_LARGE;
  if (!launchable((T + 3) / 4, 256)) return FP8Q_ERR_TOO_LARGE;
  if (score != FP8Q_SCORE_SOFTMAX && score != FP8Q_SCORE_SIGMOID) return FP8Q_ERR_SHAPE;
  if (renormalize != 0 && renormalize != 1) return FP8Q_ERR_SHAPE;
  if (!(scale >= -3.4e38f && scale <= 3.4e38f)) return FP8Q_ERR_SHAPE;
  if (!known_dtype(dtype)) return FP8Q_ERR_DTYPE;
  if (T == 0) return FP8Q_OK;
  if (!logits || !topk_ids || !dweights || !dlogits) return FP8Q_ERR_NULL;
  const uintptr_t al = dtype == FP8Q_OUT_BF16 ? 2 : 4;
  if (!aligned(logits, al) || !aligned(dlogits, al) || !aligned(topk_ids, 4) || !aligned(dweights, 4))
    return FP8Q_ERR_ALIGN;
  if (int s = check_device()) return s;
  return launched(fp8q::launch_route_bwd(logits, dtype == FP8Q_OUT_BF16, topk_ids, dweights, T, G, topk,
                                         score == FP8Q_SCORE_SIGMOID, renormalize == 1, scale,
                                         dlogits, (hipStream_t)stream));
}

int fp8q_moe_permute(const void* x, int dtype, const int32_t* topk_ids, int64_t T, int64_t K,
                     int64_t topk, int64_t G, void* xp, int64_t M_cap, int32_t* m_offsets,
                     int32_t* row_of_slot, void* workspace, int64_t workspace_bytes, void* stream) {
  int s = check_rows(T, K, topk, M_cap);
  if (s) return s;
  if (G < 1) return FP8Q_ERR_SHAPE;
  if (!known_dtype(dtype)) return FP8Q_ERR_DTYPE;
  if (G > kMaxExperts || !launchable(T + 16 * G, 256)) return FP8Q_ERR_TOO_LARGE;
  const int64_t need_rows = dispatch_max_rows(T, topk, G);
  if (need_rows > kMaxDim) return FP8Q_ERR_TOO_LARGE;
  if (M_cap < need_rows) return FP8Q_ERR_SHAPE;  // outputs too small for the worst-case padding
  if (!m_offsets || !workspace) return FP8Q_ERR_NULL;
  if (T > 0 && (!topk_ids || !row_of_slot)) return FP8Q_ERR_NULL;
  if (K > 0 && T > 0 && (!x || !xp)) return FP8Q_ERR_NULL;
  if (workspace_bytes < fp8q::dispatch_workspace_bytes(T * topk, G)) return FP8Q_ERR_SHAPE;
  if (!aligned(m_offsets, 4) || !aligned(workspace, 4)) return FP8Q_ERR_ALIGN;
  if (T > 0 && (!aligned(topk_ids, 4) || !aligned(row_of_slot, 4))) return FP8Q_ERR_ALIGN;
  if (K > 0 && T > 0 && (!aligned(x, 16) || !aligned(xp, 16))) return FP8Q_ERR_ALIGN;
  if ((s = check_device())) return s;
  return launched(fp8q::launch_moe_permute(x, dtype == FP8Q_OUT_BF16, topk_ids, T, K, topk, G, xp,
                                           m_offsets, row_of_slot, workspace, (hipStream_t)stream));
}

int fp8q_moe_combine(const void* c, int c_dtype, const int32_t* row_of_slot, const float* weights,
                     int64_t T, int64_t K, int64_t topk, int64_t M, void* y, int y_dtype,
                     void* stream) {
  int s = check_rows(T, K, topk, M);
  if (s) return s;
  if (!known_dtype(c_dtype) || !known_dtype(y_dtype)) return FP8Q_ERR_DTYPE;
  if (T > 0 && !launchable((T * ((K / 8 + 63) / 64) + 3) / 4, 256)) return FP8Q_ERR_TOO_LARGE;
  if (T == 0 || K == 0) return FP8Q_OK;
  if (!row_of_slot || !y || (M > 0 && !c)) return FP8Q_ERR_NULL;
  if (!aligned(c, 16) || !aligned(y, 16) || !aligned(row_of_slot, 4) || !aligned(weights, 4))
    return FP8Q_ERR_ALIGN;
  if ((s = check_device())) return s;
  return launched(fp8q::launch_moe_combine(c, c_dtype == FP8Q_OUT_BF16, row_of_slot, weights, T, K,
                                           topk, M, y, y_dtype == FP8Q_OUT_BF16,
                                           (hipStream_t)stream));
}

int fp8q_moe_combine_bwd(const void* dy, int dy_dtype, const void* c, int c_dtype,
                         const int32_t* row_of_slot, const float* weights,
                         const int32_t* m_offsets, int64_t T, int64_t K, int64_t topk, int64_t G,
                         int64_t M, void* dc, float* dw, void* stream) {
  int s = check_rows(T, K, topk, M);
  if (s) return s;
  if (G < 1) return FP8Q_ERR_SHAPE;
  if (!known_dtype(dy_dtype) || !known_dtype(c_dtype)) return FP8Q_ERR_DTYPE;
  if (G > kMaxExperts || !launchable(T + 16 * G, 256)) return FP8Q_ERR_TOO_LARGE;
  if (!m_offsets || (T > 0 && !row_of_slot)) return FP8Q_ERR_NULL;
  if (K > 0 && ((T > 0 && !dy) || (M > 0 && !dc) || (M > 0 && T > 0 && dw && !c))) return FP8Q_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(c, 16) || !aligned(dc, 16) || !aligned(row_of_slot, 4) ||
      !aligned(weights, 4) || !aligned(m_offsets, 4) || !aligned(dw, 4))
    return FP8Q_ERR_ALIGN;
  if ((s = check_device())) return s;
  return launched(fp8q::launch_moe_combine_bwd(dy, dy_dtype == FP8Q_OUT_BF16, c,
                                               c_dtype == FP8Q_OUT_BF16, row_of_slot, weights,
                                               m_offsets, T, K, topk, G, M, dc, dw,
                                               (hipStream_t)stream));
}

int fp8q_quant_int8_rows(const void* x_bf16, int64_t M, int64_t K, int8_t* q, float* s,
                         void* stream) {
  if (M < 0 || K < 0 || K % 16) return FP8Q_ERR_SHAPE;
  if (M > kMaxDim || K > kMaxDim || !launchable(K <= 2048 ? (M + 3) / 4 : M, 256)) return FP8Q_ERR_TOO_LARGE;
  if (M == 0) return FP8Q_OK;
  if (!s || (K > 0 && (!x_bf16 || !q))) return FP8Q_ERR_NULL;
  if (!aligned(x_bf16, 16) || !aligned(q, 16) || !aligned(s, 4)) return FP8Q_ERR_ALIGN;
  if (int st = check_device()) return st;
  return launched(fp8q::launch_quant_int8_rows(x_bf16, M, K, q, s, (hipStream_t)stream));
}

int int8_gemm_scaled(const int8_t* a, const float* sa, const int8_t* b, const float* sb, void* c,
                     int out_dtype, int64_t M, int64_t N, int64_t K, void* stream) {
  int s = check_int8(a, sa, b, sb, c, out_dtype, M, N, K);
  if (s == -1) return FP8Q_OK;
  if (s || (s = check_device())) return s;
  return launched(fp8q::launch_int8_gemm(a, sa, b, sb, c, out_dtype == FP8Q_OUT_BF16, M, N, K,
                                         (hipStream_t)stream));
}

int int8_gemm_grouped(const int8_t* a, const float* sa, const int8_t* b, const float* sb, void* c,
                      int out_dtype, const int32_t* m_offsets, int64_t G, int64_t M_total, int64_t N,
                      int64_t K, void* stream) {
  if (G < 1 || M_total % kGroup) return FP8Q_ERR_SHAPE;
  if (G > kMaxDim || N > kMaxDim || G * N > kMaxDim) return FP8Q_ERR_TOO_LARGE;
  int s = check_int8(a, sa, b, sb, c, out_dtype, M_total, N, K);
  if (s == -1) return FP8Q_OK;
  if (s) return s;
  // the grid holds up to one more tile row per expert
  if (!launchable((M_total / kGroup + G + 1) * ((N + 127) / 128), 256)) return FP8Q_ERR_TOO_LARGE;
  if (!m_offsets) return FP8Q_ERR_NULL;
  if (!aligned(m_offsets, 4)) return FP8Q_ERR_ALIGN;
  if ((s = check_device())) return s;
  return launched(fp8q::launch_int8_gemm_grouped(a, sa, b, sb, c, out_dtype == FP8Q_OUT_BF16,
                                                 m_offsets, G, M_total, N, K, (hipStream_t)stream));
}

int fp8q_norm(const void* x, int x_dtype, int64_t ldx, const void* residual, int64_t ldr,
              const void* gamma, const void* beta, int weights_dtype, float eps, int centred, int64_t M,
              int64_t K, void* y, int y_dtype, void* h, void* stream) {
  int s = check_norm(eps, centred, M, K);
  if (s) return s;
  if (!known_dtype(x_dtype) || !known_dtype(weights_dtype) || !known_dtype(y_dtype)) return FP8Q_ERR_DTYPE;
  if (beta && !centred) return FP8Q_ERR_SHAPE;
  if (M == 0 || K == 0) return FP8Q_OK;
  if (!x || !gamma || !y || (residual == nullptr) != (h == nullptr)) return FP8Q_ERR_NULL;
  if (ldx < K || (residual && ldr < K)) return FP8Q_ERR_SHAPE;
  const uintptr_t ex = element(x_dtype), ew = element(weights_dtype);
  if (!aligned(x, ex) || !aligned(residual, ex) || !aligned(h, ex) || !aligned(gamma, ew) ||
      !aligned(beta, ew) || !aligned(y, element(y_dtype)))
    return FP8Q_ERR_ALIGN;
  if ((s = check_device())) return s;
  return launched(fp8q::launch_norm_rows(x, x_dtype == FP8Q_OUT_BF16, ldx, residual, ldr, gamma, beta,
                                         weights_dtype == FP8Q_OUT_BF16, eps, centred == 1, M, K, y,
                                         y_dtype == FP8Q_OUT_BF16, h, (hipStream_t)stream));
}

int64_t fp8q_norm_bwd_workspace_bytes(int64_t M, int64_t K, int centred) {
  if (check_norm(0.0f, centred, M, K)) return -1;
  return fp8q::norm_bwd_workspace_bytes(M, K, centred == 1);
}

int fp8q_norm_bwd(const void* dy, int dy_dtype, int64_t ldy, const void* x, int x_dtype, int64_t ldx,
                  const void* gamma, int weights_dtype, const void* dres, int64_t ldr, float eps,
                  int centred, int64_t M, int64_t K, void* dx, float* dgamma, float* dbeta,
                  void* workspace, int64_t workspace_bytes, void* stream) {
  int s = check_norm(eps, centred, M, K);
  if (s) return s;
  if (!known_dtype(dy_dtype) || !known_dtype(x_dtype) || !known_dtype(weights_dtype)) return FP8Q_ERR_DTYPE;
  if (K == 0) return FP8Q_OK;
  if (!gamma || !dgamma || (dbeta != nullptr) != (centred == 1)) return FP8Q_ERR_NULL;
  const int64_t need = fp8q::norm_bwd_workspace_bytes(M, K, centred == 1);
  if (M > 0) {
    if (!dy || !x || !dx || !workspace) return FP8Q_ERR_NULL;
    if (ldy < K || ldx < K || (dres && ldr < K) || workspace_bytes < need) return FP8Q_ERR_SHAPE;
  }
  const uintptr_t ex = element(x_dtype);
  if (!aligned(dy, element(dy_dtype)) || !aligned(x, ex) || !aligned(dres, ex) || !aligned(dx, ex) ||
      !aligned(gamma, element(weights_dtype)) || !aligned(dgamma, 4) || !aligned(dbeta, 4) ||
      !aligned(workspace, 16))
    return FP8Q_ERR_ALIGN;
  if ((s = check_device())) return s;
  return launched(fp8q::launch_norm_rows_bwd(dy, dy_dtype == FP8Q_OUT_BF16, ldy, x, x_dtype == FP8Q_OUT_BF16,
                                             ldx, gamma, weights_dtype == FP8Q_OUT_BF16, dres, ldr, eps,
                                             centred == 1, M, K, dx, dgamma, dbeta, workspace,
                                             (hipStream_t)stream));
}

int fp8q_swiglu(const void* gu, int gu_dtype, int64_t ld, const int32_t* m_offsets, int64_t G, int64_t M,
                int64_t I, void* y, int y_dtype, void* stream) {
  if (!known_dtype(y_dtype)) return FP8Q_ERR_DTYPE;
  int s = check_swiglu(gu_dtype, ld, m_offsets, G, M, I);
  if (s == -1) return FP8Q_OK;
  if (s) return s;
  if (!gu || !y) return FP8Q_ERR_NULL;
  if (!aligned(gu, element(gu_dtype)) || !aligned(y, element(y_dtype))) return FP8Q_ERR_ALIGN;
  if ((s = check_device())) return s;
  return launched(fp8q::launch_swiglu(gu, gu_dtype == FP8Q_OUT_BF16, ld, m_offsets ? m_offsets + G : nullptr,
                                      M, I, y, y_dtype == FP8Q_OUT_BF16, (hipStream_t)stream));
}

int fp8q_swiglu_quant_act_1x128(const void* gu, int gu_dtype, int64_t ld, const int32_t* m_offsets,
                                int64_t G, int64_t M, int64_t I, uint8_t* q, float* sa, void* stream) {
  if (I % kGroup) return FP8Q_ERR_SHAPE;
  int s = check_swiglu(gu_dtype, ld, m_offsets, G, M, I);
  if (s == -1) return FP8Q_OK;
  if (s) return s;
  if (!gu || !q || !sa) return FP8Q_ERR_NULL;
  if (!aligned(gu, element(gu_dtype)) || !aligned(q, 16) || !aligned(sa, 4)) return FP8Q_ERR_ALIGN;
  if ((s = check_device())) return s;
  return launched(fp8q::launch_swiglu_quant(gu, gu_dtype == FP8Q_OUT_BF16, ld,
                                            m_offsets ? m_offsets + G : nullptr, M, I, q, sa,
                                            (hipStream_t)stream));
}

int fp8q_swiglu_bwd(const void* dy, int dy_dtype, int64_t ldy, const void* gu, int gu_dtype, int64_t ld,
                    const int32_t* m_offsets, int64_t G, int64_t M, int64_t I, void* dgu, void* stream) {
  if (!known_dtype(dy_dtype)) return FP8Q_ERR_DTYPE;
  int s = check_swiglu(gu_dtype, ld, m_offsets, G, M, I);
  if (s == -1) return FP8Q_OK;
  if (s) return s;
  if (ldy < I) return FP8Q_ERR_SHAPE;
  if (!dy || !gu || !dgu) return FP8Q_ERR_NULL;
  if (!aligned(dy, element(dy_dtype)) || !aligned(gu, element(gu_dtype)) || !aligned(dgu, element(gu_dtype)))
    return FP8Q_ERR_ALIGN;
  if ((s = check_device())) return s;
  return launched(fp8q::launch_swiglu_bwd(dy, dy_dtype == FP8Q_OUT_BF16, ldy, gu, gu_dtype == FP8Q_OUT_BF16,
                                          ld, m_offsets ? m_offsets + G : nullptr, M, I, dgu,
                                          (hipStream_t)stream));
}

int64_t fp8q_orthogonalize_workspace_bytes(int64_t L, int64_t M, int64_t N, int out_dtype) {
  const int s = check_ortho(L, M, N);
  if (!known_dtype(out_dtype) || s > 0) return -1;
  return s ? 0 : fp8q::ortho_workspace_bytes(L, M, N, false);  // (one number a value takes less)
}

int fp8q_orthogonalize(const void* g, int g_dtype, int64_t L, int64_t M, int64_t N, int steps, float a,
                       float b, float c, float scale, void* out, int out_dtype, void* workspace,
                       int64_t workspace_bytes, void* stream) {
  if (!known_dtype(out_dtype)) return FP8Q_ERR_DTYPE;
  return orthogonalize(g, g_dtype, L, M, N, steps, a, b, c, scale, out, out_dtype == FP8Q_OUT_BF16, false, workspace,
                       workspace_bytes, stream);
}

int fp8q_orthogonalize_f16(const void* g, int g_dtype, int64_t L, int64_t M, int64_t N, int steps, float a,
                           float b, float c, float scale, void* out, void* workspace,
                           int64_t workspace_bytes, void* stream) {
  return orthogonalize(g, g_dtype, L, M, N, steps, a, b, c, scale, out, true, true, workspace, workspace_bytes,
                       stream);
}

}  // extern "C"
