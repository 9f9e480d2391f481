// Python binding of the MoE layer's calls, of the 8-bit integer product and of a
// training step's calls around the products, as
// a CPython extension over the C ABI: argument checks, outputs, device and
// stream, and the call. A serving step's kernels take a few microseconds each,
// so the binding's own time is part of the latency: the same checks and
// allocations in Python around a ctypes call took 8.4 us for the router; these
// take 4.9, of which the launch itself is 2.9.
//
// Every function returns its outputs. Wrong types and shapes raise TypeError and
// ValueError; for a status other than FP8Q_OK the function given to on_status is
// called, which raises the binding's own error.
// The work goes to the current stream of the tensors' device, whatever device
// is current.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPStream.h>
#include <hip/hip_runtime.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <initializer_list>
#include <string>

#include "../../include/fp8q.h"

namespace {

using at::ScalarType;

[[noreturn]] void refuse(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw python_error();
}

PyObject* status_handler = nullptr;  // (name, status) -> raises

// One call's tensors: all on the device of the first.
struct Call {
  int device = -1;
  int previous = -1;
  const char* name;
  PyObject* const* args;

  Call(const char* f, PyObject* const* a, Py_ssize_t given, Py_ssize_t wanted) : name(f), args(a) {
    if (given != wanted) refuse(PyExc_TypeError, "%s: expected %d arguments", f, (int)wanted);
  }
  ~Call() {
    if (previous >= 0) (void)hipSetDevice(previous);
  }
  Call(const Call&) = delete;
  Call& operator=(const Call&) = delete;

  bool none(int i) const { return args[i] == Py_None; }

  // Argument i: a contiguous tensor of one of `types` with `dims` dimensions
  const at::Tensor& tensor(int i, const char* name, std::initializer_list<ScalarType> types, int64_t dims,
                           bool contiguous = true) {
    if (!THPVariable_Check(args[i])) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
    const at::Tensor& t = THPVariable_Unpack(args[i]);
    if (!t.is_cuda() || (device >= 0 && t.get_device() != device))
      refuse(PyExc_ValueError, "%s must be a device tensor%s", name,
                              device >= 0 ? " on the device of the call's first tensor" : "");
    if (device < 0) device = (int)t.get_device();
    bool known = false;
    for (ScalarType s : types) known |= t.scalar_type() == s;
    if (!known) refuse(PyExc_TypeError, "%s must not be of type %s here (the first allowed is %s)", name,
                                       at::toString(t.scalar_type()), at::toString(*types.begin()));
    if (t.dim() != dims) refuse(PyExc_ValueError, "%s must have %d dims, got %d", name, (int)dims, (int)t.dim());
    if (contiguous && !t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    return t;
  }

  // Argument i: a 2-dimensional tensor of one of `types` whose rows are dense but may
  // lie apart; `ld` gets the elements from one row to the next
  const at::Tensor& rows(int i, const char* name, std::initializer_list<ScalarType> types, int64_t& ld) {
    const at::Tensor& t = tensor(i, name, types, 2, false);
    const int64_t M = t.size(0), K = t.size(1);
    ld = M > 1 ? t.stride(0) : K;
    if ((K > 1 && t.stride(1) != 1) || ld < K) refuse(PyExc_ValueError, "%s must have dense rows that do not overlap", name);
    return t;
  }

  // Argument i as an output of this type and shape: the caller's, or a new one
  // (from the memory of the device's current stream) for None: straight from the
  // allocator (the router's call 4.9 us, 5.4 through the dispatcher)
  at::Tensor out(int i, const char* name, at::IntArrayRef shape, ScalarType type) {
    if (none(i)) {
      for (int64_t d : shape)
        if (d < 0) refuse(PyExc_ValueError, "%s would have a negative size", name);
      return at::Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (at::DeviceIndex)device), std::nullopt));
    }
    const at::Tensor& t = tensor(i, name, {type}, (int64_t)shape.size());
    if (t.sizes() != shape) {
      std::string want;
      for (int64_t d : shape) want += (want.empty() ? "" : ", ") + std::to_string(d);
      refuse(PyExc_ValueError, "%s must have shape (%s)", name, want.c_str());
    }
    return t;
  }

  int64_t integer(int i) const {
    const int64_t v = PyLong_AsLongLong(args[i]);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
  }
  int truth(int i) const {
    const int v = PyObject_IsTrue(args[i]);
    if (v < 0) throw python_error();
    return v;
  }
  double number(int i) const {
    const double v = PyFloat_AsDouble(args[i]);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
  }

  // The tensors' device made current (until the call is over); its current stream
  void* stream() {
    int now = -1;
    if (hipGetDevice(&now) == hipSuccess && now != device && hipSetDevice(device) == hipSuccess) previous = now;
    return (void*)c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
  }
};

constexpr std::initializer_list<ScalarType> kFloats = {ScalarType::Float, ScalarType::BFloat16};
int code(const at::Tensor& t) { return t.scalar_type() == ScalarType::BFloat16 ? FP8Q_OUT_BF16 : FP8Q_OUT_F32; }
ScalarType type_of(int64_t c) { return c == FP8Q_OUT_BF16 ? ScalarType::BFloat16 : ScalarType::Float; }
void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

PyObject* wrap(const Call& c, int i, const at::Tensor& t) {
  if (c.none(i)) return THPVariable_Wrap(t);
  Py_INCREF(c.args[i]);
  return c.args[i];
}

// The outputs (arguments `at`), or the status as an error
template <size_t n>
PyObject* result(int status, const Call& c, const int (&at)[n], const at::Tensor* const (&outs)[n]) {
  if (status) {
    PyObject* none = PyObject_CallFunction(status_handler, "si", c.name, status);
    if (none) Py_DECREF(none), refuse(PyExc_RuntimeError, "%s: status %d", c.name, status);
    throw python_error();
  }
  if (n == 1) return wrap(c, at[0], *outs[0]);
  PyObject* tuple = PyTuple_New(n);
  if (!tuple) throw python_error();
  for (size_t i = 0; i < n; ++i) {
    PyObject* o = Py_None;
    if (outs[i]->defined()) o = wrap(c, at[i], *outs[i]);
    else Py_INCREF(o);
    PyTuple_SET_ITEM(tuple, i, o);
  }
  return tuple;
}

// The library call, other Python threads running meanwhile
template <typename F>
int launch(F&& f) {
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = f();
  Py_END_ALLOW_THREADS;
  return status;
}

// logits, bias, topk, score, renormalize, scale, n_groups, topk_groups, topk_ids, weights
PyObject* moe_route(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c("fp8q_moe_route", args, n, 10);
  const at::Tensor& x = c.tensor(0, "logits", kFloats, 2);
  const int64_t T = x.size(0), G = x.size(1), topk = c.integer(2);
  at::Tensor bias;
  if (!c.none(1)) {
    bias = c.tensor(1, "bias", {ScalarType::Float}, 1);
    if (bias.size(0) != G) refuse(PyExc_ValueError, "bias must have G entries");
  }
  const int64_t score = c.integer(3), renorm = c.truth(4), groups = c.integer(6), kept = c.integer(7);
  const float scale = (float)c.number(5);
  // (more choices than experts are refused by the library: nothing is allocated for them)
  auto cols = [&](int i) { return topk < 0 || (topk > G && c.none(i)) ? 0 : topk; };
  const at::Tensor ids = c.out(8, "topk_ids", {T, cols(8)}, ScalarType::Int);
  const at::Tensor w = c.out(9, "weights", {T, cols(9)}, ScalarType::Float);
  void* s = c.stream();
  const int status = launch([&] {
    return fp8q_moe_route(ptr(x), code(x), (const float*)ptr(bias), T, G, topk, groups, kept, (int)score, (int)renorm,
                          scale, (int32_t*)ptr(ids), (float*)ptr(w), s);
  });
  return result(status, c, {8, 9}, {&ids, &w});
  END_HANDLE_TH_ERRORS
}

// logits, topk_ids, dweights, score, renormalize, scale, dlogits
PyObject* moe_route_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c("fp8q_moe_route_bwd", args, n, 7);
  const at::Tensor& x = c.tensor(0, "logits", kFloats, 2);
  const at::Tensor& ids = c.tensor(1, "topk_ids", {ScalarType::Int}, 2);
  const at::Tensor& dw = c.tensor(2, "dweights", {ScalarType::Float}, 2);
  const int64_t T = x.size(0), G = x.size(1);
  if (ids.sizes() != dw.sizes() || ids.size(0) != T) refuse(PyExc_ValueError, "topk_ids and dweights must both be T x topk");
  const int64_t score = c.integer(3), renorm = c.truth(4);
  const float scale = (float)c.number(5);
  const at::Tensor d = c.out(6, "dlogits", {T, G}, x.scalar_type());
  void* s = c.stream();
  const int status = launch([&] {
    return fp8q_moe_route_bwd(ptr(x), code(x), (const int32_t*)ptr(ids), (const float*)ptr(dw), T, G, ids.size(1),
                              (int)score, (int)renorm, scale, ptr(d), s);
  });
  return result(status, c, {6}, {&d});
  END_HANDLE_TH_ERRORS
}

// x, topk_ids, G, xp, m_offsets, row_of_slot, workspace
PyObject* moe_permute(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c("fp8q_moe_permute", args, n, 7);
  const at::Tensor& x = c.tensor(0, "x", kFloats, 2);
  const at::Tensor& ids = c.tensor(1, "topk_ids", {ScalarType::Int}, 2);
  const int64_t T = x.size(0), K = x.size(1), topk = ids.size(1), G = c.integer(2);
  if (ids.size(0) != T) refuse(PyExc_ValueError, "topk_ids must have one row per token");
  const int64_t cap = fp8q_moe_dispatch_max_rows(T, topk, G), bytes = fp8q_moe_dispatch_workspace_bytes(T, topk, G);
  if (cap < 0 || bytes < 0) refuse(PyExc_ValueError, "invalid permute sizes");
  const at::Tensor xp = c.out(3, "xp", {cap, K}, x.scalar_type());
  const at::Tensor off = c.out(4, "m_offsets", {G + 1}, ScalarType::Int);
  const at::Tensor rows = c.out(5, "row_of_slot", {T, topk}, ScalarType::Int);
  const at::Tensor ws = c.none(6) ? c.out(6, "workspace", {bytes}, ScalarType::Byte)
                                  : c.tensor(6, "workspace", {ScalarType::Byte}, 1);
  void* s = c.stream();
  const int status = launch([&] {
    return fp8q_moe_permute(ptr(x), code(x), (const int32_t*)ptr(ids), T, K, topk, G, ptr(xp), cap, (int32_t*)ptr(off),
                            (int32_t*)ptr(rows), ptr(ws), ws.numel(), s);
  });
  return result(status, c, {3, 4, 5}, {&xp, &off, &rows});
  END_HANDLE_TH_ERRORS
}

at::Tensor slot_weights(Call& c, int i, const at::Tensor& rows) {
  if (c.none(i)) return {};
  const at::Tensor& w = c.tensor(i, "weights", {ScalarType::Float}, 2);
  if (w.sizes() != rows.sizes()) refuse(PyExc_ValueError, "weights must have row_of_slot's shape");
  return w;
}

// c, row_of_slot, weights, out_dtype, y
PyObject* moe_combine(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c("fp8q_moe_combine", args, n, 5);
  const at::Tensor& x = c.tensor(0, "c", kFloats, 2);
  const at::Tensor& rows = c.tensor(1, "row_of_slot", {ScalarType::Int}, 2);
  const at::Tensor w = slot_weights(c, 2, rows);
  const int64_t out = c.integer(3), T = rows.size(0), K = x.size(1);
  const at::Tensor y = c.out(4, "y", {T, K}, type_of(out));
  void* s = c.stream();
  const int status = launch([&] {
    return fp8q_moe_combine(ptr(x), code(x), (const int32_t*)ptr(rows), (const float*)ptr(w), T, K, rows.size(1),
                            x.size(0), ptr(y), (int)out, s);
  });
  return result(status, c, {4}, {&y});
  END_HANDLE_TH_ERRORS
}

// dy, c, row_of_slot, weights, m_offsets, dc, dw, with_dw
PyObject* moe_combine_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c("fp8q_moe_combine_bwd", args, n, 8);
  const at::Tensor& dy = c.tensor(0, "dy", kFloats, 2);
  const at::Tensor& x = c.tensor(1, "c", kFloats, 2);
  const at::Tensor& rows = c.tensor(2, "row_of_slot", {ScalarType::Int}, 2);
  const at::Tensor w = slot_weights(c, 3, rows);
  const at::Tensor& off = c.tensor(4, "m_offsets", {ScalarType::Int}, 1);
  const int64_t M = x.size(0), K = x.size(1), T = rows.size(0), topk = rows.size(1);
  if (dy.size(0) != T || dy.size(1) != K) refuse(PyExc_ValueError, "dy must be T x K, one row per token and c's columns");
  if (off.size(0) < 2) refuse(PyExc_ValueError, "m_offsets must have G+1 entries");
  const at::Tensor dc = c.out(5, "dc", {M, K}, x.scalar_type());
  at::Tensor dw;
  if (c.truth(7) || !c.none(6)) dw = c.out(6, "dw", {T, topk}, ScalarType::Float);
  void* s = c.stream();
  const int status = launch([&] {
    return fp8q_moe_combine_bwd(ptr(dy), code(dy), ptr(x), code(x), (const int32_t*)ptr(rows), (const float*)ptr(w),
                                (const int32_t*)ptr(off), T, K, topk, off.size(0) - 1, M, ptr(dc), (float*)ptr(dw), s);
  });
  return result(status, c, {5, 6}, {&dc, &dw});
  END_HANDLE_TH_ERRORS
}

// x, q, s
PyObject* quant_int8_rows(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c("fp8q_quant_int8_rows", args, n, 3);
  const bool experts = THPVariable_Check(args[0]) && THPVariable_Unpack(args[0]).dim() == 3;
  const at::Tensor& x = c.tensor(0, "x", {ScalarType::BFloat16}, experts ? 3 : 2);
  const int64_t K = x.size(-1), rows = experts ? x.size(0) * x.size(1) : x.size(0);
  const at::Tensor q = c.out(1, "q", x.sizes(), ScalarType::Char);
  const at::Tensor sc = c.out(2, "s", x.sizes().slice(0, x.dim() - 1), ScalarType::Float);
  void* s = c.stream();
  const int status = launch([&] { return fp8q_quant_int8_rows(ptr(x), rows, K, (int8_t*)ptr(q), (float*)ptr(sc), s); });
  return result(status, c, {1, 2}, {&q, &sc});
  END_HANDLE_TH_ERRORS
}

// a, sa, b, sb, out_dtype, c
PyObject* int8_gemm_dense(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c("int8_gemm_scaled", args, n, 6);
  const at::Tensor& a = c.tensor(0, "a", {ScalarType::Char}, 2);
  const at::Tensor& sa = c.tensor(1, "sa", {ScalarType::Float}, 1);
  const at::Tensor& b = c.tensor(2, "b", {ScalarType::Char}, 2);
  const at::Tensor& sb = c.tensor(3, "sb", {ScalarType::Float}, 1);
  const int64_t M = a.size(0), K = a.size(1), N = b.size(0), out = c.integer(4);
  if (b.size(1) != K) refuse(PyExc_ValueError, "a and b must share K");
  if (sa.size(0) != M || sb.size(0) != N) refuse(PyExc_ValueError, "scale shapes must be (M,) and (N,)");
  const at::Tensor y = c.out(5, "c", {M, N}, type_of(out));
  void* s = c.stream();
  const int status = launch([&] {
    return int8_gemm_scaled((const int8_t*)ptr(a), (const float*)ptr(sa), (const int8_t*)ptr(b), (const float*)ptr(sb),
                            ptr(y), (int)out, M, N, K, s);
  });
  return result(status, c, {5}, {&y});
  END_HANDLE_TH_ERRORS
}

// a, sa, b, sb, m_offsets, out_dtype, c, M_total
PyObject* int8_gemm_experts(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c("int8_gemm_grouped", args, n, 8);
  const at::Tensor& a = c.tensor(0, "a", {ScalarType::Char}, 2);
  const at::Tensor& sa = c.tensor(1, "sa", {ScalarType::Float}, 1);
  const at::Tensor& b = c.tensor(2, "b", {ScalarType::Char}, 3);
  const at::Tensor& sb = c.tensor(3, "sb", {ScalarType::Float}, 2);
  const at::Tensor& off = c.tensor(4, "m_offsets", {ScalarType::Int}, 1);
  const int64_t G = b.size(0), N = b.size(1), K = b.size(2), out = c.integer(5);
  const int64_t M = c.none(7) ? a.size(0) : c.integer(7);
  if (off.size(0) != G + 1) refuse(PyExc_ValueError, "m_offsets must have G+1 entries");
  if (a.size(1) != K || a.size(0) < M || sa.size(0) < M)
    refuse(PyExc_ValueError, "a must be at least M_total x K, with a scale per row");
  if (sb.size(0) != G || sb.size(1) != N) refuse(PyExc_ValueError, "sb must be G x N");
  const at::Tensor y = c.out(6, "c", {M, N}, type_of(out));
  void* s = c.stream();
  const int status = launch([&] {
    return int8_gemm_grouped((const int8_t*)ptr(a), (const float*)ptr(sa), (const int8_t*)ptr(b), (const float*)ptr(sb),
                             ptr(y), (int)out, (const int32_t*)ptr(off), G, M, N, K, s);
  });
  return result(status, c, {6}, {&y});
  END_HANDLE_TH_ERRORS
}

// A weight of K entries, or none where `optional` and None is given
at::Tensor weight(Call& c, int i, const char* name, int64_t K, bool optional) {
  if (optional && c.none(i)) return {};
  const at::Tensor& w = c.tensor(i, name, kFloats, 1);
  if (w.size(0) != K) refuse(PyExc_ValueError, "%s must have K entries", name);
  return w;
}

// x, gamma, eps, beta, centred, residual, out_dtype, y, h
PyObject* norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c("fp8q_norm", args, n, 9);
  int64_t ldx, ldr = 0;
  const at::Tensor& x = c.rows(0, "x", kFloats, ldx);
  const int64_t M = x.size(0), K = x.size(1), out = c.integer(6);
  const at::Tensor gamma = weight(c, 1, "gamma", K, false), beta = weight(c, 3, "beta", K, true);
  if (beta.defined() && beta.scalar_type() != gamma.scalar_type())
    refuse(PyExc_TypeError, "gamma and beta must be of one type");
  const float eps = (float)c.number(2);
  const int centred = c.truth(4);
  at::Tensor res, h;
  if (!c.none(5)) {
    res = c.rows(5, "residual", {x.scalar_type()}, ldr);
    if (res.sizes() != x.sizes()) refuse(PyExc_ValueError, "residual must have x's shape");
    h = c.out(8, "h", {M, K}, x.scalar_type());
  } else if (!c.none(8)) {
    refuse(PyExc_ValueError, "h goes with a residual");
  }
  const at::Tensor y = c.out(7, "y", {M, K}, type_of(out));
  void* s = c.stream();
  const int status = launch([&] {
    return fp8q_norm(ptr(x), code(x), ldx, ptr(res), ldr, ptr(gamma), ptr(beta), code(gamma), eps, centred, M, K, ptr(y),
                     (int)out, ptr(h), s);
  });
  if (!h.defined()) return result(status, c, {7}, {&y});
  return result(status, c, {7, 8}, {&y, &h});
  END_HANDLE_TH_ERRORS
}

// dy, x, gamma, eps, centred, dres, dx, dgamma, dbeta, workspace
PyObject* norm_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c("fp8q_norm_bwd", args, n, 10);
  int64_t ldy, ldx, ldr = 0;
  const at::Tensor& dy = c.rows(0, "dy", kFloats, ldy);
  const at::Tensor& x = c.rows(1, "x", kFloats, ldx);
  if (dy.sizes() != x.sizes()) refuse(PyExc_ValueError, "dy must have x's shape");
  const int64_t M = x.size(0), K = x.size(1);
  const at::Tensor gamma = weight(c, 2, "gamma", K, false);
  const float eps = (float)c.number(3);
  const int centred = c.truth(4);
  at::Tensor res, dbeta;
  if (!c.none(5)) {
    res = c.rows(5, "dres", {x.scalar_type()}, ldr);
    if (res.sizes() != x.sizes()) refuse(PyExc_ValueError, "dres must have x's shape");
  }
  const int64_t bytes = fp8q_norm_bwd_workspace_bytes(M, K, centred);
  if (bytes < 0) refuse(PyExc_ValueError, "invalid normalization sizes");
  const at::Tensor dx = c.out(6, "dx", {M, K}, x.scalar_type());
  const at::Tensor dgamma = c.out(7, "dgamma", {K}, ScalarType::Float);
  if (centred) dbeta = c.out(8, "dbeta", {K}, ScalarType::Float);
  else if (!c.none(8)) refuse(PyExc_ValueError, "dbeta goes with the centred form");
  const at::Tensor ws = c.none(9) ? c.out(9, "workspace", {bytes}, ScalarType::Byte)
                                  : c.tensor(9, "workspace", {ScalarType::Byte}, 1);
  void* s = c.stream();
  const int status = launch([&] {
    return fp8q_norm_bwd(ptr(dy), code(dy), ldy, ptr(x), code(x), ldx, ptr(gamma), code(gamma), ptr(res), ldr, eps,
                         centred, M, K, ptr(dx), (float*)ptr(dgamma), (float*)ptr(dbeta), ptr(ws), ws.numel(), s);
  });
  return result(status, c, {6, 7, 8}, {&dx, &dgamma, &dbeta});
  END_HANDLE_TH_ERRORS
}

// gu's rows as [gate | up]; the offsets of the experts' blocks, where given
struct Gated {
  const at::Tensor& gu;
  at::Tensor off;
  int64_t ld, M, I, G = 0;

  Gated(Call& c, int i, int i_off) : gu(c.rows(i, "gu", kFloats, ld)), M(gu.size(0)), I(gu.size(1) / 2) {
    if (gu.size(1) % 2) refuse(PyExc_ValueError, "gu must have 2 I columns, gate and up");
    if (c.none(i_off)) return;
    off = c.tensor(i_off, "m_offsets", {ScalarType::Int}, 1);
    G = off.size(0) - 1;
    if (G < 1) refuse(PyExc_ValueError, "m_offsets must have G+1 entries");
  }
};

// gu, m_offsets, out_dtype, y
PyObject* swiglu(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c("fp8q_swiglu", args, n, 4);
  const Gated g(c, 0, 1);
  const int64_t out = c.integer(2);
  const at::Tensor y = c.out(3, "y", {g.M, g.I}, type_of(out));
  void* s = c.stream();
  const int status = launch([&] {
    return fp8q_swiglu(ptr(g.gu), code(g.gu), g.ld, (const int32_t*)ptr(g.off), g.G, g.M, g.I, ptr(y), (int)out, s);
  });
  return result(status, c, {3}, {&y});
  END_HANDLE_TH_ERRORS
}

// gu, m_offsets, q, sa
PyObject* swiglu_quant(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c("fp8q_swiglu_quant_act_1x128", args, n, 4);
  const Gated g(c, 0, 1);
  const at::Tensor q = c.out(2, "q", {g.M, g.I}, ScalarType::Byte);
  const at::Tensor sa = c.out(3, "sa", {g.M, g.I / 128}, ScalarType::Float);
  void* s = c.stream();
  const int status = launch([&] {
    return fp8q_swiglu_quant_act_1x128(ptr(g.gu), code(g.gu), g.ld, (const int32_t*)ptr(g.off), g.G, g.M, g.I,
                                       (uint8_t*)ptr(q), (float*)ptr(sa), s);
  });
  return result(status, c, {2, 3}, {&q, &sa});
  END_HANDLE_TH_ERRORS
}

// dy, gu, m_offsets, dgu
PyObject* swiglu_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c("fp8q_swiglu_bwd", args, n, 4);
  int64_t ldy;
  const at::Tensor& dy = c.rows(0, "dy", kFloats, ldy);
  const Gated g(c, 1, 2);
  if (dy.size(0) != g.M || dy.size(1) != g.I) refuse(PyExc_ValueError, "dy must be M x I for gu's M x 2I");
  const at::Tensor dgu = c.out(3, "dgu", {g.M, 2 * g.I}, g.gu.scalar_type());
  void* s = c.stream();
  const int status = launch([&] {
    return fp8q_swiglu_bwd(ptr(dy), code(dy), ldy, ptr(g.gu), code(g.gu), g.ld, (const int32_t*)ptr(g.off), g.G, g.M, g.I,
                           ptr(dgu), s);
  });
  return result(status, c, {3}, {&dgu});
  END_HANDLE_TH_ERRORS
}

// g, steps, a, b, c, scale, out_dtype, out, workspace, single
PyObject* orthogonalize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c("fp8q_orthogonalize", args, n, 10);
  const bool several = THPVariable_Check(args[0]) && THPVariable_Unpack(args[0]).dim() == 3;
  const at::Tensor& g = c.tensor(0, "g", kFloats, several ? 3 : 2);
  const int64_t L = several ? g.size(0) : 1, M = g.size(-2), N = g.size(-1), steps = c.integer(1), out = c.integer(6);
  if (steps < 1 || steps > 100) refuse(PyExc_ValueError, "steps must be 1 to 100");
  const float k[3] = {(float)c.number(2), (float)c.number(3), (float)c.number(4)}, scale = (float)c.number(5);
  const bool single = c.truth(9);
  if (single && out != FP8Q_OUT_BF16) refuse(PyExc_ValueError, "single goes with a bfloat16 out");
  const int64_t bytes = fp8q_orthogonalize_workspace_bytes(L, M, N, (int)out);
  if (bytes < 0) refuse(PyExc_ValueError, "invalid sizes to orthogonalize");
  const at::Tensor y = c.out(7, "out", g.sizes(), type_of(out));
  const at::Tensor ws = c.none(8) ? c.out(8, "workspace", {bytes}, ScalarType::Byte)
                                  : c.tensor(8, "workspace", {ScalarType::Byte}, 1);
  void* s = c.stream();
  const int status = launch([&] {
    if (single)
      return fp8q_orthogonalize_f16(ptr(g), code(g), L, M, N, (int)steps, k[0], k[1], k[2], scale, ptr(y), ptr(ws),
                                    ws.numel(), s);
    return fp8q_orthogonalize(ptr(g), code(g), L, M, N, (int)steps, k[0], k[1], k[2], scale, ptr(y), (int)out, ptr(ws),
                              ws.numel(), s);
  });
  return result(status, c, {7}, {&y});
  END_HANDLE_TH_ERRORS
}

PyObject* on_status(PyObject*, PyObject* handler) {
  Py_INCREF(handler);
  Py_XDECREF(status_handler);
  status_handler = handler;
  Py_RETURN_NONE;
}

#define FP8Q_METHOD(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    FP8Q_METHOD("fp8q_moe_route", moe_route),
    FP8Q_METHOD("fp8q_moe_route_bwd", moe_route_bwd),
    FP8Q_METHOD("fp8q_moe_permute", moe_permute),
    FP8Q_METHOD("fp8q_moe_combine", moe_combine),
    FP8Q_METHOD("fp8q_moe_combine_bwd", moe_combine_bwd),
    FP8Q_METHOD("fp8q_quant_int8_rows", quant_int8_rows),
    FP8Q_METHOD("int8_gemm_scaled", int8_gemm_dense),
    FP8Q_METHOD("int8_gemm_grouped", int8_gemm_experts),
    FP8Q_METHOD("fp8q_norm", norm),
    FP8Q_METHOD("fp8q_norm_bwd", norm_bwd),
    FP8Q_METHOD("fp8q_swiglu", swiglu),
    FP8Q_METHOD("fp8q_swiglu_quant_act_1x128", swiglu_quant),
    FP8Q_METHOD("fp8q_swiglu_bwd", swiglu_bwd),
    FP8Q_METHOD("fp8q_orthogonalize", orthogonalize),
    {"on_status", on_status, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
