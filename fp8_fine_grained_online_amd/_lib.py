"""Binding of libfp8q.so: argument marshalling only (ctypes; the calls that a layer
makes for single tokens through a native extension, csrc/binding.cpp)."""

import ctypes
import os

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(PKG_DIR, "libfp8q.so")

FP8Q_OUT_F32 = 0
FP8Q_OUT_BF16 = 1

STATUS = {
    0: "FP8Q_OK", 1: "FP8Q_ERR_NULL", 2: "FP8Q_ERR_SHAPE", 3: "FP8Q_ERR_ALIGN",
    4: "FP8Q_ERR_DTYPE", 5: "FP8Q_ERR_LAUNCH", 6: "FP8Q_ERR_NO_DEVICE", 7: "FP8Q_ERR_TOO_LARGE",
    8: "FP8Q_ERR_SCRATCH",
}

_lib = None


class Fp8qError(RuntimeError):
    def __init__(self, fn, status, text):
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({text})")
        self.status = status


def lib_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(
                f"{_LIB_PATH} is missing: build it with `python -m fp8_fine_grained_online_amd.build`"
                " (there is no fallback path)")
        L = ctypes.CDLL(_LIB_PATH)
        i64, vp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        L.fp8q_version.restype = i32
        L.fp8q_version.argtypes = []
        L.fp8q_status_string.restype = ctypes.c_char_p
        L.fp8q_status_string.argtypes = [i32]
        L.fp8q_quant_act_1x128.restype = i32
        L.fp8q_quant_act_1x128.argtypes = [vp, i64, i64, vp, vp, vp]
        L.fp8q_quant_act_1x128_nt.restype = i32
        L.fp8q_quant_act_1x128_nt.argtypes = [vp, i64, i64, vp, vp, vp]
        L.fp8q_quant_weight_128x128.restype = i32
        L.fp8q_quant_weight_128x128.argtypes = [vp, i64, i64, vp, vp, vp]
        L.fp8_gemm_blockscaled.restype = i32
        L.fp8_gemm_blockscaled.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp]
        L.fp8_gemm_blockscaled_bf16a.restype = i32
        L.fp8_gemm_blockscaled_bf16a.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, vp, vp, vp]
        L.fp8_gemm_blockscaled_ws.restype = i32
        L.fp8_gemm_blockscaled_ws.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp, i64, vp]
        L.fp8_gemm_blockscaled_noalloc.restype = i32
        L.fp8_gemm_blockscaled_noalloc.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp]
        L.fp8_gemm_blockscaled_ws_bytes.restype = i64
        L.fp8_gemm_blockscaled_ws_bytes.argtypes = [i64, i64, i64]
        L.fp8_gemm_grouped.restype = i32
        L.fp8_gemm_grouped.argtypes = [vp, vp, vp, vp, vp, i32, vp, i64, i64, i64, i64, vp]
        L.fp8q_quant_act_128x1.restype = i32
        L.fp8q_quant_act_128x1.argtypes = [vp, i64, i64, vp, vp, vp]
        L.fp8q_moe_dispatch_1x128.restype = i32
        L.fp8q_moe_dispatch_1x128.argtypes = [vp, vp, i64, i64, i64, i64, vp, vp, i64, vp, vp, vp,
                                              i64, vp]
        L.fp8q_moe_dispatch_workspace_bytes.restype = i64
        L.fp8q_moe_dispatch_workspace_bytes.argtypes = [i64, i64, i64]
        L.fp8q_moe_dispatch_max_rows.restype = i64
        L.fp8q_moe_dispatch_max_rows.argtypes = [i64, i64, i64]
        L.fp8q_norm_quant_act_1x128.restype = i32
        L.fp8q_norm_quant_act_1x128.argtypes = [vp, vp, vp, ctypes.c_float, i32, i64, i64, vp, vp, vp]
        L.fp8q_quant_act_1x128_128x1.restype = i32
        L.fp8q_quant_act_1x128_128x1.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp]
        L.fp8q_requant_1x128_to_128x1.restype = i32
        L.fp8q_requant_1x128_to_128x1.argtypes = [vp, vp, i64, i64, vp, vp, vp]
        L.fp8q_transpose_weight_128x128.restype = i32
        L.fp8q_transpose_weight_128x128.argtypes = [vp, vp, i64, i64, vp, vp, vp]
        L.fp8_gemm_rowscaled.restype = i32
        L.fp8_gemm_rowscaled.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp]
        f32 = ctypes.c_float
        L.fp8q_moe_route.restype = i32
        L.fp8q_moe_route.argtypes = [vp, i32, vp, i64, i64, i64, i64, i64, i32, i32, f32, vp, vp, vp]
        L.fp8q_moe_route_bwd.restype = i32
        L.fp8q_moe_route_bwd.argtypes = [vp, i32, vp, vp, i64, i64, i64, i32, i32, f32, vp, vp]
        L.fp8q_moe_permute.restype = i32
        L.fp8q_moe_permute.argtypes = [vp, i32, vp, i64, i64, i64, i64, vp, i64, vp, vp, vp, i64, vp]
        L.fp8q_moe_combine.restype = i32
        L.fp8q_moe_combine.argtypes = [vp, i32, vp, vp, i64, i64, i64, i64, vp, i32, vp]
        L.fp8q_moe_combine_bwd.restype = i32
        L.fp8q_moe_combine_bwd.argtypes = [vp, i32, vp, i32, vp, vp, vp, i64, i64, i64, i64, i64, vp,
                                           vp, vp]
        L.fp8q_quant_int8_rows.restype = i32
        L.fp8q_quant_int8_rows.argtypes = [vp, i64, i64, vp, vp, vp]
        L.int8_gemm_scaled.restype = i32
        L.int8_gemm_scaled.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp]
        L.int8_gemm_grouped.restype = i32
        L.int8_gemm_grouped.argtypes = [vp, vp, vp, vp, vp, i32, vp, i64, i64, i64, i64, vp]
        L.fp8q_norm.restype = i32
        L.fp8q_norm.argtypes = [vp, i32, i64, vp, i64, vp, vp, i32, f32, i32, i64, i64, vp, i32, vp, vp]
        L.fp8q_norm_bwd_workspace_bytes.restype = i64
        L.fp8q_norm_bwd_workspace_bytes.argtypes = [i64, i64, i32]
        L.fp8q_norm_bwd.restype = i32
        L.fp8q_norm_bwd.argtypes = [vp, i32, i64, vp, i32, i64, vp, i32, vp, i64, f32, i32, i64, i64, vp, vp,
                                    vp, vp, i64, vp]
        L.fp8q_swiglu.restype = i32
        L.fp8q_swiglu.argtypes = [vp, i32, i64, vp, i64, i64, i64, vp, i32, vp]
        L.fp8q_swiglu_quant_act_1x128.restype = i32
        L.fp8q_swiglu_quant_act_1x128.argtypes = [vp, i32, i64, vp, i64, i64, i64, vp, vp, vp]
        L.fp8q_swiglu_bwd.restype = i32
        L.fp8q_swiglu_bwd.argtypes = [vp, i32, i64, vp, i32, i64, vp, i64, i64, i64, vp, vp]
        L.fp8q_orthogonalize_workspace_bytes.restype = i64
        L.fp8q_orthogonalize_workspace_bytes.argtypes = [i64, i64, i64, i32]
        L.fp8q_orthogonalize.restype = i32
        L.fp8q_orthogonalize.argtypes = [vp, i32, i64, i64, i64, i32, f32, f32, f32, f32, vp, i32, vp, i64, vp]
        L.fp8q_orthogonalize_f16.restype = i32
        L.fp8q_orthogonalize_f16.argtypes = [vp, i32, i64, i64, i64, i32, f32, f32, f32, f32, vp, vp, i64, vp]
        _lib = L
    return _lib


def fp8q_version() -> int:
    return lib().fp8q_version()


def _check(fn, status):
    if status != 0:
        raise Fp8qError(fn, status, lib().fp8q_status_string(status).decode())


def _torch():
    import torch
    return torch


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t, name, dtype, ndim):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _out(t, name, shape, dtype, device):
    torch = _torch()
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _dev(t, name, dtype, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def fp8q_quant_act_1x128(x, q=None, sa=None, stream=None):
    """x: bf16 M x K device tensor -> (q uint8 M x K, sa float32 M x K/128)."""
    torch = _torch()
    px = _dev(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    q = _out(q, "q", (M, K), torch.uint8, x.device)
    sa = _out(sa, "sa", (M, K // 128 if K % 128 == 0 else 0), torch.float32, x.device)
    _check("fp8q_quant_act_1x128",
           lib().fp8q_quant_act_1x128(px, M, K, q.data_ptr(), sa.data_ptr(), _stream(stream)))
    return q, sa


def fp8q_quant_act_1x128_nt(x, q=None, sa=None, stream=None):
    """fp8q_quant_act_1x128 with non-temporal stores (same results; for codes
    that are not read next on this GPU)."""
    torch = _torch()
    px = _dev(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    q = _out(q, "q", (M, K), torch.uint8, x.device)
    sa = _out(sa, "sa", (M, K // 128 if K % 128 == 0 else 0), torch.float32, x.device)
    _check("fp8q_quant_act_1x128_nt",
           lib().fp8q_quant_act_1x128_nt(px, M, K, q.data_ptr(), sa.data_ptr(), _stream(stream)))
    return q, sa


def fp8q_quant_weight_128x128(w, q=None, sb=None, stream=None):
    """w: bf16 N x K (or G x N x K) device tensor -> (q uint8 like w, sb float32 .../128 x K/128)."""
    torch = _torch()
    if w.dim() == 3:
        G, N, K = w.shape
        q = _out(q, "q", (G, N, K), torch.uint8, w.device)
        sb = _out(sb, "sb", (G, N // 128, K // 128), torch.float32, w.device)
        _dev(w, "w", torch.bfloat16, 3)
        rows = G * N
    else:
        _dev(w, "w", torch.bfloat16, 2)
        N, K = w.shape
        q = _out(q, "q", (N, K), torch.uint8, w.device)
        sb = _out(sb, "sb", (N // 128, K // 128), torch.float32, w.device)
        rows = N
    if w.dim() == 3 and N % 128:
        raise ValueError("per-expert N must be a multiple of 128")
    _check("fp8q_quant_weight_128x128",
           lib().fp8q_quant_weight_128x128(w.data_ptr(), rows, K, q.data_ptr(), sb.data_ptr(),
                                           _stream(stream)))
    return q, sb


def _out_dtype(out_dtype):
    torch = _torch()
    if out_dtype in (torch.bfloat16, "bf16", FP8Q_OUT_BF16):
        return FP8Q_OUT_BF16, torch.bfloat16
    if out_dtype in (torch.float32, "f32", FP8Q_OUT_F32):
        return FP8Q_OUT_F32, torch.float32
    raise ValueError(f"unsupported out_dtype {out_dtype}")


def fp8_gemm_blockscaled(a, sa, b, sb, out_dtype="bf16", c=None, stream=None):
    """C = A * B^T with per-1x128 (sa) and per-128x128 (sb) scales. Returns c (M x N)."""
    torch = _torch()
    code, tdt = _out_dtype(out_dtype)
    pa = _dev(a, "a", torch.uint8, 2)
    psa = _dev(sa, "sa", torch.float32, 2)
    pb = _dev(b, "b", torch.uint8, 2)
    psb = _dev(sb, "sb", torch.float32, 2)
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K:
        raise ValueError("a and b must share K")
    if K % 128 == 0 and N % 128 == 0:
        if tuple(sa.shape) != (M, K // 128) or tuple(sb.shape) != (N // 128, K // 128):
            raise ValueError("scale shapes must be (M, K/128) and (N/128, K/128)")
    c = _out(c, "c", (M, N), tdt, a.device)
    _check("fp8_gemm_blockscaled",
           lib().fp8_gemm_blockscaled(pa, psa, pb, psb, c.data_ptr(), code, M, N, K,
                                      _stream(stream)))
    return c


def fp8_gemm_blockscaled_bf16a(a, b, sb, out_dtype="bf16", c=None, qa=None, sa=None,
                               with_codes=False, stream=None):
    """Quantize-on-load GEMM: a is bf16 M x K, quantized to 1x128 tiles inside
    the GEMM. Returns c, or (c, qa, sa) with with_codes (A's codes and scales,
    as fp8q_quant_act_1x128 gives them)."""
    torch = _torch()
    code, tdt = _out_dtype(out_dtype)
    pa = _dev(a, "a", torch.bfloat16, 2)
    pb = _dev(b, "b", torch.uint8, 2)
    psb = _dev(sb, "sb", torch.float32, 2)
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K:
        raise ValueError("a and b must share K")
    if K % 128 == 0 and N % 128 == 0 and tuple(sb.shape) != (N // 128, K // 128):
        raise ValueError("sb must have shape (N/128, K/128)")
    c = _out(c, "c", (M, N), tdt, a.device)
    pq = ps = None
    if with_codes or qa is not None or sa is not None:
        qa = _out(qa, "qa", (M, K), torch.uint8, a.device)
        sa = _out(sa, "sa", (M, K // 128), torch.float32, a.device)
        pq, ps = qa.data_ptr(), sa.data_ptr()
    _check("fp8_gemm_blockscaled_bf16a",
           lib().fp8_gemm_blockscaled_bf16a(pa, pb, psb, c.data_ptr(), code, M, N, K, pq, ps,
                                            _stream(stream)))
    return (c, qa, sa) if pq is not None else c


def fp8_gemm_blockscaled_ws(a, sa, b, sb, out_dtype="bf16", c=None, workspace=None, stream=None):
    """fp8_gemm_blockscaled with a workspace (split-K for small-M shapes).
    The workspace (uint8 device tensor) is allocated when not given."""
    torch = _torch()
    code, tdt = _out_dtype(out_dtype)
    pa = _dev(a, "a", torch.uint8, 2)
    psa = _dev(sa, "sa", torch.float32, 2)
    pb = _dev(b, "b", torch.uint8, 2)
    psb = _dev(sb, "sb", torch.float32, 2)
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K:
        raise ValueError("a and b must share K")
    if K % 128 == 0 and N % 128 == 0:
        if tuple(sa.shape) != (M, K // 128) or tuple(sb.shape) != (N // 128, K // 128):
            raise ValueError("scale shapes must be (M, K/128) and (N/128, K/128)")
    c = _out(c, "c", (M, N), tdt, a.device)
    need = lib().fp8_gemm_blockscaled_ws_bytes(M, N, K)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=a.device)
    pw = workspace.data_ptr() if workspace is not None else None
    nw = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("fp8_gemm_blockscaled_ws",
           lib().fp8_gemm_blockscaled_ws(pa, psa, pb, psb, c.data_ptr(), code, M, N, K, pw, nw,
                                         _stream(stream)))
    return c


def _grouped_shapes(a, sa, b, sb, m_offsets, M_total):
    """Shape checks of the grouped GEMM's operands (before any device access):
    the kernel indexes expert e's block scales at sb + e * (N/128) * (K/128), so
    sb must be exactly G x N/128 x K/128 for the b it goes with."""
    if b.dim() != 3 or a.dim() != 2 or sa.dim() != 2 or sb.dim() != 3 or m_offsets.dim() != 1:
        raise ValueError("a, sa: 2 dims; b, sb: 3 dims; m_offsets: 1 dim")
    G, N, K = b.shape
    if m_offsets.shape[0] != G + 1:
        raise ValueError("m_offsets must have G+1 entries")
    M = a.shape[0] if M_total is None else int(M_total)
    if a.shape[1] != K or a.shape[0] < M:
        raise ValueError("a must be at least M_total x K")
    if K % 128 == 0 and N % 128 == 0:
        if sa.shape[0] < M or sa.shape[1] != K // 128:
            raise ValueError("sa must be at least M_total x K/128")
        if tuple(sb.shape) != (G, N // 128, K // 128):
            raise ValueError(f"sb must have shape {(G, N // 128, K // 128)}, got {tuple(sb.shape)}")
    return G, N, K, M


def fp8_gemm_blockscaled_noalloc(a, sa, b, sb, out_dtype="bf16", c=None, stream=None):
    """fp8_gemm_blockscaled_ws with the split-K partials in the library's
    static per-GPU scratch (no workspace; pass c to allocate nothing at all)."""
    torch = _torch()
    code, tdt = _out_dtype(out_dtype)
    pa = _dev(a, "a", torch.uint8, 2)
    psa = _dev(sa, "sa", torch.float32, 2)
    pb = _dev(b, "b", torch.uint8, 2)
    psb = _dev(sb, "sb", torch.float32, 2)
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K:
        raise ValueError("a and b must share K")
    if K % 128 == 0 and N % 128 == 0:
        if tuple(sa.shape) != (M, K // 128) or tuple(sb.shape) != (N // 128, K // 128):
            raise ValueError("scale shapes must be (M, K/128) and (N/128, K/128)")
    c = _out(c, "c", (M, N), tdt, a.device)
    _check("fp8_gemm_blockscaled_noalloc",
           lib().fp8_gemm_blockscaled_noalloc(pa, psa, pb, psb, c.data_ptr(), code, M, N, K,
                                              _stream(stream)))
    return c


def fp8_gemm_grouped(a, sa, b, sb, m_offsets, out_dtype="bf16", c=None, M_total=None, stream=None):
    """Grouped GEMM. b: G x N x K codes, sb: G x N/128 x K/128, m_offsets: int32[G+1] device.

    M_total defaults to a.shape[0] (the host-side row count; m_offsets is never
    read on the host).
    """
    torch = _torch()
    code, tdt = _out_dtype(out_dtype)
    G, N, K, M = _grouped_shapes(a, sa, b, sb, m_offsets, M_total)
    pa = _dev(a, "a", torch.uint8, 2)
    psa = _dev(sa, "sa", torch.float32, 2)
    pb = _dev(b, "b", torch.uint8, 3)
    psb = _dev(sb, "sb", torch.float32, 3)
    poff = _dev(m_offsets, "m_offsets", torch.int32, 1)
    c = _out(c, "c", (M, N), tdt, a.device)
    _check("fp8_gemm_grouped",
           lib().fp8_gemm_grouped(pa, psa, pb, psb, c.data_ptr(), code, poff, G, M, N, K,
                                  _stream(stream)))
    return c


def _div128(n):
    return n // 128 if n % 128 == 0 else 0


def fp8q_quant_act_128x1(x, qt=None, st=None, stream=None):
    """x: bf16 M x K device tensor -> (qt uint8 K x M, st float32 K x M/128): 128x1 tiles, transposed."""
    torch = _torch()
    px = _dev(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    qt = _out(qt, "qt", (K, M), torch.uint8, x.device)
    st = _out(st, "st", (K, _div128(M)), torch.float32, x.device)
    _check("fp8q_quant_act_128x1",
           lib().fp8q_quant_act_128x1(px, M, K, qt.data_ptr(), st.data_ptr(), _stream(stream)))
    return qt, st


def fp8q_moe_dispatch_1x128(x, topk_ids, G, q=None, sa=None, m_offsets=None, row_of_slot=None,
                            workspace=None, stream=None):
    """FP8 dispatch: x bf16 T x K, topk_ids int32 T x topk (device) ->
    (q uint8 M_cap x K, sa float32 M_cap x K/128, m_offsets int32[G+1], row_of_slot int32 T x topk).

    M_cap = fp8q_moe_dispatch_max_rows(T, topk, G); only rows below m_offsets[G]
    are written. Pass q.shape[0] as M_total to fp8_gemm_grouped (no host sync).
    """
    torch = _torch()
    px = _dev(x, "x", torch.bfloat16, 2)
    pid = _dev(topk_ids, "topk_ids", torch.int32, 2)
    T, K = x.shape
    if topk_ids.shape[0] != T:
        raise ValueError("topk_ids must have one row per token")
    topk = topk_ids.shape[1]
    L = lib()
    M_cap = L.fp8q_moe_dispatch_max_rows(T, topk, G)
    ws_bytes = L.fp8q_moe_dispatch_workspace_bytes(T, topk, G)
    if M_cap < 0 or ws_bytes < 0:
        raise ValueError("invalid dispatch sizes")
    q = _out(q, "q", (M_cap, K), torch.uint8, x.device)
    sa = _out(sa, "sa", (M_cap, _div128(K)), torch.float32, x.device)
    m_offsets = _out(m_offsets, "m_offsets", (G + 1,), torch.int32, x.device)
    row_of_slot = _out(row_of_slot, "row_of_slot", (T, topk), torch.int32, x.device)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 4), dtype=torch.uint8, device=x.device)
    _check("fp8q_moe_dispatch_1x128",
           L.fp8q_moe_dispatch_1x128(px, pid, T, K, topk, G, q.data_ptr(), sa.data_ptr(), M_cap,
                                     m_offsets.data_ptr(), row_of_slot.data_ptr(),
                                     workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return q, sa, m_offsets, row_of_slot


def fp8q_norm_quant_act_1x128(x, gamma, eps, beta=None, centred=False, q=None, sa=None,
                              stream=None):
    """Normalize rows of x (bf16 M x K; RMS, or centred with beta) and quantize the
    binary32 result per 1x128 tile -> (q uint8 M x K, sa float32 M x K/128)."""
    torch = _torch()
    px = _dev(x, "x", torch.bfloat16, 2)
    pg = _dev(gamma, "gamma", torch.bfloat16, 1)
    pb = _dev(beta, "beta", torch.bfloat16, 1) if beta is not None else None
    M, K = x.shape
    if gamma.shape[0] != K or (beta is not None and beta.shape[0] != K):
        raise ValueError("gamma and beta must have K entries")
    q = _out(q, "q", (M, K), torch.uint8, x.device)
    sa = _out(sa, "sa", (M, _div128(K)), torch.float32, x.device)
    _check("fp8q_norm_quant_act_1x128",
           lib().fp8q_norm_quant_act_1x128(px, pg, pb, float(eps), int(bool(centred)), M, K,
                                           q.data_ptr(), sa.data_ptr(), _stream(stream)))
    return q, sa


def fp8q_quant_act_1x128_128x1(x, q=None, sa=None, qt=None, st=None, stream=None):
    """x: bf16 M x K -> (q M x K, sa M x K/128, qt K x M, st K x M/128): both tilings, one read."""
    torch = _torch()
    px = _dev(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    q = _out(q, "q", (M, K), torch.uint8, x.device)
    sa = _out(sa, "sa", (M, _div128(K)), torch.float32, x.device)
    qt = _out(qt, "qt", (K, M), torch.uint8, x.device)
    st = _out(st, "st", (K, _div128(M)), torch.float32, x.device)
    _check("fp8q_quant_act_1x128_128x1",
           lib().fp8q_quant_act_1x128_128x1(px, M, K, q.data_ptr(), sa.data_ptr(), qt.data_ptr(),
                                            st.data_ptr(), _stream(stream)))
    return q, sa, qt, st


def fp8q_requant_1x128_to_128x1(q, sa, qt=None, st=None, stream=None):
    """Stored 1x128 codes q (M x K) and sa (M x K/128) -> (qt K x M, st K x M/128)."""
    torch = _torch()
    pq = _dev(q, "q", torch.uint8, 2)
    psa = _dev(sa, "sa", torch.float32, 2)
    M, K = q.shape
    if tuple(sa.shape) != (M, _div128(K)):
        raise ValueError("sa must have shape (M, K/128)")
    qt = _out(qt, "qt", (K, M), torch.uint8, q.device)
    st = _out(st, "st", (K, _div128(M)), torch.float32, q.device)
    _check("fp8q_requant_1x128_to_128x1",
           lib().fp8q_requant_1x128_to_128x1(pq, psa, M, K, qt.data_ptr(), st.data_ptr(),
                                             _stream(stream)))
    return qt, st


def fp8q_transpose_weight_128x128(q, sb, qt=None, sbt=None, stream=None):
    """Weight codes q (N x K) and block scales sb (N/128 x K/128) -> (qt K x N, sbt K/128 x N/128)."""
    torch = _torch()
    pq = _dev(q, "q", torch.uint8, 2)
    psb = _dev(sb, "sb", torch.float32, 2)
    N, K = q.shape
    if tuple(sb.shape) != (_div128(N), _div128(K)):
        raise ValueError("sb must have shape (N/128, K/128)")
    qt = _out(qt, "qt", (K, N), torch.uint8, q.device)
    sbt = _out(sbt, "sbt", (_div128(K), _div128(N)), torch.float32, q.device)
    _check("fp8q_transpose_weight_128x128",
           lib().fp8q_transpose_weight_128x128(pq, psb, N, K, qt.data_ptr(), sbt.data_ptr(),
                                               _stream(stream)))
    return qt, sbt


def fp8_gemm_rowscaled(a, sa, b, sb, out_dtype="f32", c=None, stream=None):
    """C = A * B^T with 1x128 scales on both operands: sa (M x K/128), sb (N x K/128)."""
    torch = _torch()
    code, tdt = _out_dtype(out_dtype)
    pa = _dev(a, "a", torch.uint8, 2)
    psa = _dev(sa, "sa", torch.float32, 2)
    pb = _dev(b, "b", torch.uint8, 2)
    psb = _dev(sb, "sb", torch.float32, 2)
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K:
        raise ValueError("a and b must share K")
    if K % 128 == 0:
        if tuple(sa.shape) != (M, K // 128) or tuple(sb.shape) != (N, K // 128):
            raise ValueError("scale shapes must be (M, K/128) and (N, K/128)")
    c = _out(c, "c", (M, N), tdt, a.device)
    _check("fp8_gemm_rowscaled",
           lib().fp8_gemm_rowscaled(pa, psa, pb, psb, c.data_ptr(), code, M, N, K, _stream(stream)))
    return c


# ---- MoE layer around the experts' products, the 8-bit integer product, a training step ----
#
# These calls are short enough for a binding's own time to count, so their
# argument checks and allocations are native (csrc/binding.cpp).

_native = None  # the extension module, once a call has needed it


def _binding():
    global _native
    if _native is None:
        _torch()  # the extension links to its libraries
        path = os.path.join(PKG_DIR, "_binding.so")
        if not os.path.exists(path):
            raise ImportError(
                f"{path} is missing: build it with `python -m fp8_fine_grained_online_amd.build`"
                " (there is no fallback path)")
        lib()
        from . import _binding as module
        module.on_status(_check)
        _native = module
    return _native


def _on_stream(stream, fn, first, *args):
    """A call with `stream` current: new outputs then come from that stream's memory too
    (memory freed on another stream may still be in use there). Without a stream the
    calls below run on the current stream of the tensors' device."""
    cuda = _torch().cuda
    device = getattr(first, "device", None)
    if not hasattr(stream, "cuda_stream"):
        # (ExternalStream takes 0 as a wish for a new stream)
        stream = cuda.ExternalStream(int(stream), device=device) if int(stream) else cuda.default_stream(device)
    if getattr(first, "is_cuda", False) and stream.device != device:
        raise ValueError(f"{fn.__name__}: the stream is on {stream.device}, the tensors on {device}")
    with cuda.stream(stream):
        return fn(first, *args)


SCORES = {"softmax": 0, "sigmoid": 1}
_OUT_CODES = {"bf16": FP8Q_OUT_BF16, "f32": FP8Q_OUT_F32}


def _out_code(out_dtype):
    return _OUT_CODES[out_dtype] if out_dtype in _OUT_CODES else _out_dtype(out_dtype)[0]


def _score(score):
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    return SCORES[score]


def fp8q_moe_route(logits, topk, bias=None, score="softmax", renormalize=True, scale=1.0, n_groups=1,
                   topk_groups=1, topk_ids=None, weights=None, stream=None):
    """Router: logits T x G (float32 or bfloat16) -> (topk_ids int32 T x topk, weights float32
    T x topk). bias (float32, G) is added to the probabilities for the choice only; with
    n_groups > 1 experts come from the topk_groups best groups."""
    if stream is not None:
        return _on_stream(stream, fp8q_moe_route, logits, topk, bias, score, renormalize, scale, n_groups, topk_groups,
                          topk_ids, weights)
    return (_native or _binding()).fp8q_moe_route(logits, bias, topk, _score(score), renormalize, scale, n_groups,
                                                   topk_groups, topk_ids, weights)


def fp8q_moe_route_bwd(logits, topk_ids, dweights, score="softmax", renormalize=True, scale=1.0,
                       dlogits=None, stream=None):
    """Gradient of fp8q_moe_route's weights: dweights (float32 T x topk) -> dlogits (T x G, like logits)."""
    if stream is not None:
        return _on_stream(stream, fp8q_moe_route_bwd, logits, topk_ids, dweights, score, renormalize, scale, dlogits)
    return (_native or _binding()).fp8q_moe_route_bwd(logits, topk_ids, dweights, _score(score), renormalize,
                                                       scale, dlogits)


def fp8q_moe_permute(x, topk_ids, G, xp=None, m_offsets=None, row_of_slot=None, workspace=None,
                     stream=None):
    """Rows sorted by expert: x T x K (bfloat16 or float32), topk_ids int32 T x topk ->
    (xp M_cap x K, m_offsets int32[G+1], row_of_slot int32 T x topk), the layout of
    fp8q_moe_dispatch_1x128; rows of xp from m_offsets[G] on are not written."""
    if stream is not None:
        return _on_stream(stream, fp8q_moe_permute, x, topk_ids, G, xp, m_offsets, row_of_slot, workspace)
    return (_native or _binding()).fp8q_moe_permute(x, topk_ids, G, xp, m_offsets, row_of_slot, workspace)


def fp8q_moe_combine(c, row_of_slot, weights=None, out_dtype="bf16", y=None, stream=None):
    """The way back: y[t] = sum_j weights[t, j] * c[row_of_slot[t, j]] (weights None: ones; rows
    outside c are skipped). c M x K (bfloat16 or float32) -> y T x K of out_dtype."""
    if stream is not None:
        return _on_stream(stream, fp8q_moe_combine, c, row_of_slot, weights, out_dtype, y)
    return (_native or _binding()).fp8q_moe_combine(c, row_of_slot, weights, _out_code(out_dtype), y)


def fp8q_moe_combine_bwd(dy, c, row_of_slot, weights, m_offsets, dc=None, dw=None, with_dw=True,
                         stream=None):
    """Gradient of fp8q_moe_combine: dy T x K, c M x K -> (dc M x K like c, dw float32 T x topk);
    padding rows of dc are zero, rows from m_offsets[G] on are not written. with_dw=False: dw is
    None (unless given) and c is only used for its shape and type."""
    if stream is not None:
        return _on_stream(stream, fp8q_moe_combine_bwd, dy, c, row_of_slot, weights, m_offsets, dc, dw, with_dw)
    return (_native or _binding()).fp8q_moe_combine_bwd(dy, c, row_of_slot, weights, m_offsets, dc, dw, with_dw)


def fp8q_quant_int8_rows(x, q=None, s=None, stream=None):
    """x: bf16 ... x K device tensor (2 or 3 dims: tokens, channels or experts' channels) ->
    (q int8 like x, s float32 without the last dim): one scale amax / 127 per row."""
    if stream is not None:
        return _on_stream(stream, fp8q_quant_int8_rows, x, q, s)
    return (_native or _binding()).fp8q_quant_int8_rows(x, q, s)


def int8_gemm_scaled(a, sa, b, sb, out_dtype="bf16", c=None, stream=None):
    """c[m, n] = (sum_k a[m, k] b[n, k]) * sa[m] * sb[n]: a int8 M x K, sa float32 M, b int8 N x K,
    sb float32 N. Returns c (M x N)."""
    if stream is not None:
        return _on_stream(stream, int8_gemm_scaled, a, sa, b, sb, out_dtype, c)
    return (_native or _binding()).int8_gemm_scaled(a, sa, b, sb, _out_code(out_dtype), c)


def int8_gemm_grouped(a, sa, b, sb, m_offsets, out_dtype="bf16", c=None, M_total=None, stream=None):
    """Grouped form: a int8 M x K, sa float32 M, b int8 G x N x K, sb float32 G x N, m_offsets
    int32[G+1] (device, multiples of 128, never read on the host). M_total defaults to a.shape[0]."""
    if stream is not None:
        return _on_stream(stream, int8_gemm_grouped, a, sa, b, sb, m_offsets, out_dtype, c, M_total)
    return (_native or _binding()).int8_gemm_grouped(a, sa, b, sb, m_offsets, _out_code(out_dtype), c,
                                                      M_total)


def fp8q_norm(x, gamma, eps, beta=None, centred=False, residual=None, out_dtype="bf16", y=None, h=None, stream=None):
    """Rows of x (M x K, bfloat16 or float32), or of x + residual, normalized: RMS, or centred with an
    optional beta -> y (M x K of out_dtype); with a residual (y, h), h the sum in x's type. Rows of x
    and residual may lie apart; gamma and beta are of one type, bfloat16 or float32."""
    if stream is not None:
        return _on_stream(stream, fp8q_norm, x, gamma, eps, beta, centred, residual, out_dtype, y, h)
    return (_native or _binding()).fp8q_norm(x, gamma, eps, beta, centred, residual, _out_code(out_dtype), y, h)


def fp8q_norm_bwd(dy, x, gamma, eps, centred=False, dres=None, dx=None, dgamma=None, dbeta=None, workspace=None,
                  stream=None):
    """Gradient of fp8q_norm, or of the normalization in fp8q_norm_quant_act_1x128, of x (fp8q_norm's h
    where it had a residual): dy M x K -> (dx M x K like x, dgamma float32 K, dbeta float32 K or None
    where not centred). dres (like x) is added to dx: the residual stream's own gradient."""
    if stream is not None:
        return _on_stream(stream, fp8q_norm_bwd, dy, x, gamma, eps, centred, dres, dx, dgamma, dbeta, workspace)
    return (_native or _binding()).fp8q_norm_bwd(dy, x, gamma, eps, centred, dres, dx, dgamma, dbeta, workspace)


def fp8q_swiglu(gu, out_dtype="bf16", m_offsets=None, y=None, stream=None):
    """gu = [gate | up] (M x 2I, bfloat16 or float32) -> y = silu(gate) * up (M x I of out_dtype). With
    m_offsets (int32[G+1], device) rows from m_offsets[G] on are neither read nor written."""
    if stream is not None:
        return _on_stream(stream, fp8q_swiglu, gu, out_dtype, m_offsets, y)
    return (_native or _binding()).fp8q_swiglu(gu, m_offsets, _out_code(out_dtype), y)


def fp8q_swiglu_quant_act_1x128(gu, m_offsets=None, q=None, sa=None, stream=None):
    """fp8q_swiglu's binary32 result in 1x128 FP8 tiles -> (q uint8 M x I, sa float32 M x I/128)."""
    if stream is not None:
        return _on_stream(stream, fp8q_swiglu_quant_act_1x128, gu, m_offsets, q, sa)
    return (_native or _binding()).fp8q_swiglu_quant_act_1x128(gu, m_offsets, q, sa)


def fp8q_swiglu_bwd(dy, gu, m_offsets=None, dgu=None, stream=None):
    """Gradient of fp8q_swiglu: dy M x I -> dgu = [dgate | dup] (M x 2I, like gu)."""
    if stream is not None:
        return _on_stream(stream, fp8q_swiglu_bwd, dy, gu, m_offsets, dgu)
    return (_native or _binding()).fp8q_swiglu_bwd(dy, gu, m_offsets, dgu)


def fp8q_orthogonalize(g, steps=5, coeffs=(3.4445, -4.7750, 2.0315), scale=1.0, out_dtype="bf16", out=None,
                       workspace=None, stream=None, single=False):
    """scale times the matrix that `steps` Newton-Schulz steps with p(s) = a s + b s^3 + c s^5, coeffs =
    (a, b, c), make of g / |g| (Frobenius): g M x N, or L x M x N for a matrix each (bfloat16 or float32)
    -> out like g, of out_dtype. A zero matrix gives zeros. As exact as in float32; `single`, for a bfloat16
    out, multiplies FP16 numbers instead of pairs of them: up to 3.5 times as fast for large matrices, and
    off by about 1e-3 before the rounding, by up to 1e-2 for matrices of few magnitudes."""
    if stream is not None:
        return _on_stream(stream, fp8q_orthogonalize, g, steps, coeffs, scale, out_dtype, out, workspace, None, single)
    a, b, c = coeffs
    return (_native or _binding()).fp8q_orthogonalize(g, steps, a, b, c, scale, _out_code(out_dtype), out, workspace,
                                                      single)
