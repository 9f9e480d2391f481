"""Host-side refusals of the training step's calls.

Every call here fails validation or is a zero-size no-op, before the first HIP
call; like the other ABI checks the module runs only where no GPU is visible."""

import os

import pytest

from conftest import gpu_available

pytestmark = pytest.mark.skipif(gpu_available() or os.path.exists("/dev/kfd"),
                                reason="fake device addresses: runs only without a GPU")

P = 0x100000
X, R, G, B, Y, H, DG, DB, WS, OFF = (P * i for i in range(1, 11))
SHAPE, NULL, ALIGN, DTYPE, LARGE = 2, 1, 3, 4, 7
F32, BF16 = 0, 1
NAN, INF = float("nan"), float("inf")


def _lib():
    from fp8_fine_grained_online_amd import _lib as L
    return L.lib()


def refuses(f, good, changes):
    for at, value, status in changes:
        args = list(good)
        args[at] = value
        assert f(*args) == status, (at, value)


def test_norm():
    f = _lib().fp8q_norm
    #       0  1     2   3  4   5  6  7    8     9  10 11  12 13  14 15
    good = [X, BF16, 40, R, 36, G, B, F32, 1e-6, 1, 5, 33, Y, F32, H, None]
    refuses(f, good, [
        (1, 2, DTYPE), (7, -1, DTYPE), (13, 2, DTYPE), (2, 32, SHAPE), (4, 32, SHAPE), (8, NAN, SHAPE), (8, -1.0, SHAPE),
        (8, INF, SHAPE), (9, 2, SHAPE), (9, -1, SHAPE), (9, 0, SHAPE), (10, -1, SHAPE), (11, -1, SHAPE), (11, 16385, LARGE),
        (10, 1 << 31, LARGE), (10, 1 << 23, LARGE), (0, None, NULL), (5, None, NULL), (12, None, NULL), (3, None, NULL),
        (14, None, NULL), (0, X + 1, ALIGN), (3, R + 1, ALIGN), (5, G + 2, ALIGN), (6, B + 2, ALIGN), (12, Y + 2, ALIGN),
        (14, H + 1, ALIGN)])
    assert f(None, BF16, 0, None, 0, None, None, F32, 1e-6, 0, 0, 33, None, F32, None, None) == 0
    assert f(None, BF16, 0, None, 0, None, None, F32, 1e-6, 0, 5, 0, None, F32, None, None) == 0


def test_norm_bwd():
    L = _lib()
    f, need = L.fp8q_norm_bwd, L.fp8q_norm_bwd_workspace_bytes(5, 33, 1)
    assert need >= 2 * 33 * 4 and L.fp8q_norm_bwd_workspace_bytes(0, 33, 1) >= 0
    assert L.fp8q_norm_bwd_workspace_bytes(-1, 33, 1) == -1 and L.fp8q_norm_bwd_workspace_bytes(5, 16385, 0) == -1
    assert L.fp8q_norm_bwd_workspace_bytes(5, 33, 2) == -1
    #       0  1    2   3  4     5   6  7    8  9   10    11 12 13 14 15  16  17  18    19
    good = [Y, F32, 34, X, BF16, 40, G, F32, R, 36, 1e-6, 1, 5, 33, H, DG, DB, WS, need, None]
    refuses(f, good, [
        (1, 2, DTYPE), (4, 2, DTYPE), (7, 2, DTYPE), (2, 32, SHAPE), (5, 32, SHAPE), (9, 32, SHAPE), (10, NAN, SHAPE),
        (11, 2, SHAPE), (11, 0, NULL), (12, -1, SHAPE), (13, -1, SHAPE), (13, 16385, LARGE), (12, 1 << 23, LARGE),
        (18, need - 1, SHAPE), (0, None, NULL), (3, None, NULL), (6, None, NULL), (14, None, NULL), (15, None, NULL),
        (16, None, NULL), (17, None, NULL), (0, Y + 2, ALIGN), (3, X + 1, ALIGN), (6, G + 2, ALIGN), (8, R + 1, ALIGN),
        (14, H + 1, ALIGN), (15, DG + 2, ALIGN), (16, DB + 2, ALIGN), (17, WS + 8, ALIGN)])
    assert f(None, F32, 0, None, BF16, 0, None, F32, None, 0, 1e-6, 0, 5, 0, None, None, None, None, 0, None) == 0


def test_swiglu():
    f = _lib().fp8q_swiglu
    #       0  1     2   3    4  5  6   7  8    9
    good = [X, BF16, 66, OFF, 3, 5, 33, Y, F32, None]
    refuses(f, good, [
        (1, 2, DTYPE), (8, 2, DTYPE), (2, 65, SHAPE), (4, 0, SHAPE), (5, -1, SHAPE), (6, -1, SHAPE), (5, 1 << 31, LARGE),
        (6, 1 << 30, LARGE), (0, None, NULL), (7, None, NULL), (0, X + 1, ALIGN), (3, OFF + 2, ALIGN), (7, Y + 2, ALIGN)])
    assert f(X, BF16, 1 << 20, OFF, 3, 1 << 30, 1 << 10, Y, F32, None) == LARGE
    assert f(None, BF16, 0, None, 0, 0, 33, None, F32, None) == 0
    assert f(None, BF16, 0, None, 0, 5, 0, None, F32, None) == 0


def test_swiglu_quant():
    f = _lib().fp8q_swiglu_quant_act_1x128
    #       0  1     2    3    4  5  6    7  8  9
    good = [X, BF16, 256, OFF, 3, 5, 128, Y, H, None]
    refuses(f, good, [
        (1, 2, DTYPE), (2, 255, SHAPE), (4, 0, SHAPE), (5, -1, SHAPE), (6, 100, SHAPE), (6, -128, SHAPE), (0, None, NULL),
        (7, None, NULL), (8, None, NULL), (0, X + 1, ALIGN), (7, Y + 8, ALIGN), (8, H + 2, ALIGN)])
    assert f(None, BF16, 0, None, 0, 0, 128, None, None, None) == 0


def test_swiglu_bwd():
    f = _lib().fp8q_swiglu_bwd
    #       0  1    2   3  4     5   6    7  8  9   10 11
    good = [R, F32, 34, X, BF16, 66, OFF, 3, 5, 33, Y, None]
    refuses(f, good, [
        (1, 2, DTYPE), (4, 2, DTYPE), (2, 32, SHAPE), (5, 65, SHAPE), (7, 0, SHAPE), (8, -1, SHAPE), (9, -1, SHAPE),
        (0, None, NULL), (3, None, NULL), (10, None, NULL), (0, R + 2, ALIGN), (3, X + 1, ALIGN), (10, Y + 1, ALIGN)])
    assert f(None, F32, 0, None, BF16, 0, None, 0, 0, 33, None, None) == 0


def test_orthogonalize():
    L = _lib()
    f, need = L.fp8q_orthogonalize, L.fp8q_orthogonalize_workspace_bytes(2, 133, 270, BF16)
    size = L.fp8q_orthogonalize_workspace_bytes
    # X and both X^T, high parts at least
    assert need >= 3 * 2 * 192 * 320 * 2 and size(2, 133, 270, F32) >= need and size(0, 133, 270, F32) == 0
    assert size(2, 33, 70, BF16) == 0  # small matrices need none
    assert size(2, 33, 70, 2) == -1 and size(-1, 33, 70, F32) == -1 and size(1, 65537, 4, F32) == -1
    assert size(65536, 4, 4, F32) == -1 and size(65535, 4096, 4096, BF16) == -1
    #       0  1    2  3   4   5  6       7       8       9    10 11    12  13    14
    good = [X, F32, 2, 133, 270, 5, 3.4445, -4.775, 2.0315, 0.5, Y, BF16, WS, need, None]
    refuses(f, good, [
        (1, 2, DTYPE), (11, -1, DTYPE), (2, -1, SHAPE), (3, -1, SHAPE), (4, -1, SHAPE), (5, 0, SHAPE), (5, 101, SHAPE),
        (6, NAN, SHAPE), (7, INF, SHAPE), (8, NAN, SHAPE), (9, INF, SHAPE), (9, NAN, SHAPE), (13, need - 1, SHAPE),
        (3, 65537, LARGE), (4, 65537, LARGE), (2, 65536, LARGE), (0, None, NULL), (10, None, NULL), (12, None, NULL),
        (0, X + 2, ALIGN), (10, Y + 1, ALIGN), (12, WS + 8, ALIGN)])
    refuses(f, good[:3] + [33, 70] + good[5:12] + [None, 0, None], [
        (0, None, NULL), (10, None, NULL), (13, -1, SHAPE), (12, WS + 8, ALIGN), (0, X + 2, ALIGN), (10, Y + 1, ALIGN)])
    assert f(None, F32, 0, 33, 70, 5, 2.0, -1.5, 0.5, 1.0, None, BF16, None, 0, None) == 0
    assert f(None, F32, 2, 33, 0, 5, 2.0, -1.5, 0.5, 1.0, None, BF16, None, 0, None) == 0


def test_orthogonalize_refuses_polynomials_that_grow():
    """Singular values above 3 or an inner polynomial above 7.5 in any step; those below pass on to the NULL check."""
    f = _lib().fp8q_orthogonalize

    def status(steps, a, b, c):
        return f(None, F32, 1, 4, 4, steps, a, b, c, 1.0, Y, F32, WS, 1 << 40, None)
    for ok in ((5, 3.4445, -4.775, 2.0315), (100, 3.4445, -4.775, 2.0315), (9, 2.0, -1.5, 0.5), (9, 1.5, -0.5, 0.0),
               (3, 1.0, 0.0, 0.0), (1, 3.0, 0.0, 0.0), (1, 4.0848, -6.8946, 2.9270)):
        assert status(*ok) == NULL, ok
    for bad in ((2, 3.0, 0.0, 0.0), (1, 3.1, 0.0, 0.0), (1, 1.0, -8.0, 0.0), (2, 5.0, -3.0, 0.0), (3, 3.4445, -4.775, 4.0),
                (1, 10.0, -20.0, 10.0)):
        assert status(*bad) == SHAPE, bad
    # the largest value inside the interval: s (1 - s^2) 7.9 has its top, 3.04, at s^2 = 1/3
    assert status(1, 7.9, -7.9, 0.0) == SHAPE and status(1, 7.5, -7.5, 0.0) == NULL


def test_binding_refuses_before_any_device_call():
    import torch
    import fp8_fine_grained_online_amd as F
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64)
    for call in (lambda: F.fp8q_norm(x, w, 1e-6), lambda: F.fp8q_norm_bwd(x, x, w, 1e-6), lambda: F.fp8q_swiglu(x),
                 lambda: F.fp8q_swiglu_quant_act_1x128(x), lambda: F.fp8q_swiglu_bwd(x, x),
                 lambda: F.fp8q_orthogonalize(x)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(TypeError):
        F.fp8q_norm(None, w, 1e-6)
    with pytest.raises(ValueError, match="out_dtype"):
        F.fp8q_swiglu(x, out_dtype="f16")
