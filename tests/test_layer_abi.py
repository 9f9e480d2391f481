"""Host-side refusals of the MoE layer's calls and of the 8-bit integer product.

Every call here fails validation or is a zero-size no-op, before the first HIP
call; like the other ABI checks the module runs only where no GPU is visible."""

import os

import pytest

from conftest import gpu_available

pytestmark = pytest.mark.skipif(gpu_available() or os.path.exists("/dev/kfd"),
                                reason="fake device addresses: runs only without a GPU")

P = 0x100000
A, SA, B, SB, C, OFF, X, IDS, W, WS = (P * i for i in range(1, 11))
SHAPE, NULL, ALIGN, DTYPE, LARGE = 2, 1, 3, 4, 7
F32, BF16 = 0, 1


def _lib():
    from fp8_fine_grained_online_amd import _lib as L
    return L.lib()


def refuses(f, good, changes):
    for at, value, status in changes:
        args = list(good)
        args[at] = value
        assert f(*args) == status, (at, value)


def test_route():
    f = _lib().fp8q_moe_route
    #       0  1    2  3  4   5  6  7  8  9  10   11   12 13
    good = [X, F32, B, 4, 64, 8, 8, 4, 1, 1, 2.5, IDS, W, None]
    refuses(f, good, [
        (1, 2, DTYPE), (1, -1, DTYPE), (3, -1, SHAPE), (3, 1 << 31, LARGE), (4, 0, SHAPE), (4, 1025, LARGE),
        (4, 60, SHAPE), (5, 0, SHAPE), (5, 65, LARGE), (5, 33, SHAPE), (6, 0, SHAPE), (6, 65, LARGE), (6, 7, SHAPE),
        (7, 0, SHAPE), (7, 9, SHAPE), (8, 2, SHAPE), (9, 2, SHAPE), (10, float("nan"), SHAPE),
        (10, float("inf"), SHAPE), (0, None, NULL), (11, None, NULL), (12, None, NULL), (0, X + 2, ALIGN),
        (2, B + 2, ALIGN), (11, IDS + 1, ALIGN), (12, W + 2, ALIGN)])
    assert f(X + 1, BF16, None, 4, 64, 8, 1, 1, 0, 0, 1.0, IDS, W, None) == ALIGN
    assert f(X, F32, None, 4, 4, 8, 1, 1, 0, 0, 1.0, IDS, W, None) == SHAPE  # topk > G
    assert f(None, F32, None, 0, 64, 8, 1, 1, 0, 0, 1.0, None, None, None) == 0


def test_route_bwd():
    f = _lib().fp8q_moe_route_bwd
    #       0  1    2    3  4  5   6  7  8  9    10 11
    good = [X, F32, IDS, W, 4, 64, 8, 1, 1, 2.5, C, None]
    refuses(f, good, [
        (1, 3, DTYPE), (4, -1, SHAPE), (5, 0, SHAPE), (5, 2000, LARGE), (6, 0, SHAPE), (6, 65, LARGE), (7, -1, SHAPE),
        (8, 2, SHAPE), (9, float("nan"), SHAPE), (0, None, NULL), (2, None, NULL), (3, None, NULL), (10, None, NULL),
        (0, X + 2, ALIGN), (2, IDS + 2, ALIGN), (3, W + 1, ALIGN), (10, C + 2, ALIGN)])
    assert f(None, F32, None, None, 0, 64, 8, 1, 1, 1.0, None, None) == 0


def test_permute():
    L = _lib()
    f = L.fp8q_moe_permute
    rows, ws = L.fp8q_moe_dispatch_max_rows(4, 2, 8), L.fp8q_moe_dispatch_workspace_bytes(4, 2, 8)
    #       0  1     2    3  4   5  6  7  8     9    10  11  12  13
    good = [X, BF16, IDS, 4, 64, 2, 8, C, rows, OFF, SA, WS, ws, None]
    refuses(f, good, [
        (1, 2, DTYPE), (3, -1, SHAPE), (4, 60, SHAPE), (4, -8, SHAPE), (5, 0, SHAPE), (6, 0, SHAPE), (6, 1025, LARGE),
        (8, rows - 1, SHAPE), (8, -1, SHAPE), (12, ws - 1, SHAPE), (0, None, NULL), (2, None, NULL), (7, None, NULL),
        (9, None, NULL), (10, None, NULL), (11, None, NULL), (0, X + 8, ALIGN), (2, IDS + 2, ALIGN), (7, C + 4, ALIGN),
        (9, OFF + 1, ALIGN), (10, SA + 2, ALIGN), (11, WS + 2, ALIGN), (3, 1 << 30, LARGE)])


def test_combine():
    f = _lib().fp8q_moe_combine
    #       0  1     2    3  4  5   6  7    8  9    10
    good = [C, BF16, IDS, W, 4, 64, 2, 128, X, F32, None]
    refuses(f, good, [
        (1, 2, DTYPE), (9, 2, DTYPE), (4, -1, SHAPE), (5, 60, SHAPE), (5, -8, SHAPE), (6, 0, SHAPE), (7, -1, SHAPE),
        (7, 1 << 31, LARGE), (4, 1 << 31, LARGE), (0, None, NULL), (2, None, NULL), (8, None, NULL), (0, C + 8, ALIGN),
        (2, IDS + 1, ALIGN), (3, W + 2, ALIGN), (8, X + 4, ALIGN)])
    assert f(C, BF16, IDS, W, (1 << 30) - 1, 8192, 2, 128, X, F32, None) == LARGE  # 16 runs per token
    assert f(None, BF16, None, None, 0, 64, 2, 128, None, F32, None) == 0
    assert f(None, BF16, None, None, 4, 0, 2, 128, None, F32, None) == 0


def test_combine_bwd():
    f = _lib().fp8q_moe_combine_bwd
    #       0  1    2  3     4    5  6    7  8   9  10 11   12 13 14
    good = [X, F32, C, BF16, IDS, W, OFF, 4, 64, 2, 8, 128, B, SB, None]
    refuses(f, good, [
        (1, 2, DTYPE), (3, 2, DTYPE), (7, -1, SHAPE), (8, 4, SHAPE), (9, 0, SHAPE), (10, 0, SHAPE), (10, 1025, LARGE),
        (11, -1, SHAPE), (0, None, NULL), (2, None, NULL), (4, None, NULL), (6, None, NULL), (12, None, NULL),
        (0, X + 8, ALIGN), (2, C + 8, ALIGN), (4, IDS + 2, ALIGN), (5, W + 2, ALIGN), (6, OFF + 2, ALIGN),
        (12, B + 8, ALIGN), (13, SB + 2, ALIGN)])


def test_quant_int8_rows():
    f = _lib().fp8q_quant_int8_rows
    good = [X, 4, 64, A, SA, None]
    refuses(f, good, [(1, -1, SHAPE), (2, 24, SHAPE), (2, -16, SHAPE), (1, 1 << 31, LARGE), (2, 1 << 31, LARGE),
                      (0, None, NULL), (3, None, NULL), (4, None, NULL), (0, X + 8, ALIGN), (3, A + 8, ALIGN),
                      (4, SA + 2, ALIGN)])
    assert f(None, 0, 64, None, None, None) == 0


def test_int8_gemm():
    f = _lib().int8_gemm_scaled
    #       0  1   2  3   4  5     6  7  8   9
    good = [A, SA, B, SB, C, BF16, 5, 7, 64, None]
    refuses(f, good, [(5, 2, DTYPE), (6, -1, SHAPE), (7, -1, SHAPE), (8, 24, SHAPE), (8, 131072, LARGE),
                      (6, 1 << 31, LARGE), (0, None, NULL), (1, None, NULL), (2, None, NULL), (3, None, NULL),
                      (4, None, NULL), (0, A + 8, ALIGN), (1, SA + 2, ALIGN), (2, B + 4, ALIGN), (3, SB + 1, ALIGN),
                      (4, C + 8, ALIGN)])
    assert f(A, SA, B, SB, C, BF16, 1 << 20, 1 << 20, 64, None) == LARGE
    assert f(A + 8, SA, B, SB, C, BF16, 5, 7, 131056, None) == ALIGN  # the largest K passes the size checks
    assert f(None, None, None, None, None, BF16, 0, 7, 64, None) == 0
    assert f(None, None, None, None, None, BF16, 5, 0, 64, None) == 0


def test_int8_grouped():
    f = _lib().int8_gemm_grouped
    #       0  1   2  3   4  5    6    7  8    9  10  11
    good = [A, SA, B, SB, C, F32, OFF, 3, 256, 7, 64, None]
    refuses(f, good, [(5, 2, DTYPE), (7, 0, SHAPE), (8, 200, SHAPE), (9, -1, SHAPE), (10, 8, SHAPE), (7, 1 << 31, LARGE),
                      (6, None, NULL), (0, None, NULL), (4, None, NULL), (6, OFF + 2, ALIGN), (2, B + 8, ALIGN)])
    assert f(None, None, None, None, None, F32, None, 3, 0, 7, 64, None) == 0


def test_binding_refuses_before_any_device_call():
    import torch
    import fp8_fine_grained_online_amd as F
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        F.fp8q_quant_int8_rows(x)
    with pytest.raises(ValueError, match="device tensor"):
        F.fp8q_moe_route(x, 2)
    with pytest.raises(TypeError):
        F.fp8q_moe_permute(None, x, 4)
    with pytest.raises(ValueError, match="device tensor"):
        F.fp8q_moe_combine(x, torch.zeros(4, 2, dtype=torch.int32))


def test_binding_refuses_a_stream_of_another_device():
    import torch
    import fp8_fine_grained_online_amd as F

    class Stream:
        cuda_stream, device = 64, torch.device("cuda", 1)

    class Tensor:
        is_cuda, device = True, torch.device("cuda", 0)

    with pytest.raises(ValueError, match="cuda:1"):
        F.fp8q_quant_int8_rows(Tensor(), stream=Stream())
