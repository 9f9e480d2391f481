"""Host-side checks of the training step's calls: the orthogonalization with one FP16 number a value.

Every call here fails validation or is a zero-size no-op, before the first HIP
call; like the other ABI checks the module runs only where no GPU is visible."""

import os

import pytest

from conftest import gpu_available
from test_step_abi import ALIGN, BF16, DTYPE, F32, INF, LARGE, NAN, NULL, SHAPE, WS, X, Y, _lib, refuses

pytestmark = pytest.mark.skipif(gpu_available() or os.path.exists("/dev/kfd"),
                                reason="fake device addresses: runs only without a GPU")


def test_orthogonalize_f16():
    L = _lib()
    f, need = L.fp8q_orthogonalize_f16, L.fp8q_orthogonalize_workspace_bytes(2, 133, 270, BF16)
    #       0  1    2  3   4   5  6       7       8       9    10 11  12    13
    good = [X, F32, 2, 133, 270, 5, 3.4445, -4.775, 2.0315, 0.5, Y, WS, need, None]
    refuses(f, good, [
        (1, 2, DTYPE), (2, -1, SHAPE), (3, -1, SHAPE), (4, -1, SHAPE), (5, 0, SHAPE), (5, 101, SHAPE),
        (6, NAN, SHAPE), (7, INF, SHAPE), (8, 4.0, SHAPE), (9, INF, SHAPE), (12, need // 4, SHAPE),
        (3, 65537, LARGE), (4, 65537, LARGE), (2, 65536, LARGE), (0, None, NULL), (10, None, NULL), (11, None, NULL),
        (0, X + 2, ALIGN), (10, Y + 1, ALIGN), (11, WS + 8, ALIGN)])
    assert f(None, F32, 0, 33, 70, 5, 2.0, -1.5, 0.5, 1.0, None, None, 0, None) == 0


def test_the_workspace_is_that_of_two_numbers_a_value():
    """X, both X^T, A and B, in two parts each, whatever out's type."""
    size = _lib().fp8q_orthogonalize_workspace_bytes
    for L, M, N in ((1, 512, 512), (2, 333, 1000), (1, 4096, 700)):
        m, n = ((v + 63) // 64 * 64 for v in (min(M, N), max(M, N)))
        assert size(L, M, N, BF16) == size(L, M, N, F32) >= L * 2 * (6 * m * n + 4 * m * m)


def test_polynomials_with_a_vanishing_last_coefficient():
    """s (8.4 - 7.4 s^2) has its top, 3.44, inside [0, 1]; a last coefficient near nothing changes neither that nor
    that s (2 - 1.5 s^2) stays below 3. 0.1 s (1 - s^2)^2 is flat at its double root."""
    f = _lib().fp8q_orthogonalize

    def status(steps, a, b, c):
        return f(None, F32, 1, 4, 4, steps, a, b, c, 1.0, Y, F32, WS, 1 << 40, None)
    for c in (0.0, 1e-45, 1e-30, 1e-20, -1e-20, 1e-10, -1e-10, 1e-6):
        assert status(1, 8.4, -7.4, c) == SHAPE, c
        assert status(5, 2.0, -1.5, c) == NULL, c
        assert status(1, -8.4, 7.4, c) == SHAPE, c
    assert status(9, 0.1, -0.2, 0.1) == NULL and status(9, 0.0, 0.0, 0.0) == NULL and status(1, 0.0, 0.0, 2.9) == NULL
    assert status(1, 0.0, 7.0, 1e-20) == SHAPE and status(1, 0.0, 2.9, 1e-20) == NULL


def test_rows_of_the_normalization():
    """2^22 rows are refused only where a row takes 1024 threads."""
    L = _lib()
    size, f = L.fp8q_norm_bwd_workspace_bytes, L.fp8q_norm
    for M, K, ok in ((1 << 22, 64, True), ((1 << 23) - 1, 128, True), ((1 << 23) - 1, 12288, True), (1 << 23, 64, False),
                     ((1 << 22) - 1, 16384, True), (1 << 22, 12289, False)):
        assert (size(M, K, 1) > 0) == ok, (M, K)
        # (the missing x is looked at after the sizes)
        assert f(None, BF16, K, None, 0, X, None, F32, 1e-6, 1, M, K, Y, F32, None, None) == (NULL if ok else LARGE), (M, K)
    # (nor do sizes pass whose threads, counted in 64 bits, wrap)
    for M in (1 << 31, 1 << 55, 1 << 56, (1 << 63) - 1):
        assert size(M, 64, 1) == -1 and f(None, BF16, 64, None, 0, X, None, F32, 1e-6, 1, M, 64, Y, F32, None, None) == LARGE, M
