"""What an orthogonalized update may be off by, on matrices whose roundings could add up, and the form with one
FP16 number a value.

The default form keeps every operand as two FP16 numbers, off by h = 2^-22 of the value. Where all values of
a plane share one magnitude those roundings go the same way, and a singular value s takes per step

  h (s^3 |b + 2 c s^2| (2 + 1) + 2 s |b s^2 + c s^4| + 1)   (X twice in A, A; B and X in the update; X)

For the default polynomial, whose iterates of equal singular values stay in [0.68, 1.21], that is at most (3 * 1.9
+ 2 * 3.1 + 1) h < 13 h; a step passes it on with a slope of at most 1.7 there on the mean, over five steps at most
19 * 13 h < 2^-14. What binary32's own sums are off by comes on top: at most four times what the same steps in
binary32 are off by.

A bfloat16 result is that of the same arithmetic, rounded once: bit for bit the float32 result's rounding."""

import numpy as np
import pytest

from conftest import gpu_available
from fp8_fine_grained_online_amd import synthetic as S
from oracle import step
from test_gpu_ortho import COEFFS, SHAPES, binary32, bound, dev, fro, host, matrix

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

F32_COEFFS = tuple(float(np.float32(v)) for v in COEFFS)


def alike(M, N, kind):
    """Matrices of few magnitudes."""
    rng = S.rng_for(3600, M * 7 + N)
    if kind == "constant":
        return np.ones((M, N))
    if kind == "signs":
        return np.sign(rng.standard_normal((M, 1))) @ np.sign(rng.standard_normal((1, N)))
    if kind == "identity":
        return np.eye(M, N)
    g = np.zeros((M, N))  # "blocks": equal values on the diagonal's blocks, of a magnitude each
    for i in range(0, min(M, N), 16):
        g[i:i + 16, i:i + 16] = 1.0 + rng.random()
    return g


def equal_when_rounded(g, **kw):
    """The float32 result, whose rounding the bfloat16 one is."""
    import torch
    import fp8_fine_grained_online_amd as F
    exact = F.fp8q_orthogonalize(g, out_dtype="f32", **kw)
    assert torch.equal(F.fp8q_orthogonalize(g, out_dtype="bf16", **kw), exact.bfloat16())
    return exact


@pytest.mark.parametrize("M,N", [(531, 595), (307, 371), (325, 389), (566, 566), (201, 402), (200, 333), (333, 200), (40, 60), (90, 1700)])
@pytest.mark.parametrize("kind", ["constant", "signs", "identity", "blocks"])
def test_matrices_of_few_magnitudes(M, N, kind):
    g = dev(alike(M, N, kind), "f32")
    got = host(equal_when_rounded(g))
    want = step.orthogonalize(host(g), 5, F32_COEFFS)
    assert fro(got - want) <= 4 * fro(binary32(host(g), 5, F32_COEFFS) - want) + 2.0 ** -14 * fro(want)


@pytest.mark.parametrize("M,N", [(1024, 2048), (2100, 1900), (1230, 1294)])
@pytest.mark.parametrize("kind", ["constant", "blocks"])
def test_large_matrices_of_few_magnitudes(M, N, kind):
    """The tiles' kernels, against float64 on the GPU."""
    import torch
    g = dev(alike(M, N, kind), "f32")
    got = equal_when_rounded(g).double()
    a, b, c = F32_COEFFS

    def steps(x):
        x = x / torch.linalg.norm(x)
        x = x.t().contiguous() if M > N else x
        for _ in range(5):
            A = x @ x.t().contiguous()
            x = a * x + (b * A + c * (A @ A)) @ x
        return (x.t() if M > N else x).double()
    want = steps(g.double())
    off = torch.linalg.norm(steps(g) - want)
    assert torch.linalg.norm(got - want) <= 4 * off + 2.0 ** -14 * torch.linalg.norm(want)


@pytest.mark.parametrize("steps", [8, 10, 20])
@pytest.mark.parametrize("kind", ["gauss", "floor"])
def test_many_steps(steps, kind):
    """As near the definition as the same steps in binary32; `floor`: one strong direction over much weaker ones."""
    M, N = 300, 400
    rng = S.rng_for(3610, 0)
    g = rng.standard_normal((M, N))
    if kind == "floor":
        g = 1e-3 * g + rng.standard_normal((M, 1)) @ rng.standard_normal((1, N))
    g = dev(g, "f32")
    got = host(equal_when_rounded(g, steps=steps))
    want = step.orthogonalize(host(g), steps, F32_COEFFS)
    assert fro(got - want) <= 4 * fro(binary32(host(g), steps, F32_COEFFS) - want) + 2.0 ** -22 * fro(want)


def test_a_steep_polynomial():
    coeffs = (7.5, -7.5, 0.0)
    rng = S.rng_for(3620, 0)
    g = dev(1e-3 * rng.standard_normal((200, 300)) + rng.standard_normal((200, 1)) @ rng.standard_normal((1, 300)), "f32")
    got = host(equal_when_rounded(g, steps=1, coeffs=coeffs))
    want = step.orthogonalize(host(g), 1, coeffs)
    assert fro(got - want) <= 4 * fro(binary32(host(g), 1, coeffs) - want) + 2.0 ** -18 * fro(want)


@pytest.mark.parametrize("L,M,N", [(1, m, n) for m, n in SHAPES] + [(5, 300, 150), (3, 250, 140), (1, 256, 300), (1, 600, 4200)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_shape_rounds_once(L, M, N, dtype):
    g = dev(np.stack([matrix(M, N, "gauss", 3630 + i) for i in range(L)]), dtype)
    equal_when_rounded(g, scale=-0.2)


# ---------------------------------------------------------------------------
# one FP16 number a value
# ---------------------------------------------------------------------------
def check_single(g, got, said):
    """Within the rounding analysis, and within what the documentation says."""
    want = step.orthogonalize(g, 5, F32_COEFFS)
    off = min(bound(g, 5, F32_COEFFS, True), said * fro(want))
    assert fro(got - want) <= off + 2.0 ** -8 * fro(want), fro(got - want) / fro(want)


@pytest.mark.parametrize("L,M,N", [(1, m, n) for m, n in SHAPES if min(m, n) > 128] + [(5, 300, 150), (3, 250, 140), (1, 256, 300),
                                   (1, 500, 350), (1, 130, 4200), (1, 600, 4200), (8, 190, 240)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_single(L, M, N, dtype):
    import torch
    import fp8_fine_grained_online_amd as F
    kinds = ("gauss", "few", "decay")
    g = dev(np.stack([matrix(M, N, kinds[i % 3], 3640 + i) for i in range(L)]), dtype)
    o = torch.full((L * M * N + 5,), 7.0, dtype=torch.bfloat16, device="cuda")
    F.fp8q_orthogonalize(g, out=o[:L * M * N].view(L, M, N), single=True)
    assert torch.all(o[L * M * N:] == 7.0)
    for i in range(L):
        check_single(host(g[i]), host(o[:L * M * N].view(L, M, N)[i]), 2e-3)


@pytest.mark.parametrize("M,N", [(531, 595), (307, 371), (201, 402)])
@pytest.mark.parametrize("kind", ["constant", "signs", "identity", "blocks"])
def test_single_of_few_magnitudes(M, N, kind):
    import fp8_fine_grained_online_amd as F
    g = dev(alike(M, N, kind), "f32")
    check_single(host(g), host(F.fp8q_orthogonalize(g, single=True)), 1.2e-2)


@pytest.mark.parametrize("M,N", [(1024, 4096), (2100, 1900), (4096, 700)])
def test_single_in_the_larger_tiles(M, N):
    import torch
    import fp8_fine_grained_online_amd as F
    g = torch.randn(M, N, device="cuda", generator=torch.Generator("cuda").manual_seed(M + N))
    exact = F.fp8q_orthogonalize(g, out_dtype="f32")
    got = F.fp8q_orthogonalize(g, single=True).float()
    assert torch.linalg.norm(got - exact) <= (2e-3 + 2.0 ** -8) * torch.linalg.norm(exact)


def test_single_of_few_rows_is_the_other_form():
    """Up to 128 rows there is nothing to gain, and the result is the exact form's."""
    import torch
    import fp8_fine_grained_online_amd as F
    for M, N in ((16, 100), (128, 700), (900, 128)):
        g = dev(matrix(M, N, "gauss", 3650), "f32")
        assert torch.equal(F.fp8q_orthogonalize(g, single=True), F.fp8q_orthogonalize(g))


def test_single_in_a_captured_graph_and_on_a_stream():
    import torch
    import fp8_fine_grained_online_amd as F
    g = torch.randn(300, 200, device="cuda")
    need = F.lib().fp8q_orthogonalize_workspace_bytes(1, 300, 200, F.FP8Q_OUT_BF16)
    space = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    F.fp8q_orthogonalize(g, workspace=space[:need], stream=stream, single=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = F.fp8q_orthogonalize(g, workspace=space[:need], single=True)
    for _ in range(3):
        g.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, F.fp8q_orthogonalize(g, single=True)) and torch.all(space[need:] == 0xFF)
    with pytest.raises(ValueError):
        F.fp8q_orthogonalize(g, out_dtype="f32", single=True)


# a matrix in a workgroup, the joint kernel, a gram in runs of K, blocks of 16 and 32, tiles, tall ones
PATHS = [(30, 40), (128, 700), (16, 8192), (200, 333), (333, 500), (700, 333), (600, 640), (900, 800), (1400, 1400), (1500, 2000),
         (2100, 1900)]


@pytest.mark.parametrize("M,N", PATHS)
@pytest.mark.parametrize("out,single", [("f32", False), ("bf16", False), ("bf16", True)])
def test_what_is_not_finite_fills_its_matrix(M, N, out, single):
    """An infinity or NaN reaches every value of its own matrix (A A has it everywhere), whatever the way, and no other's."""
    import torch
    import fp8_fine_grained_online_amd as F
    g = torch.randn(3, M, N, device="cuda", generator=torch.Generator("cuda").manual_seed(M))
    want = F.fp8q_orthogonalize(g, out_dtype=out, single=single)[1]
    g[0, M - 1, N // 2], g[2, M // 3, N - 1] = float("nan"), -float("inf")
    got = F.fp8q_orthogonalize(g, out_dtype=out, single=single)
    assert torch.isnan(got[0]).all() and torch.isnan(got[2]).all() and torch.equal(got[1], want)
    # and alone, which may go another way
    assert torch.isnan(F.fp8q_orthogonalize(g[0], out_dtype=out, single=single)).all()
    assert torch.isnan(F.fp8q_orthogonalize(g[2], out_dtype=out, single=single)).all()


@pytest.mark.parametrize("M,N", [(1, 65536), (65536, 1), (65536, 3), (60, 65536), (65536, 64), (129, 65535)])
@pytest.mark.parametrize("out,single", [("f32", False), ("bf16", True)])
def test_the_longest_sides(M, N, out, single):
    """Matrices of one direction, +-1 / sqrt(M N): the result is the polynomial of 1, with that direction."""
    import torch
    import fp8_fine_grained_online_amd as F
    gen = torch.Generator("cuda").manual_seed(M + N)
    u, v = (torch.randint(0, 2, (k,), device="cuda", generator=gen).float() * 2 - 1 for k in (M, N))
    got = F.fp8q_orthogonalize(u[:, None] * v[None], out_dtype=out, single=single).float()
    s = 1.0
    a, b, c = F32_COEFFS
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    want = s / np.sqrt(M * N)
    # (of two numbers: 2^-14 as at the top, and binary32 sums of 65536 products, 4 sqrt(65536) 2^-24 in each of three
    # products of five steps; of one number 1.2e-2 and the rounding)
    tol = 2.0 ** -14 + 15 * 4 * 256 * 2.0 ** -24 if out == "f32" else 1.2e-2 + 2.0 ** -8
    assert float((got * (u[:, None] * v[None]) - want).abs().max()) <= tol * want


@pytest.mark.parametrize("L,M,N", [(65535, 3, 5), (500, 130, 140), (1200, 70, 300), (3000, 700, 1050)])
@pytest.mark.parametrize("single", [False, True])
def test_many_matrices(L, M, N, single):
    """As many as the call takes; and more values than 32 bits count. Matrices from here and there against the same alone."""
    import torch
    import fp8_fine_grained_online_amd as F
    gen = torch.Generator("cuda").manual_seed(L)
    g = torch.randn(L, M, N, device="cuda", generator=gen, dtype=torch.bfloat16)
    got = F.fp8q_orthogonalize(g, single=single)
    for i in (0, 1, L // 2, L - 2, L - 1):
        want = F.fp8q_orthogonalize(g[i], out_dtype="f32")
        # the exact form, alone, may sum in another order (4e-5 at most, as documented); one FP16 number 2e-3
        tol = (2e-3 if single and min(M, N) > 128 else 8e-5) + 2.0 ** -8
        assert torch.linalg.norm(got[i].float() - want) <= tol * torch.linalg.norm(want), i
