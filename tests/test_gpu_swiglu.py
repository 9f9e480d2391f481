"""The gated activation, its FP8 form and its gradient on the GPU, against float64.

u = 2^-24. t = exp(-gate) is within 4 u (the hardware's power of two 2 u, a last multiply-add u, what its
argument lacks less than u), 1 / (1 + t) within 3 u of its own argument's (the sum u, the hardware's
reciprocal 2 u), so the sigmoid is within 7 u and y = gate s up within 9 u. A gate below -87 counts as -87:
that is worth 2^-118 of `up`, at most."""

import numpy as np
import pytest

from conftest import gpu_available
from fp8_fine_grained_online_amd import synthetic as S
from oracle import e4m3, step

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

U = 2.0 ** -24


def torch_dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def tensor(a, dtype="f32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch_dtype(dtype)).cuda()


def host(t):
    return t.double().cpu().numpy()


def half_step(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 0.0


def gate_up(M, I, seed, dtype="bf16", wide=0):
    """Gates over the whole range that matters, among them the far ends."""
    rng = S.rng_for(seed, M + I)
    x = 4 * rng.standard_normal((M, 2 * I + wide))
    ends = np.array([0.0, -0.0, 20.0, -20.0, -60.0, -86.9, -87.1, -104.0, 100.0, 1e30, -1e30, 1e-30, -1.2785, 3e38, -3e38])
    at = rng.integers(0, I, (M, 4))
    np.put_along_axis(x, at, ends[rng.integers(0, ends.size, (M, 4))], axis=1)
    return tensor(x, dtype)[:, :2 * I]


def forward_tol(gu, want):
    I = gu.shape[1] // 2
    return 10 * U * np.abs(want) + 2.0 ** -118 * np.abs(gu[:, I:]) + 2.0 ** -126


SIZES = [(1, 1), (1, 7), (3, 8), (2, 9), (5, 128), (33, 200), (1, 2048), (300, 257), (7, 4100), (2500, 24)]


@pytest.mark.parametrize("M,I", SIZES)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_swiglu(M, I, dtype, out):
    import torch
    import fp8_fine_grained_online_amd as F
    gu = gate_up(M, I, 3200, dtype, wide=(M % 3) * 5)
    y = torch.full((M + 1, I), 7.0, dtype=torch_dtype(out), device="cuda")
    got = host(F.fp8q_swiglu(gu, out_dtype=out, y=y[:M]))
    want = step.swiglu(host(gu))
    tol = forward_tol(host(gu), want)
    tol += half_step(out) * (np.abs(want) + tol)
    fits = np.abs(want) < 3.3e38  # beyond, an infinity
    assert np.all(np.abs(got - want)[fits] <= tol[fits]), float(np.max((np.abs(got - want) / tol)[fits]))
    assert np.all(np.isinf(got[~fits]) | (np.abs(got[~fits]) > 3.3e38))
    assert torch.all(y[M] == 7.0)


@pytest.mark.parametrize("M,I", SIZES)
@pytest.mark.parametrize("dtype,ddtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_swiglu_bwd(M, I, dtype, ddtype):
    import torch
    import fp8_fine_grained_online_amd as F
    gu = gate_up(M, I, 3210, dtype, wide=(M % 2) * 3)
    dy = tensor(S.rng_for(3211, M + I).standard_normal((M, I + 2)), ddtype)[:, :I]
    dgu = torch.full((M + 1, 2 * I), 7.0, dtype=torch_dtype(dtype), device="cuda")
    got = host(F.fp8q_swiglu_bwd(dy, gu, dgu=dgu[:M]))
    x, d = host(gu), host(dy)
    want = step.swiglu_bwd(d, x)
    gate, up = x[:, :I], x[:, I:]
    s, c = step.sigmoid(gate), step.sigmoid(-gate)
    y = gate * s
    # slope = s + y (1 - s): 7 u of s, 8 + 7 + 1 of the product, one of the sum; then two products
    tol_gate = U * np.abs(d * up) * (7 * s + 17 * np.abs(y * c) + 3 * np.abs(s + y * c)) + 2.0 ** -111 * np.abs(d * up)
    tol_up = 10 * U * np.abs(d * y) + 2.0 ** -118 * np.abs(d)
    tol = np.concatenate([tol_gate, tol_up], axis=1) + 2.0 ** -126
    tol += half_step(dtype) * (np.abs(want) + tol)
    fits = np.abs(want) < 3.3e38
    # dy up is formed first: where it overflows, so does the gradient
    fits[:, :I] &= np.abs(d * up) < 3.3e38
    fits[:, I:] &= np.abs(y) < 3.3e38
    assert np.all(np.abs(got - want)[fits] <= tol[fits]), float(np.max((np.abs(got - want) / tol)[fits]))
    assert torch.all(dgu[M] == 7.0)


@pytest.mark.parametrize("M,I", [(1, 128), (8, 2048), (33, 384), (700, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_swiglu_quant(M, I, dtype):
    """Scales within the value's error; codes those of the quotient, which is off by the value's and the scale's."""
    import fp8_fine_grained_online_amd as F
    rng = S.rng_for(3220, M + I)
    gu = 3 * rng.standard_normal((M, 2 * I))
    gu[0, I:I + 128] = 0.0  # a tile of nothing
    gu = tensor(gu, dtype)
    q, sa = F.fp8q_swiglu_quant_act_1x128(gu)
    want = step.swiglu(host(gu)).reshape(M, -1, 128)
    amax = np.abs(want).max(2)
    assert sa.shape == (M, I // 128) and np.all(np.abs(host(sa) - amax / 448) <= 11 * U * amax / 448)
    assert not q[0, :128].view(-1).remainder(128).any() and sa[0, 0] == 0
    quotient = want / np.where(amax > 0, amax / 448, 1.0)[:, :, None]
    got = e4m3.decode(q.cpu().numpy()).reshape(M, -1, 128)
    lo, hi = (e4m3.decode(e4m3.encode(quotient + s * 22 * U * np.abs(quotient))) for s in (-1, 1))
    assert np.all((got >= lo) & (got <= hi))
    assert np.mean(lo != hi) < 1e-3  # nearly every code is fixed


@pytest.mark.parametrize("G,used", [(1, [128]), (3, [128, 0, 256]), (4, [0, 0, 0, 0])])
def test_rows_behind_the_last_block(G, used):
    import torch
    import fp8_fine_grained_online_amd as F
    M, I = 640, 256
    off = torch.tensor(np.concatenate([[0], np.cumsum(used)]).astype(np.int32), device="cuda")
    last = int(off[-1])
    gu = gate_up(M, I, 3230)
    gu[last:] = float("nan")
    dy = tensor(S.rng_for(3231, 0).standard_normal((M, I)), "bf16")
    y = torch.full((M, I), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.full((M, I), 9, dtype=torch.uint8, device="cuda")
    sa = torch.full((M, I // 128), 5.0, device="cuda")
    dgu = torch.full((M, 2 * I), 7.0, dtype=torch.bfloat16, device="cuda")
    F.fp8q_swiglu(gu, m_offsets=off, y=y)
    F.fp8q_swiglu_quant_act_1x128(gu, m_offsets=off, q=q, sa=sa)
    F.fp8q_swiglu_bwd(dy, gu, m_offsets=off, dgu=dgu)
    for got, fill, want in ((y, 7.0, F.fp8q_swiglu(gu)), (q, 9, F.fp8q_swiglu_quant_act_1x128(gu)[0]),
                            (sa, 5.0, F.fp8q_swiglu_quant_act_1x128(gu)[1]), (dgu, 7.0, F.fp8q_swiglu_bwd(dy, gu))):
        # bit for bit: tiles whose product overflows have a scale that is not finite
        assert torch.equal(got[:last].view(torch.uint8), want[:last].view(torch.uint8)) and torch.all(got[last:] == fill)
    # offsets outside the rows are clamped
    for bad, rows in ((M + 1000, M), (-5, 0)):
        off[-1] = bad
        y.fill_(7.0)
        F.fp8q_swiglu(torch.zeros_like(gu), m_offsets=off, y=y)
        assert int((y == 0).all(1).sum()) == rows


def test_gates_that_are_not_finite():
    import torch
    import fp8_fine_grained_online_amd as F
    inf, nan = float("inf"), float("nan")
    gu = tensor([[-inf, inf, nan, 1.0, 2.0, 2.0, 2.0, nan]])
    y = F.fp8q_swiglu(gu, out_dtype="f32")[0]
    assert abs(y[0]) < 2.0 ** -117 and y[1] == inf and torch.isnan(y[2:]).all()
    d = F.fp8q_swiglu_bwd(torch.ones(1, 4, device="cuda"), gu)[0]
    assert d[0] == 0 and d[1] == 2.0 and torch.isnan(d[2:4]).all()
    assert abs(d[4]) < 2.0 ** -117 and d[5] == inf and torch.isnan(d[6]) and torch.isfinite(d[7])


def test_against_differences():
    """sum(y dy) along a direction, from the forward call, against the gradient call: the difference's own
    error is 10 u of each term over the step, the third derivative's that of float64's difference."""
    import fp8_fine_grained_online_amd as F
    M, I, t = 8, 130, 2.0 ** -7
    rng = S.rng_for(3240, 0)
    x, v = (np.round(2 * rng.standard_normal((M, 2 * I)) * 256) / 256 for _ in range(2))
    dy = np.round(rng.standard_normal((M, I)) * 256) / 256
    up, down = (host(F.fp8q_swiglu(tensor(x + s * t * v), out_dtype="f32")) for s in (1, -1))
    slope = ((up - down) * dy).sum(1) / (2 * t)
    got = host(F.fp8q_swiglu_bwd(tensor(dy), tensor(x)))
    third = np.abs(((step.swiglu(x + t * v) - step.swiglu(x - t * v)) * dy).sum(1) / (2 * t)
                   - (step.swiglu_bwd(dy, x) * v).sum(1))
    noise = 10 * U * ((np.abs(up) + np.abs(down)) * np.abs(dy)).sum(1) / (2 * t) + 40 * U * (np.abs(got) * np.abs(v)).sum(1)
    assert np.all(np.abs(slope - (got * v).sum(1)) <= third + noise)


def test_refusals():
    import torch
    import fp8_fine_grained_online_amd as F
    gu = gate_up(4, 128, 3250)
    dy = torch.zeros(4, 128, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    for call in (lambda: F.fp8q_swiglu(gu[:, :255]), lambda: F.fp8q_swiglu(gu.t()), lambda: F.fp8q_swiglu(gu[:1].expand(4, 256)),
                 lambda: F.fp8q_swiglu(gu, m_offsets=off[:1]), lambda: F.fp8q_swiglu(gu, m_offsets=off.cpu()),
                 lambda: F.fp8q_swiglu_bwd(dy[:3], gu), lambda: F.fp8q_swiglu_bwd(dy[:, :64], gu),
                 lambda: F.fp8q_swiglu(gu, y=dy[:, :64].bfloat16())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        F.fp8q_swiglu(gu, m_offsets=off.long())
    with pytest.raises(TypeError):
        F.fp8q_swiglu(gu.half())
    with pytest.raises(F.Fp8qError):
        F.fp8q_swiglu_quant_act_1x128(gu[:, :200])
    for shape in ((0, 256), (4, 0)):
        assert F.fp8q_swiglu(torch.empty(shape, device="cuda")).shape == (shape[0], shape[1] // 2)
