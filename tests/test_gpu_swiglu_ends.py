"""The gated activation at the ends of its types' range: far gates, products that overflow, gradients whose
factors do. u = 2^-24 is the largest relative error of a binary32 rounding."""

import numpy as np
import pytest

from conftest import gpu_available
from oracle import step

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

U = 2.0 ** -24


def tensor(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()


def host(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_codes_of_a_tile_that_overflows_are_its_own(dtype):
    """Whatever lies beside it: ordinary tiles, tiles of nothing, tiny ones; and it leaves their codes alone."""
    import torch
    import fp8_fine_grained_online_amd as F
    I = 1024
    gu = torch.randn(6, 2 * I, device="cuda", generator=torch.Generator("cuda").manual_seed(37))
    plain = gu.clone()
    gu[:, 5], gu[:, I + 5] = 1e20, 3e38 * torch.tensor([1, -1, 1, 1, -1, 1.0], device="cuda")
    for t in (gu, plain):
        t[1, I + 128:I + 256] = 0  # beside it in its wavefront
        t[2, I + 256:I + 384] *= 2.0 ** -80
        t[4, I + 768:I + 896] = 0
    base = gu[0, :128].clone(), gu[0, I:I + 128].clone()
    for m in range(1, 6):
        gu[m, :128], gu[m, I:I + 128] = base
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    q, sa = F.fp8q_swiglu_quant_act_1x128(gu.to(t))
    want, _ = F.fp8q_swiglu_quant_act_1x128(plain.to(t))
    assert not torch.isfinite(sa[:, 0]).any() and torch.isfinite(sa[:, 1:]).all()
    for m in range(1, 6):
        assert torch.equal(q[m, :128], q[0, :128]), m
    assert torch.equal(q[:, 128:], want[:, 128:])


def far_gates(I, dtype):
    """Gates about and below -87, and ordinary ones, with values of `up` that make the products ordinary numbers."""
    import torch
    rng = np.random.default_rng(38)
    gate = np.concatenate([rng.uniform(-130, -80, I - 8), [-86.5, -87.0, -87.5, -88.0, -104.0, -3.0, 5.0, 90.0]])
    exact = torch.from_numpy(gate.astype(np.float32)).to(dtype).double().numpy()
    up = np.minimum(np.exp(np.minimum(-exact, 80.0)), 1e30) * rng.choice([-1.5, 0.75], I)
    return torch.from_numpy(np.concatenate([gate, up])[None].astype(np.float32)).to(dtype).cuda()


@pytest.mark.parametrize("I", [128, 129])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_gates(I, dtype):
    """The value is gate exp(gate) up to any distance: the sigmoid at -87 is within 7 u, exp(gate + 87) within 4 u and
    what its argument lacks: gate + 87 is rounded where gate is a float32 beyond -174 only, which is not here. Four
    products more: 16 u."""
    import torch
    import fp8_fine_grained_online_amd as F
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    gu = far_gates(I, t)
    x = host(gu)
    want = step.swiglu(x)
    got = host(F.fp8q_swiglu(gu, out_dtype="f32"))
    tol = 16 * U * np.abs(want) + 2.0 ** -149
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / tol))
    dy = torch.from_numpy(np.random.default_rng(39).standard_normal((1, I)).astype(np.float32)).cuda()
    d, gate, up = host(dy), x[:, :I], x[:, I:]
    got = host(F.fp8q_swiglu_bwd(dy, gu))
    want = step.swiglu_bwd(d, x)
    s, c = step.sigmoid(gate), step.sigmoid(-gate)
    tol = np.concatenate([U * np.abs(d * up) * (11 * s + 21 * np.abs(gate * s * c) + 7 * np.abs(s + gate * s * c)), 16 * U * np.abs(d * gate * s)], 1)
    tol += (2.0 ** -8 if dtype == "bf16" else 0.0) * (np.abs(want) + tol) + 2.0 ** -133
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / tol))


def test_the_farthest_gates_give_nothing():
    import fp8_fine_grained_online_amd as F
    inf = float("inf")
    gu = tensor([[-200.0, -1e4, -3e38, -inf, 3e38, -3e38, 3e38, 2.0]])
    assert not F.fp8q_swiglu(gu, out_dtype="f32").any()
    import torch
    assert not F.fp8q_swiglu_bwd(torch.ones(1, 4, device="cuda"), gu).any()


def test_a_tile_of_far_gates_has_their_scale():
    """1x128 tiles whose values all come from far gates."""
    import torch
    import fp8_fine_grained_online_amd as F
    gu = far_gates(128, torch.float32)
    gu[:, 120:128] = -95.0
    want = np.abs(step.swiglu(host(gu))).max() / 448
    q, sa = F.fp8q_swiglu_quant_act_1x128(gu)
    assert abs(float(sa[0, 0]) - want) <= 18 * U * want
    assert abs(q.view(torch.float8_e4m3fn).float().abs().max().item() - 448) == 0


def test_one_far_gate_leaves_the_others_as_they_are():
    import torch
    import fp8_fine_grained_online_amd as F
    for t in (torch.bfloat16, torch.float32):
        gu = (3 * torch.randn(3, 512, device="cuda", generator=torch.Generator("cuda").manual_seed(40))).to(t)
        far = gu.clone()
        far[1, 77] = -99.0
        dy = torch.randn(3, 256, device="cuda").to(t)
        for f in (lambda x: F.fp8q_swiglu(x, out_dtype="f32"), lambda x: F.fp8q_swiglu_bwd(dy, x)):
            a, b = f(gu), f(far)
            b[1, 77] = a[1, 77]
            if a.shape[1] == 512:
                b[1, 256 + 77] = a[1, 256 + 77]
            assert torch.equal(a, b)


def test_gradients_whose_factors_overflow():
    """dy up beyond binary32, the gradient within: three products and the slope, as elsewhere."""
    import fp8_fine_grained_online_amd as F
    gate = np.array([-40.0, -60.0, -86.0, -100.0, -120.0, -10.0, -5.0, -1.2784645])
    up = np.array([1e20, 1e20, 3e38, 1e25, 3e38, -1e21, 2.0, 1e20])
    d = np.array([1e20, -1e20, 1e20, 1e30, 3e38, 1e18, 3.3e38, 1e19])
    gu = tensor(np.concatenate([gate, up])[None])
    dy = tensor(d[None])
    x, d = host(gu), host(dy)
    gate, up = x[:, :8], x[:, 8:]
    got = host(F.fp8q_swiglu_bwd(dy, gu))
    want = step.swiglu_bwd(d, x)
    s, c = step.sigmoid(gate), step.sigmoid(-gate)
    tol = np.concatenate([U * np.abs(d * up) * (11 * s + 21 * np.abs(gate * s * c) + 7 * np.abs(s + gate * s * c)), 16 * U * np.abs(d * gate * s)], 1)
    assert np.all(np.isfinite(got)) and np.all(np.abs(want) < 3e38)
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / tol))
    # what does overflow is an infinity
    assert F.fp8q_swiglu_bwd(tensor([[1e20]]), tensor([[2.0, 1e20]]))[0, 0] == float("inf")


def test_more_values_than_32_bits_count():
    """Rows at either side of 2^31 values of gu and of y, and the last, are the smaller call's, bit for bit."""
    import torch
    import fp8_fine_grained_online_amd as F
    M, I = 1050000, 2176
    gu = torch.empty(M, 2 * I, device="cuda", dtype=torch.bfloat16).normal_(generator=torch.Generator("cuda").manual_seed(41))
    parts = [slice(0, 3)] + [slice((1 << 31) // w - 2, (1 << 31) // w + 3) for w in (2 * I, I)] + [slice(M - 3, M)]
    y = F.fp8q_swiglu(gu)
    for p in parts:
        assert torch.equal(y[p], F.fp8q_swiglu(gu[p]))
    q, sa = F.fp8q_swiglu_quant_act_1x128(gu)
    for p in parts:
        q1, s1 = F.fp8q_swiglu_quant_act_1x128(gu[p])
        assert torch.equal(q[p], q1) and torch.equal(sa[p], s1)
    del q, sa
    dgu = F.fp8q_swiglu_bwd(y, gu)
    for p in parts:
        assert torch.equal(dgu[p], F.fp8q_swiglu_bwd(y[p], gu[p]))
