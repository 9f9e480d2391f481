"""GPU router and its gradient against the float64 oracle: ids equal, weights and
gradients within the one rounding to the output type."""

import numpy as np
import pytest

from conftest import gpu_available
from fp8_fine_grained_online_amd import synthetic as S
from oracle import route

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # half a step, relative
TINY = 2.0 ** -149                              # and of a subnormal, absolute (binary32)


def logits_of(T, G, dtype, seed, ties=False, masked=0.0):
    import torch
    rng = S.rng_for(seed, 0)
    x = 1.5 * rng.standard_normal((T, G))
    if ties:
        x = np.round(x)  # many equal scores
    if masked:
        x[rng.random((T, G)) < masked] = -np.inf
    t = torch.from_numpy(x).to(torch.float32 if dtype == "f32" else torch.bfloat16).cuda()
    return t, t.double().cpu().numpy()


def check(x_dev, x, topk, bias=None, **kw):
    import torch
    import fp8_fine_grained_online_amd as F
    b = None if bias is None else torch.from_numpy(bias).float().cuda()
    T = x.shape[0]
    ids = torch.full((T, topk), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, topk), float("nan"), device="cuda")
    F.fp8q_moe_route(x_dev, topk, bias=b, topk_ids=ids, weights=w, **kw)
    want_ids, want_w = route.route(x, topk, None if b is None else b.double().cpu().numpy(), **kw)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = w.double().cpu().numpy()
    # float64 arithmetic (a few hundred roundings of 2^-53 at most), then one rounding to binary32
    assert np.all(np.abs(got - want_w) <= np.abs(want_w) * (HALF["f32"] + 2.0 ** -44) + TINY)
    return ids, want_ids


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("T,G,topk,dtype", [(1, 1, 1, "f32"), (1, 256, 8, "f32"), (7, 63, 6, "bf16"),
                                            (33, 65, 10, "f32"), (130, 128, 64, "bf16"), (5, 1024, 8, "f32"),
                                            (65, 257, 3, "bf16"), (9, 520, 9, "f32")])
def test_route(T, G, topk, dtype, score, renormalize):
    xd, x = logits_of(T, G, dtype, 2200 + T)
    bias = 0.1 * S.rng_for(2200, G).standard_normal(G) if T % 2 else None
    check(xd, x, topk, bias, score=score, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("G,groups,kept,topk", [(256, 8, 4, 8), (256, 8, 1, 8), (60, 6, 2, 7), (64, 64, 5, 5),
                                                (24, 2, 2, 10), (1024, 2, 1, 8), (128, 16, 3, 1)])
@pytest.mark.parametrize("ties", [False, True])
def test_groups(G, groups, kept, topk, ties):
    xd, x = logits_of(37, G, "f32", 2300 + G, ties=ties)
    check(xd, x, topk, score="sigmoid", n_groups=groups, topk_groups=kept)
    check(xd, x, topk, score="softmax", renormalize=False, n_groups=groups, topk_groups=kept)


@pytest.mark.parametrize("G,groups,kept,topk", [(88, 4, 2, 8), (96, 8, 3, 9), (160, 32, 7, 10), (360, 8, 4, 8),
                                                (520, 4, 2, 10), (1000, 8, 5, 64), (1024, 64, 9, 8), (1023, 31, 8, 12),
                                                (66, 33, 12, 10), (300, 2, 1, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_that_end_inside_lanes(G, groups, kept, topk, score):
    """Several experts per lane and groups that are no power-of-two run of whole lanes (and one that is, of 16 per
    lane): with ties, masked logits and a bias."""
    for seed, ties, masked in ((2410, False, 0.0), (2411, True, 0.0), (2412, False, 0.6), (2413, True, 0.97)):
        xd, x = logits_of(41, G, "f32" if seed % 2 else "bf16", seed + G, ties=ties, masked=masked)
        bias = S.rng_for(seed, G).standard_normal(G)
        if ties:
            bias = np.round(bias)
        check(xd, x, topk, score=score, n_groups=groups, topk_groups=kept)
        check(xd, x, topk, 0.2 * bias, score=score, renormalize=False, scale=2.5, n_groups=groups, topk_groups=kept)


def test_ties_go_to_the_lowest_index():
    xd, x = logits_of(200, 100, "bf16", 2400, ties=True)
    check(xd, x, 9, score="softmax")
    check(xd, x, 9, score="sigmoid", bias=np.round(S.rng_for(2401, 0).standard_normal(100)))


def test_masked_logits_and_empty_rows():
    import torch
    xd, x = logits_of(64, 40, "f32", 2402, masked=0.9)
    xd[3], x[3] = -float("inf"), -np.inf   # nothing left
    xd[5], x[5] = float("nan"), np.nan
    xd[6, 7], x[6, 7] = float("nan"), np.nan
    for kw in ({"score": "softmax"}, {"score": "sigmoid", "renormalize": False},
               {"score": "sigmoid", "n_groups": 8, "topk_groups": 3}):
        ids, want = check(xd, x, 6, **kw)
        assert (want[3] == -1).all() and (want[5] == -1).all() and (want == -1).sum() > 40
        g = torch.ones(64, 6, device="cuda")
        kw = {k: v for k, v in kw.items() if k in ("score", "renormalize")}
        import fp8_fine_grained_online_amd as F
        d = F.fp8q_moe_route_bwd(xd, ids, g, **kw).cpu().numpy()
        assert np.isfinite(d).all() and not d[3].any() and not d[5].any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_masked_bias_bars_the_choice_alone(score, renormalize):
    """An expert with a bias of -infinity or NaN is never chosen, and its logit still counts in the softmax."""
    xd, x = logits_of(50, 40, "f32", 2406)
    bias = 0.1 * S.rng_for(2407, 0).standard_normal(40)
    bias[[3, 17, 18, 19]] = -np.inf
    bias[[5, 30]] = np.nan
    for kw in ({}, {"n_groups": 8, "topk_groups": 3}, {"n_groups": 20, "topk_groups": 4}):
        _, want = check(xd, x, 5, bias, score=score, renormalize=renormalize, **kw)
        assert not np.isin(want, [3, 17, 18, 19, 5, 30]).any()
    p = route.scores(x, score)
    if score == "softmax" and not renormalize:
        import fp8_fine_grained_online_amd as F
        import torch
        b = torch.from_numpy(bias).float().cuda()
        ids, w = F.fp8q_moe_route(xd, 34, bias=b, score=score, renormalize=False)
        free = np.setdiff1d(np.arange(40), [3, 17, 18, 19, 5, 30])
        # 34 weights rounded to binary32, and their sum in float64
        assert np.allclose(w.double().cpu().numpy().sum(1), p[:, free].sum(1), rtol=2.0 ** -24 + 2.0 ** -44, atol=0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_logits_at_any_element(dtype):
    """Contiguous logits that start one element past an aligned address."""
    import torch
    xd, x = logits_of(33, 256, dtype, 2404)
    shifted = torch.empty(33 * 256 + 1, dtype=xd.dtype, device="cuda")[1:].view(33, 256)
    shifted.copy_(xd)
    check(shifted, x, 8, score="sigmoid", n_groups=8, topk_groups=4)
    check(shifted, x, 8, score="softmax", renormalize=False)


def test_logits_past_32_bits():
    import torch
    import fp8_fine_grained_online_amd as F
    T, G = 4200000, 1024  # 8.6 GB
    xd, x = logits_of(5, G, "bf16", 2405)
    big = torch.zeros((T, G), dtype=torch.bfloat16, device="cuda")
    big[-5:] = xd
    ids, w = F.fp8q_moe_route(big, 6, score="softmax")
    few, wf = F.fp8q_moe_route(xd, 6, score="softmax")
    assert torch.equal(ids[-5:], few) and torch.equal(w[-5:], wf)
    assert torch.equal(ids[0], torch.arange(6, dtype=torch.int32, device="cuda"))
    d = F.fp8q_moe_route_bwd(big, ids, w)
    assert torch.equal(d[-5:], F.fp8q_moe_route_bwd(xd, few, wf))


def test_extreme_logits():
    """Scores that underflow, saturate, or differ in the last bit of binary32."""
    import torch
    x = torch.tensor([[100.0, -100.0, 3e38, -3e38, 0.0, 1e-38, 88.0, 800.0],
                      [1.0, 1.0 + 2 ** -23, 1.0, 1.0 - 2 ** -24, 0, 0, 0, 0]], device="cuda")
    for score in ("softmax", "sigmoid"):
        check(x, x.double().cpu().numpy(), 5, score=score)
        check(x, x.double().cpu().numpy(), 8, score=score, renormalize=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("T,G,topk,dtype", [(1, 1, 1, "f32"), (3, 256, 8, "f32"), (70, 64, 6, "bf16"),
                                            (17, 100, 10, "f32"), (6, 1024, 64, "bf16"), (9, 300, 2, "f32")])
def test_gradient(T, G, topk, dtype, score, renormalize):
    import torch
    import fp8_fine_grained_online_amd as F
    xd, x = logits_of(T, G, dtype, 2500 + T)
    rng = S.rng_for(2501, T)
    ids = np.argsort(rng.random((T, G)), axis=1)[:, :topk].astype(np.int32)
    if T > 2 and topk > 1:
        ids[1, 0] = -1
        ids[2, 1] = G        # not an expert
        ids[0, 1] = ids[0, 0]  # listed twice
    g = rng.standard_normal((T, topk)).astype(np.float32)
    d = torch.full((T, G), float("nan"), dtype=xd.dtype, device="cuda")
    F.fp8q_moe_route_bwd(xd, torch.from_numpy(ids).cuda(), torch.from_numpy(g).cuda(), score=score,
                         renormalize=renormalize, scale=2.5, dlogits=d)
    want = route.route_bwd(x, ids, g, score, renormalize, 2.5)
    # float64 with cancellation against the row's sum of |g| (a few hundred roundings), then one
    # rounding to binary32 and one to the output type
    slack = 2.0 ** -44 * 2.5 * np.abs(g).sum(1, keepdims=True)
    half = HALF["f32"] + (HALF["bf16"] if dtype == "bf16" else 0.0)
    assert np.all(np.abs(d.double().cpu().numpy() - want) <= half * (1 + 2.0 ** -8) * np.abs(want) + slack + TINY)


# rows of two chosen logits whose probabilities underflow, or nearly, and of ordinary ones beside them
FAR = [(-707, -706), (-720, -721), (-745.5, -744), (-800, -801), (-3e38, -2e38), (-720, 3), (0, -750), (40, -40),
       (-709.5, -709.25), (-1, 0.5)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_renormalized_gradient_of_far_logits(score, dtype):
    """The renormalized weights are ratios: their gradient is ordinary however small the probabilities are."""
    import torch
    import fp8_fine_grained_online_amd as F
    x = np.array([(1.0, a, 0.25, b, -2.0) for a, b in FAR])
    xd = torch.from_numpy(x).to(torch.float32 if dtype == "f32" else torch.bfloat16).cuda()
    ids = np.tile(np.array([[3, 1]], np.int32), (len(FAR), 1))
    g = np.array([(200.0, -200.0), (1.0, -2.0)] * (len(FAR) // 2), np.float32)
    d = F.fp8q_moe_route_bwd(xd, torch.from_numpy(ids).cuda(), torch.from_numpy(g).cuda(), score=score, scale=2.5)
    want = route.route_bwd(xd.double().cpu().numpy(), ids, g, score, True, 2.5)
    assert (np.abs(want[:4]).max(axis=1) > 0.1).all()
    # as in test_gradient
    slack = 2.0 ** -44 * 2.5 * np.abs(g).sum(1, keepdims=True)
    half = HALF["f32"] + (HALF["bf16"] if dtype == "bf16" else 0.0)
    assert np.all(np.abs(d.double().cpu().numpy() - want) <= half * (1 + 2.0 ** -8) * np.abs(want) + slack + TINY)


@pytest.mark.parametrize("score,renormalize", [("softmax", False), ("sigmoid", True)])
def test_bfloat16_gradient_is_rounded_once(score, renormalize):
    """Gradients go from float64 to bfloat16 in one rounding: two (by way of binary32) would move about one value in
    2^17 across the middle between two bfloat16 numbers."""
    import torch
    import fp8_fine_grained_online_amd as F
    T, G, topk = 8192, 256, 8
    gen = torch.Generator("cuda").manual_seed(7)
    x = (1.5 * torch.randn(T, G, device="cuda", generator=gen)).to(torch.bfloat16)
    ids = torch.rand(T, G, device="cuda", generator=gen).topk(topk, 1).indices.int().contiguous()
    g = torch.randn(T, topk, device="cuda", generator=gen)
    if renormalize:  # few gradients of a row are not 0: more rows
        ids, topk = torch.arange(G, device="cuda").int().repeat(T, 1)[:, :64].contiguous(), 64
        g = torch.randn(T, topk, device="cuda", generator=gen)
    d = F.fp8q_moe_route_bwd(x, ids, g, score=score, renormalize=renormalize).double().cpu().numpy()
    x64, at, g64 = x.double().cpu().numpy(), ids.cpu().numpy(), g.double().cpu().numpy()
    p = route.scores(x64, score)
    pj = np.take_along_axis(p, at, 1)
    want = np.zeros_like(p)
    if renormalize:
        q = pj / pj.sum(1, keepdims=True)
        np.put_along_axis(want, at, q * (1 - pj) * (g64 - (g64 * q).sum(1, keepdims=True)), 1)
    else:
        dp = np.zeros_like(p)
        np.put_along_axis(dp, at, g64, 1)
        want = p * (dp - (dp * p).sum(1, keepdims=True))
    # half a step of a value 1.b 2^e is 2^(e-8); beyond it only float64's own errors
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -120))) - 7)
    slack = 2.0 ** -44 * np.abs(g64).sum(1, keepdims=True)
    assert np.all(np.abs(d - want) <= step / 2 + slack)


def test_sigmoid_of_far_logits():
    """Probabilities below 2^-1022 order the experts down to float64's smallest; then they tie."""
    import torch
    x = np.array([[-709.5, -709.25, -720, -715, -744, -746, -800, -3e38], [-701, -700, -699, -700.5, -1, 1, 30, -30]],
                 np.float32)
    ids, want = check(torch.from_numpy(x).cuda(), x.astype(np.float64), 8, score="sigmoid", renormalize=False)
    assert want[0].tolist() == [1, 0, 3, 2, 4, 5, 6, 7]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_renormalized_weights_that_underflow(score):
    """A bias steers the choice to experts whose probabilities are 0 in float64: their weights are still the ratios."""
    import torch
    x = np.array([(1.0, a, 0.25, b, -2.0, a - 0.5) for a, b in FAR]).astype(np.float32)
    bias = np.array([-9.0, 0, -9.0, 0, -9.0, 0])
    xd = torch.from_numpy(x).cuda()
    x64 = x.astype(np.float64)
    ids, want = check(xd, x64, 2, bias, score=score)
    assert set(want[3]) <= {1, 3, 5}
    check(xd, x64, 3, bias, score=score, scale=2.5)
    check(xd, x64, 6, bias, score=score)          # beside experts with ordinary probabilities
    check(xd, x64, 2, score=score, bias=np.array([-9.0, -9, 0, 0, -9, 0]), n_groups=3, topk_groups=2)
    x = np.array([[-709.5, -709.25, -720, -715, -744, -746, -800, -3e38], [-701, -700, -699, -700.5, -1, 1, 30, -30]],
                 np.float32)
    for topk in (2, 8):
        check(torch.from_numpy(x).cuda(), x.astype(np.float64), topk, score=score)


def test_no_tokens():
    import torch
    import fp8_fine_grained_online_amd as F
    x = torch.empty((0, 16), device="cuda")
    ids, w = F.fp8q_moe_route(x, 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    assert F.fp8q_moe_route_bwd(x, ids, w).shape == (0, 16)


def test_refusals():
    import torch
    import fp8_fine_grained_online_amd as F
    x = torch.zeros(4, 16, device="cuda")
    for bad in (lambda: F.fp8q_moe_route(x, 0), lambda: F.fp8q_moe_route(x, 17),
                lambda: F.fp8q_moe_route(x, 5, n_groups=4, topk_groups=1),
                lambda: F.fp8q_moe_route(x, 2, n_groups=3), lambda: F.fp8q_moe_route(x, 2, scale=float("nan"))):
        with pytest.raises(F.Fp8qError):
            bad()
    with pytest.raises(ValueError):
        F.fp8q_moe_route(x, 2, score="tanh")
    with pytest.raises(TypeError):
        F.fp8q_moe_route(x.double(), 2)
    with pytest.raises(ValueError):
        F.fp8q_moe_route(x.t(), 2)
    with pytest.raises(ValueError):
        F.fp8q_moe_route(x, 2, bias=torch.zeros(15, device="cuda"))


def test_too_many_choices_allocate_nothing():
    import torch
    import fp8_fine_grained_online_amd as F
    x = torch.zeros(4, 16, device="cuda")
    for topk in (17, 10 ** 12, 2 ** 62):
        before = torch.cuda.memory_reserved()
        with pytest.raises(F.Fp8qError):
            F.fp8q_moe_route(x, topk)
        assert torch.cuda.memory_reserved() == before
    with pytest.raises(F.Fp8qError):
        F.fp8q_moe_route(x, 17, topk_ids=torch.zeros(4, 17, dtype=torch.int32, device="cuda"),
                         weights=torch.zeros(4, 17, device="cuda"))
