"""The MoE layer's calls together, as a layer uses them: forward in INT8 and in FP8,
backward through the way back, the router and the sorted rows, in a captured graph
with changing inputs, and on streams of the caller's."""

import numpy as np
import pytest

from conftest import gpu_available
from helpers import to_dev, to_dev_bf16
from fp8_fine_grained_online_amd import synthetic as S
from oracle import int8, route, tokens

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

T, G, TOPK, K, N = 150, 16, 4, 256, 384
ROUTE = {"score": "sigmoid", "renormalize": True, "scale": 2.5, "n_groups": 4, "topk_groups": 2}


def inputs(seed):
    import torch
    rng = S.rng_for(2800 + seed, 0)
    f = {"x": to_dev_bf16(S.activations(T, K, rng)),
         "logits": to_dev(rng.standard_normal((T, G)).astype(np.float32)),
         "bias": to_dev((0.1 * rng.standard_normal(G)).astype(np.float32)),
         "up": to_dev_bf16(np.stack([S.weights(2 * N, K, rng) for _ in range(G)])),
         "down": to_dev_bf16(np.stack([S.weights(K, N, rng) for _ in range(G)])),
         "dy": to_dev_bf16(S.activations(T, K, rng))}
    f["logits"][3] = -float("inf")  # a padded token: no expert may be chosen
    torch.cuda.synchronize()
    return f


def forward(f, qw):
    """The layer in INT8; every intermediate, and no host synchronization."""
    import torch
    import fp8_fine_grained_online_amd as F
    (qu, su), (qd, sd) = qw
    ids, w = F.fp8q_moe_route(f["logits"], TOPK, bias=f["bias"], **ROUTE)
    xp, off, rows = F.fp8q_moe_permute(f["x"], ids, G)
    M = xp.shape[0]
    # rows behind the last block are not written: what is read there stays behind it
    q1, s1 = F.fp8q_quant_int8_rows(xp)
    h = F.int8_gemm_grouped(q1, s1, qu, su, off, "bf16", c=torch.zeros(M, 2 * N, dtype=torch.bfloat16, device="cuda"))
    gate, up = h.float().chunk(2, dim=1)
    act = (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)
    q2, s2 = F.fp8q_quant_int8_rows(act)
    c = F.int8_gemm_grouped(q2, s2, qd, sd, off, "bf16", c=torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"))
    y = F.fp8q_moe_combine(c, rows, w)
    return dict(ids=ids, w=w, xp=xp, off=off, rows=rows, q1=q1, s1=s1, h=h, act=act, q2=q2, s2=s2, c=c, y=y)


def backward(f, o):
    import fp8_fine_grained_online_amd as F
    import torch
    dc, dw = F.fp8q_moe_combine_bwd(f["dy"], o["c"], o["rows"], o["w"], o["off"], dc=torch.zeros_like(o["c"]))
    kw = {k: ROUTE[k] for k in ("score", "renormalize", "scale")}
    dlogits = F.fp8q_moe_route_bwd(f["logits"], o["ids"], dw, **kw)
    dx = F.fp8q_moe_combine(dc, o["rows"], out_dtype="f32")  # as if the experts were the identity
    return dict(dc=dc, dw=dw, dlogits=dlogits, dx=dx)


def weights(f):
    import fp8_fine_grained_online_amd as F
    return F.fp8q_quant_int8_rows(f["up"]), F.fp8q_quant_int8_rows(f["down"])


def host(t):
    return t.float().cpu().numpy() if t.dtype.is_floating_point else t.cpu().numpy()


def test_int8_layer_step_by_step():
    """Every step of the run is its oracle's on the run's own inputs to that step."""
    import torch
    f = inputs(0)
    qw = weights(f)
    o = {k: host(v) for k, v in forward(f, qw).items()}
    (qu, su), (qd, sd) = [(host(q), host(s)) for q, s in qw]
    ids, w = route.route(host(f["logits"]), TOPK, host(f["bias"]).astype(np.float64), **ROUTE)
    assert np.array_equal(o["ids"], ids) and (ids[3] == -1).all()
    assert np.allclose(o["w"], w, rtol=2.0 ** -23, atol=0)
    xp, off, rows = tokens.permute(host(f["x"]), ids, G)
    M = int(off[-1])
    assert np.array_equal(o["off"], off) and np.array_equal(o["rows"], rows) and np.array_equal(o["xp"][:M], xp)

    def product(q, s, qb, sb):
        return torch.from_numpy(int8.gemm_grouped(q[:M], s[:M], qb, sb, off)).bfloat16().float().numpy()
    for src, q, s in (("xp", "q1", "s1"), ("act", "q2", "s2")):
        want_q, want_s = int8.quant_rows(o[src][:M])
        assert np.array_equal(o[q][:M], want_q) and np.array_equal(o[s][:M], want_s)
    assert np.array_equal(o["h"][:M], product(o["q1"], o["s1"], qu, su))
    assert np.array_equal(o["c"][:M], product(o["q2"], o["s2"], qd, sd))
    assert not o["c"][M:].any()
    want, mag = tokens.combine(o["c"], rows, o["w"])
    # one rounding per term, then one to bfloat16 (half a step: 2^-8)
    slack = TOPK * 2.0 ** -24 * mag
    assert np.all(np.abs(o["y"] - want) <= slack + 2.0 ** -8 * (np.abs(want) + slack))
    assert not o["y"][3].any()  # the padded token


def test_fp8_dispatch_and_way_back():
    """The FP8 dispatch's row map serves the way back and its gradient."""
    import torch
    import fp8_fine_grained_online_amd as F
    f = inputs(1)
    ids, w = F.fp8q_moe_route(f["logits"], TOPK, bias=f["bias"], **ROUTE)
    q, s, off, rows = F.fp8q_moe_dispatch_1x128(f["x"], ids, G)
    qb, sb = F.fp8q_quant_weight_128x128(f["up"])
    c = F.fp8_gemm_grouped(q, s, qb, sb, off, "f32", c=torch.zeros(q.shape[0], 2 * N, device="cuda"))
    y = F.fp8q_moe_combine(c, rows, w, out_dtype="f32")
    want, mag = tokens.combine(host(c), host(rows), host(w))
    assert np.all(np.abs(host(y) - want) <= TOPK * 2.0 ** -24 * mag)
    dy = torch.randn_like(y)
    dc, dw = F.fp8q_moe_combine_bwd(dy, c, rows, w, off, dc=torch.zeros_like(c))
    want_dc, want_dw, mag = tokens.combine_bwd(host(dy), host(c), host(rows), host(w), host(off))
    M = int(off[-1])
    assert np.all(np.abs(host(dc) - want_dc)[:M] <= 2.0 ** -24 * np.abs(want_dc[:M]))
    assert np.all(np.abs(host(dw) - want_dw) <= (2 * N / 64 + 24) * 2.0 ** -24 * mag)


def test_layer_gradient_against_autograd():
    """dlogits and dx of y = sum_j w_j(logits) x W_e^T, ids held fixed, against float64 autograd."""
    import torch
    import fp8_fine_grained_online_amd as F
    rng = S.rng_for(2810, 0)
    x = torch.from_numpy(rng.standard_normal((T, K))).float()
    lg = torch.from_numpy(rng.standard_normal((T, G))).float()
    W = torch.from_numpy(rng.standard_normal((G, N, K)) * K ** -0.5).float()
    dy = torch.from_numpy(rng.standard_normal((T, N))).float()
    for score, renorm in (("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)):
        ids, w = F.fp8q_moe_route(lg.cuda(), TOPK, score=score, renormalize=renorm)
        xp, off, rows = F.fp8q_moe_permute(x.cuda(), ids, G)
        offs = off.tolist()
        c = torch.zeros(xp.shape[0], N, device="cuda")
        for e in range(G):
            c[offs[e]:offs[e + 1]] = (xp[offs[e]:offs[e + 1]].double() @ W[e].cuda().double().t()).float()
        dc, dw = F.fp8q_moe_combine_bwd(dy.cuda(), c, rows, w, off)
        dlg = F.fp8q_moe_route_bwd(lg.cuda(), ids, dw, score=score, renormalize=renorm)
        dxp = torch.zeros_like(xp)
        for e in range(G):
            dxp[offs[e]:offs[e + 1]] = (dc[offs[e]:offs[e + 1]].double() @ W[e].cuda().double()).float()
        dx = F.fp8q_moe_combine(dxp, rows, out_dtype="f32")

        x64, lg64 = x.double().requires_grad_(), lg.double().requires_grad_()
        p = torch.sigmoid(lg64) if score == "sigmoid" else torch.softmax(lg64, 1)
        w64 = p.gather(1, ids.cpu().long())
        if renorm:
            w64 = w64 / w64.sum(1, keepdim=True)
        out = torch.einsum("tk,tjnk->tjn", x64, W.double()[ids.cpu().long()])
        (w64.unsqueeze(2) * out).sum(1).mul(dy.double()).sum().backward()
        # dw's terms: K-term products rounded once (c), N of them summed in binary32 in a chain of at most
        # N / 64 + 24 roundings; dlogits is at most sum_j |dw_j| times 1. dx: w dy, the product and the sum
        # over choices are each rounded, at most TOPK + 3 roundings of the terms' magnitudes.
        mag_dw = torch.einsum("tn,tjn->tj", dy.double().abs(), out.detach().abs())
        bound = ((N / 64 + 26) * 2.0 ** -24) * mag_dw.sum(1, keepdim=True)
        assert torch.all((dlg.cpu().double() - lg64.grad).abs() <= bound)
        mag_dx = torch.einsum("tj,tn,tjnk->tk", w64.detach().abs(), dy.double().abs(), W.double()[ids.cpu().long()].abs())
        assert torch.all((dx.cpu().double() - x64.grad).abs() <= (TOPK + 4) * 2.0 ** -24 * mag_dx)


def test_layer_in_a_captured_graph():
    """Forward and backward captured once, replayed over changing inputs with other work in between."""
    import torch
    f = inputs(2)
    qw = weights(f)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        o = forward(f, qw)
        backward(f, o)
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        o = forward(f, qw)
        g = backward(f, o)
    for seed in (3, 4, 5, 3):
        new = inputs(seed)
        for k in ("x", "logits", "bias", "dy"):
            f[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        want = forward(f, qw)
        want_g = backward(f, want)
        torch.randn(1 << 20, device="cuda").sum().item()  # the program's own work
        M = int(want["off"][-1])
        behind = ("xp", "q1", "s1", "q2", "s2", "act")  # rows behind the last block hold anything
        for k in o:
            a, b = (o[k][:M], want[k][:M]) if k in behind else (o[k], want[k])
            assert torch.equal(a, b), (seed, k)
        for k in g:
            assert torch.equal(g[k], want_g[k]), (seed, k)


def test_many_tokens_in_a_captured_graph():
    """The permutation's counting and scanning kernels and their workspace, captured: enough slots for
    them to run, and other choices on every replay."""
    import torch
    import fp8_fine_grained_online_amd as F
    tok, experts, k = 3000, 40, 3
    x = torch.randn(tok, 64, device="cuda")
    logits = torch.randn(tok, experts, device="cuda")

    def step():
        ids, w = F.fp8q_moe_route(logits, k)
        xp, off, rows = F.fp8q_moe_permute(x, ids, experts, xp=torch.zeros(cap, 64, device="cuda"))
        y = F.fp8q_moe_combine(xp, rows, w, out_dtype="f32")
        dc, dw = F.fp8q_moe_combine_bwd(x, xp, rows, w, off, dc=torch.zeros_like(xp))
        return ids, w, xp, off, rows, y, dc, dw

    cap = F.lib().fp8q_moe_dispatch_max_rows(tok, k, experts)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = step()
    for _ in range(4):
        logits.normal_()
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    import torch
    fs = [inputs(6), inputs(7)]
    qws = [weights(f) for f in fs]
    want = [forward(f, q) for f, q in zip(fs, qws)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in fs]
    for _ in range(3):
        got = []
        for f, q, s in zip(fs, qws, streams):
            with torch.cuda.stream(s):
                got.append(forward(f, q))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for k in ("ids", "w", "rows", "off", "y"):
                assert torch.equal(a[k], b[k]), k


def test_stream_argument():
    """A stream given by handle: new outputs come from its pool and the work runs on it."""
    import torch
    import fp8_fine_grained_online_amd as F
    f = inputs(8)
    ids, w = F.fp8q_moe_route(f["logits"], TOPK, bias=f["bias"], **ROUTE)
    xp, off, rows = F.fp8q_moe_permute(f["x"], ids, G)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        ids2, w2 = F.fp8q_moe_route(f["logits"], TOPK, bias=f["bias"], stream=stream, **ROUTE)
        xp2, off2, rows2 = F.fp8q_moe_permute(f["x"], ids2, G, stream=stream)
        y2 = F.fp8q_moe_combine(xp2, rows2, w2, stream=stream)
        s.synchronize()
        M = int(off[-1])
        assert torch.equal(ids, ids2) and torch.equal(w, w2) and torch.equal(off, off2) and torch.equal(rows, rows2)
        assert torch.equal(xp[:M], xp2[:M]) and torch.equal(y2, F.fp8q_moe_combine(xp, rows, w))


def test_null_stream_by_handle():
    """Handle 0 is the default stream, whatever stream is current: its earlier work is waited for."""
    import torch
    import fp8_fine_grained_online_amd as F
    x = torch.zeros(64, 512, dtype=torch.bfloat16, device="cuda")
    late = torch.randn(64, 512, device="cuda").to(torch.bfloat16)
    want_q, want_s = F.fp8q_quant_int8_rows(late)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)  # about 10 ms on the default stream, then the values
    x.copy_(late)
    with torch.cuda.stream(side):
        q, s = F.fp8q_quant_int8_rows(x, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(q, want_q) and torch.equal(s, want_s)
