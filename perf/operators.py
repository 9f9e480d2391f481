"""Cases that time the MoE layer's operators around the experts' products, and the 8-bit integer product.

Three operators, each in the directions a layer needs:

* route: router scores (softmax or sigmoid, an optional selection bias, experts chosen inside the
  best groups) -> expert ids and weights; and its gradient;
* tokens: rows sorted by expert into the grouped GEMM's padded layout (permute), back with the
  router's weights (combine), and the gradient of the way back;
* int8: a linear layer in 8-bit integers with one scale per token and one per output channel,
  dense and per expert (grouped).

`run` computes the plain form, elementary torch operations, or with `own` the framework's kernels.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TILE = 128  # rows of an expert's block are padded to a multiple of this
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _pkg():
    import fp8_fine_grained_online_amd as F
    return F


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a serving step's routing: 16 tokens, 256 experts in 8 groups of which 4 may be used
        {"name": "route_decode_16x256", "op": "route", "T": 16, "G": 256, "topk": 8, "dtype": "f32",
         "score": "sigmoid", "bias": True, "renorm": True, "scale": 2.5, "groups": 8, "topk_groups": 4},
        # a training batch's routing: softmax over 64 experts, bf16 logits, weights as they are
        {"name": "route_train_8192x64", "op": "route", "T": 8192, "G": 64, "topk": 6, "dtype": "bf16",
         "score": "softmax", "bias": False, "renorm": False, "scale": 1.0, "groups": 1, "topk_groups": 1},
        # the router's gradient for a training batch of 256 experts
        {"name": "route_bwd_8192x256", "op": "route_bwd", "T": 8192, "G": 256, "topk": 8, "dtype": "f32",
         "score": "sigmoid", "renorm": True, "scale": 2.5},
        # one serving step's tokens to 32 experts
        {"name": "permute_decode_16", "op": "permute", "T": 16, "G": 32, "topk": 8, "K": 7168, "dtype": "bf16",
         "drop": 0.0},
        # a training batch's tokens to 32 experts
        {"name": "permute_train_8192", "op": "permute", "T": 8192, "G": 32, "topk": 8, "K": 7168, "dtype": "bf16",
         "drop": 0.0},
        # the same batch's way back, weighted
        {"name": "combine_train_8192", "op": "combine", "T": 8192, "G": 32, "topk": 8, "K": 7168, "dtype": "bf16",
         "out": "bf16", "weighted": True, "drop": 0.0},
        # a ragged batch's input gradient: rows summed without weights, some choices dropped, fp32 out
        {"name": "combine_ragged_1237", "op": "combine", "T": 1237, "G": 64, "topk": 6, "K": 2056, "dtype": "bf16",
         "out": "f32", "weighted": False, "drop": 0.05},
        # the gradient of the way back for a training batch
        {"name": "combine_bwd_8192", "op": "combine_bwd", "T": 8192, "G": 32, "topk": 8, "K": 7168, "dtype": "bf16",
         "drop": 0.0},
        # single-token serving: one row through a 7168 x 7168 layer
        {"name": "int8_token_7168x7168", "op": "int8", "M": 1, "N": 7168, "K": 7168, "out": "bf16"},
        # a ragged prompt: sizes that end inside every tile
        {"name": "int8_ragged_333x2050x2064", "op": "int8", "M": 333, "N": 2050, "K": 2064, "out": "f32"},
        # an ordinary large product
        {"name": "int8_4096x4096x4096", "op": "int8", "M": 4096, "N": 4096, "K": 4096, "out": "bf16"},
        # the experts' up projection for a training batch
        {"name": "int8_grouped_8192_top8_g32", "op": "int8_grouped", "T": 8192, "G": 32, "topk": 8, "N": 4096,
         "K": 7168, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _up(n, m):
    return (n + m - 1) // m * m


def draw(rng):
    op = rng.choice(["route", "route_bwd", "permute", "combine", "combine_bwd", "int8", "int8", "int8_grouped"])
    if op in ("route", "route_bwd"):
        groups = rng.choice([1, 1, 4, 8]) if op == "route" else 1
        G = _up(_log(rng, 8, 512), groups * 2)
        topk = min(rng.randint(1, 10), G)
        tg = 1
        if groups > 1:
            tg = rng.randint(1, groups)
            topk = min(topk, tg * (G // groups))
        c = {"op": op, "T": _log(rng, 1, 16384), "G": G, "topk": topk, "dtype": rng.choice(["bf16", "f32"]),
             "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.5,
             "scale": rng.choice([1.0, 2.5])}
        if op == "route":
            c.update(bias=rng.random() < 0.5, groups=groups, topk_groups=tg)
        return c
    if op in ("permute", "combine", "combine_bwd"):
        G = _log(rng, 2, 256)
        topk = min(rng.randint(1, 8), G)
        T = _log(rng, 1, 8192)
        K = _up(_log(rng, 64, 7168), 8)
        c = {"op": op, "T": T, "G": G, "topk": topk, "K": K, "dtype": rng.choice(["bf16", "bf16", "f32"]),
             "drop": rng.choice([0.0, 0.1])}
        if c["dtype"] == "f32":
            c["T"] = max(1, T // 2)
        if op == "combine":
            c.update(out=rng.choice(["bf16", "f32"]), weighted=rng.random() < 0.7)
        return c
    if op == "int8":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 32, 8192), "K": _up(_log(rng, 64, 8192), 16),
                "out": rng.choice(["bf16", "f32"])}
    return {"op": op, "T": _log(rng, 4, 8192), "G": _log(rng, 2, 32), "topk": rng.randint(1, 8),
            "N": _log(rng, 64, 4096), "K": _up(_log(rng, 128, 7168), 16), "out": rng.choice(["bf16", "f32"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _activations(rows, cols, g):
    """N(0, 1) with one value in a thousand a hundred times larger."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x *= torch.where(torch.rand(rows, cols, generator=g, device=DEV) < 0.001, 100.0, 1.0)
    return x


def _routing(T, G, topk, drop, g):
    """Distinct experts per token, uniform; a share `drop` of the choices dropped (-1)."""
    ids = torch.rand(T, G, generator=g, device=DEV).topk(topk, dim=1).indices.to(torch.int32)
    if drop:
        ids = torch.where(torch.rand(T, topk, generator=g, device=DEV) < drop, torch.full_like(ids, -1), ids)
    return ids.contiguous()


def _cap(T, topk, G):
    return _up(T * topk + (TILE - 1) * G, TILE)


def _layout(ids, G):
    """(row of each slot or -1, offsets of the experts' padded blocks), both int32, without a host wait."""
    T, topk = ids.shape
    flat = ids.reshape(-1).long()
    valid = (flat >= 0) & (flat < G)
    e = torch.where(valid, flat, torch.full_like(flat, G))
    counts = torch.zeros(G + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, e, torch.ones_like(e))
    padded = (counts[:G] + TILE - 1) // TILE * TILE
    off = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    first = counts.cumsum(0) - counts
    es, order = torch.sort(e, stable=True)
    row = off[es.clamp(max=G - 1)] + torch.arange(e.numel(), device=e.device) - first[es]
    row = torch.where(es < G, row, torch.full_like(row, -1))
    rows = torch.empty_like(row).scatter_(0, order, row)
    return rows.reshape(T, topk).to(torch.int32), off.to(torch.int32)


def _slot_of_row(rows, M):
    """For each of M rows the slot that maps to it, or -1."""
    flat = rows.reshape(-1).long()
    at = torch.where((flat >= 0) & (flat < M), flat, torch.full_like(flat, M))
    slots = torch.arange(flat.numel(), device=flat.device)
    return torch.full((M + 1,), -1, dtype=torch.int64, device=flat.device).scatter_(0, at, slots)[:M]


def _quant_rows(x):
    """8-bit codes and one scale per row: s = amax / 127, q = round(x / s), each in 32 bits.
    (The divisor is a tensor: a division by a number may be done as a product.)"""
    xf = x.float()
    s = xf.abs().amax(dim=-1) / torch.full((), 127.0, device=x.device)
    q = torch.round(xf / torch.where(s > 0, s, torch.ones_like(s)).unsqueeze(-1)).clamp(-127, 127)
    return q, s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op in ("route", "route_bwd"):
        T, G = case["T"], case["G"]
        st["logits"] = (1.5 * torch.randn(T, G, generator=g, device=DEV)).to(DT[case["dtype"]])
        if op == "route":
            st["bias"] = 0.1 * torch.randn(G, generator=g, device=DEV) if case["bias"] else None
        else:
            st["ids"] = _routing(T, G, case["topk"], 0.0, g)
            st["dweights"] = torch.randn(T, case["topk"], generator=g, device=DEV)
        return st
    if op in ("permute", "combine", "combine_bwd"):
        T, G, topk, K, dt = case["T"], case["G"], case["topk"], case["K"], DT[case["dtype"]]
        M = _cap(T, topk, G)
        ids = _routing(T, G, topk, case["drop"], g)
        if op == "permute":
            st.update(x=_activations(T, K, g).to(dt), ids=ids, xp=torch.zeros(M, K, dtype=dt, device=DEV))
            return st
        st["rows"], st["off"] = _layout(ids, G)
        st["c"] = torch.randn(M, K, generator=g, device=DEV).to(dt)
        w = torch.rand(T, topk, generator=g, device=DEV)
        st["w"] = (w / w.sum(1, keepdim=True)).contiguous()
        if op == "combine":
            st["w"] = st["w"] if case["weighted"] else None
        else:
            st["dy"] = torch.randn(T, K, generator=g, device=DEV).to(dt)
            st["dc"] = torch.zeros(M, K, dtype=dt, device=DEV)
        return st
    N, K = case["N"], case["K"]
    if op == "int8":
        st["x"] = _activations(case["M"], K, g).to(torch.bfloat16)
        w = (0.02 * torch.randn(N, K, generator=g, device=DEV)).to(torch.bfloat16)
        q, st["sw"] = _quant_rows(w)
        st["qw"] = q.to(torch.int8)
        return st
    T, G, topk = case["T"], case["G"], case["topk"]
    topk = min(topk, G)
    M = _cap(T, topk, G)
    rows, st["off"] = _layout(_routing(T, G, topk, 0.0, g), G)
    slot = _slot_of_row(rows, M)
    x = _activations(T, K, g).to(torch.bfloat16)
    st["xp"] = torch.where((slot >= 0).unsqueeze(1), x[(slot // topk).clamp(min=0)], x.new_zeros(()))
    st["qw"] = torch.empty(G, N, K, dtype=torch.int8, device=DEV)
    st["sw"] = torch.empty(G, N, device=DEV)
    for e in range(G):
        q, st["sw"][e] = _quant_rows((0.02 * torch.randn(N, K, generator=g, device=DEV)).to(torch.bfloat16))
        st["qw"][e] = q.to(torch.int8)
    st["c"] = torch.zeros(M, N, dtype=DT[case["out"]], device=DEV)
    st["most"] = int((st["off"][1:] - st["off"][:-1]).max())  # the largest block, known to the host
    return st


# ---------------------------------------------------------------------------
# the passes
# ---------------------------------------------------------------------------
def run(state):
    c = state["case"]
    return {"route": _route, "route_bwd": _route_bwd, "permute": _permute, "combine": _combine,
            "combine_bwd": _combine_bwd, "int8": _int8, "int8_grouped": _int8_grouped}[c["op"]](state, c)


def _scores(logits, score):
    """Router probabilities in 64 bits: choices next to a border depend on every bit."""
    x = logits.double()
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    p = torch.exp(x - x.amax(dim=1, keepdim=True))
    return p / p.sum(dim=1, keepdim=True)


def _route(st, c):
    logits, bias = st["logits"], st["bias"]
    if own:
        return _pkg().fp8q_moe_route(logits, c["topk"], bias=bias, score=c["score"], renormalize=c["renorm"],
                                     scale=c["scale"], n_groups=c["groups"], topk_groups=c["topk_groups"])
    T, G = logits.shape
    p = _scores(logits, c["score"])
    z = p if bias is None else p + bias.double()
    if c["groups"] > 1:
        best = z.reshape(T, c["groups"], -1).sort(dim=2, descending=True).values[:, :, :2].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        open_ = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        z = torch.where(open_.repeat_interleave(G // c["groups"], dim=1), z, torch.full_like(z, -math.inf))
    ids = z.sort(dim=1, descending=True, stable=True).indices[:, :c["topk"]]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), (c["scale"] * w).float()


def _route_bwd(st, c):
    logits, ids, dw = st["logits"], st["ids"], st["dweights"]
    if own:
        return _pkg().fp8q_moe_route_bwd(logits, ids, dw, score=c["score"], renormalize=c["renorm"],
                                         scale=c["scale"])
    p = _scores(logits, c["score"])
    at = ids.long()
    pj, g = p.gather(1, at), dw.double() * c["scale"]
    if c["renorm"]:  # weights p_j / sum: dL/dp_j
        total = pj.sum(dim=1, keepdim=True)
        g = (g - (g * pj).sum(dim=1, keepdim=True) / total) / total
    dp = torch.zeros_like(p).scatter_add_(1, at, g)
    if c["score"] == "sigmoid":
        d = dp * p * (1 - p)
    else:
        d = p * (dp - (dp * p).sum(dim=1, keepdim=True))
    return d.to(logits.dtype)


def _permute(st, c):
    x, ids, xp = st["x"], st["ids"], st["xp"]
    if own:
        return _pkg().fp8q_moe_permute(x, ids, c["G"], xp=xp)
    rows, off = _layout(ids, c["G"])
    M = xp.shape[0]
    slot = _slot_of_row(rows, M)
    behind = (torch.arange(M, device=x.device) >= off[-1]).unsqueeze(1)
    filled = torch.where((slot >= 0).unsqueeze(1), x[(slot // ids.shape[1]).clamp(min=0)], x.new_zeros(()))
    xp.copy_(torch.where(behind, xp, filled))
    return xp, off, rows


def _combine(st, c):
    src, rows, w = st["c"], st["rows"], st["w"]
    if own:
        return _pkg().fp8q_moe_combine(src, rows, w, out_dtype=c["out"])
    got = src[rows.long().clamp(min=0)].float()
    if w is not None:
        got = got * w.unsqueeze(2)
    return torch.where((rows >= 0).unsqueeze(2), got, got.new_zeros(())).sum(dim=1).to(DT[c["out"]])


def _combine_bwd(st, c):
    dy, src, rows, w, off, dc = st["dy"], st["c"], st["rows"], st["w"], st["off"], st["dc"]
    if own:
        return _pkg().fp8q_moe_combine_bwd(dy, src, rows, w, off, dc=dc)
    M = src.shape[0]
    dot = (src[rows.long().clamp(min=0)].float() * dy.float().unsqueeze(1)).sum(dim=2)
    dw = torch.where(rows >= 0, dot, dot.new_zeros(()))
    slot = _slot_of_row(rows, M)
    at = slot.clamp(min=0)
    scaled = w.reshape(-1)[at].unsqueeze(1) * dy[at // rows.shape[1]].float()
    filled = torch.where((slot >= 0).unsqueeze(1), scaled, scaled.new_zeros(())).to(dc.dtype)
    behind = (torch.arange(M, device=dy.device) >= off[-1]).unsqueeze(1)
    dc.copy_(torch.where(behind, dc, filled))
    return dc, dw


def _int8(st, c):
    if own:
        F = _pkg()
        q, s = F.fp8q_quant_int8_rows(st["x"])
        return F.int8_gemm_scaled(q, s, st["qw"], st["sw"], out_dtype=c["out"])
    q, s = _quant_rows(st["x"])
    return (q @ st["qw"].float().t() * s.unsqueeze(1) * st["sw"]).to(DT[c["out"]])


def _blocks(off, most, M):
    """Row of each place of the experts' blocks laid side by side (G x most), M where there is none."""
    at = off[:-1].long().unsqueeze(1) + torch.arange(most, device=off.device)
    return torch.where(at < off[1:].long().unsqueeze(1), at, torch.full_like(at, M))


def _int8_grouped(st, c):
    xp, off, out = st["xp"], st["off"], st["c"]
    if own:
        F = _pkg()
        q, s = F.fp8q_quant_int8_rows(xp)
        return F.int8_gemm_grouped(q, s, st["qw"], st["sw"], off, out_dtype=c["out"], c=out)
    M = xp.shape[0]
    at = _blocks(off, st["most"], M)
    q, s = _quant_rows(xp)
    a = q[at.clamp(max=M - 1)]
    y = torch.bmm(a, st["qw"].float().transpose(1, 2).contiguous())
    y = (y * s[at.clamp(max=M - 1)].unsqueeze(2) * st["sw"].unsqueeze(1)).to(out.dtype)
    slot = torch.full((M + 1,), -1, dtype=torch.int64, device=xp.device)
    slot = slot.scatter_(0, at.reshape(-1), torch.arange(at.numel(), device=xp.device))[:M]
    inside = (torch.arange(M, device=xp.device) < off[-1]).unsqueeze(1)
    out.copy_(torch.where(inside, y.reshape(-1, y.shape[2])[slot.clamp(min=0)], out))
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _rows_expected(T, topk, G):
    """Rows of the padded layout for uniform routing: full tiles of the experts that got a token."""
    n = T * topk
    if n < 100 * G:  # at most about one tile each
        return G * (1 - (1 - min(topk, G) / G) ** T) * TILE
    return n + G * TILE / 2


def work(case):
    op = case["op"]
    if op in ("route", "route_bwd"):
        T, G, topk = case["T"], case["G"], case["topk"]
        es = 2 if case["dtype"] == "bf16" else 4
        if op == "route":
            return {"bytes": T * G * es + T * topk * 8 + (G * 4 if case["bias"] else 0), "flops": 8 * T * G}
        return {"bytes": 2 * T * G * es + T * topk * 8, "flops": 8 * T * G}
    if op in ("permute", "combine", "combine_bwd"):
        T, G, topk, K = case["T"], case["G"], case["topk"], case["K"]
        es = 2 if case["dtype"] == "bf16" else 4
        n = T * topk * (1 - case["drop"])
        rows = _rows_expected(T, topk, G)
        if op == "permute":
            return {"bytes": (T + rows) * K * es + T * topk * 8, "flops": 0}
        if op == "combine":
            eo = 2 if case["out"] == "bf16" else 4
            return {"bytes": n * K * es + T * K * eo + T * topk * (8 if case["weighted"] else 4), "flops": 2 * n * K}
        return {"bytes": (T + n + rows) * K * es + T * topk * 12, "flops": 3 * n * K}
    N, K = case["N"], case["K"]
    eo = 2 if case["out"] == "bf16" else 4
    if op == "int8":
        M = case["M"]
        return {"bytes": M * K * 2 + N * K + N * 4 + M * N * eo, "flops": 2 * M * N * K}
    topk = min(case["topk"], case["G"])
    n, rows = case["T"] * topk, _rows_expected(case["T"], topk, case["G"])
    return {"bytes": rows * K * 2 + case["G"] * N * (K + 4) + rows * N * eo, "flops": 2 * n * N * K}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "route":
        x = st["logits"].double()
        p = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
        z = p.cpu().numpy() + (0 if st["bias"] is None else st["bias"].double().cpu().numpy())
        if case["groups"] > 1:
            z = z.reshape(z.shape[0], case["groups"], -1)
            best = np.partition(z, -2, axis=2)[:, :, -2:].sum(2)
            rank = np.argsort(np.argsort(-best, axis=1, kind="stable"), axis=1)
            z = np.where((rank < case["topk_groups"])[:, :, None], z, -np.inf).reshape(z.shape[0], -1)
        ids = np.argsort(-z, axis=1, kind="stable")[:, :case["topk"]].copy()
        w = p.gather(1, torch.from_numpy(ids).to(p.device))
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return None, w * case["scale"]
    if op == "route_bwd":
        with torch.enable_grad():
            x = st["logits"].double().requires_grad_()
            p = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
            w = p.gather(1, st["ids"].long())
            if case["renorm"]:
                w = w / w.sum(1, keepdim=True)
            return torch.autograd.grad((case["scale"] * w * st["dweights"].double()).sum(), x)[0]
    if op == "permute":
        ids, xp = st["ids"].cpu().numpy().reshape(-1), st["xp"].double()
        slots = np.argsort(np.where(ids < 0, case["G"], ids), kind="stable")
        place, at, last = {}, 0, -1
        for slot in slots[:int((ids >= 0).sum())]:
            at = at if ids[slot] == last else _up(at, TILE)
            place[at], at, last = int(slot) // case["topk"], at + 1, ids[slot]
        xp[:_up(at, TILE)] = 0
        if place:
            to, src = (torch.tensor(list(v), device=DEV) for v in (place.keys(), place.values()))
            xp[to] = st["x"].double()[src]
        return xp, None, None
    if op in ("combine", "combine_bwd"):
        rows, w, src = st["rows"].long(), st["w"], st["c"]
        T, topk = rows.shape
        y = torch.zeros(T, case["K"], dtype=torch.float64, device=DEV)
        dw = torch.zeros(T, topk, dtype=torch.float64, device=DEV)
        if op == "combine_bwd":
            dc = st["dc"].double()
        for j in range(topk):
            t = torch.nonzero(rows[:, j] >= 0).squeeze(1)
            r = rows[t, j]
            if op == "combine":
                y[t] += src[r].double() * (w[t, j].double().unsqueeze(1) if w is not None else 1.0)
            else:
                d = st["dy"][t].double()
                dw[t, j] = torch.linalg.vecdot(src[r].double(), d)
                dc[r] = d * w[t, j].double().unsqueeze(1)
        return y if op == "combine" else (dc, dw)
    x = st["x"] if op == "int8" else st["xp"]
    x64 = x.double()
    s = (x64.abs().amax(1) / 127).float().double()  # the scale is kept in 32 bits
    quotient = x64 / torch.where(s > 0, s, torch.ones_like(s)).unsqueeze(1)
    q = torch.round(quotient.float().double()).clamp(-127, 127)  # codes are of the quotient in 32 bits
    if op == "int8":
        return torch.matmul(q, st["qw"].double().t()) * torch.outer(s, st["sw"].double())
    y = st["c"].double()
    off = st["off"].tolist()
    for e in range(case["G"]):
        r = slice(off[e], off[e + 1])
        y[r] = torch.matmul(q[r], st["qw"][e].double().t()) * torch.outer(s[r], st["sw"][e].double())
    return y
