"""Cases that time a training step's operators around the FP8 products of a layer.

Three operators, each in the directions a training step needs:

* norm: RMS or centred normalization of rows, with the residual sum before it; its gradient with
  the reduction of the weights' gradients over all rows;
* swiglu: the gated activation between an MLP's two products, as rows of 16 or 32 bits or as
  1x128 FP8 tiles, over plain rows or the experts' padded blocks; its gradient;
* orthogonalize: a weight gradient's update made orthogonal by Newton-Schulz products, for one
  matrix or one per expert.

`run` computes the plain form, elementary torch operations, or with `own` the framework's kernels.
"""

import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TILE = 128  # rows of an expert's block are padded to a multiple of this; columns of a quantized tile
FP8_MAX = 448.0
EPS = 1e-6
STEPS, COEFFS = 5, (3.4445, -4.7750, 2.0315)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _pkg():
    import fp8_fine_grained_online_amd as F
    return F


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of a serving step: residual sum and RMS normalization
        {"name": "norm_token_1x7168", "op": "norm", "T": 1, "K": 7168, "dtype": "bf16", "out": "bf16",
         "centred": False, "residual": True, "wide": 0},
        # a prompt of odd length, centred, columns of a wider fp32 projection
        {"name": "norm_ragged_1237x2050", "op": "norm", "T": 1237, "K": 2050, "dtype": "f32", "out": "f32",
         "centred": True, "residual": False, "wide": 64},
        # a training batch between two layers
        {"name": "norm_train_8192x7168", "op": "norm", "T": 8192, "K": 7168, "dtype": "bf16", "out": "bf16",
         "centred": False, "residual": True, "wide": 0},
        # a small batch's gradient, fp32, odd columns
        {"name": "norm_bwd_ragged_333x2049", "op": "norm_bwd", "T": 333, "K": 2049, "dtype": "f32", "dy": "f32",
         "centred": True, "residual": False, "wide": 0},
        # the training batch's gradient, the residual stream's added
        {"name": "norm_bwd_train_8192x7168", "op": "norm_bwd", "T": 8192, "K": 7168, "dtype": "bf16", "dy": "bf16",
         "centred": False, "residual": True, "wide": 0},
        # one token's eight experts, straight to FP8
        {"name": "swiglu_quant_token_8x2048", "op": "swiglu_quant", "T": 8, "I": 2048, "dtype": "bf16", "G": 0},
        # 8192 tokens of 8 choices in the experts' padded blocks, straight to FP8
        {"name": "swiglu_quant_experts_65536", "op": "swiglu_quant", "T": 65536, "I": 2048, "dtype": "bf16", "G": 32},
        # a dense MLP's gradient
        {"name": "swiglu_bwd_16384x2048", "op": "swiglu_bwd", "T": 16384, "I": 2048, "dtype": "bf16", "dy": "bf16",
         "G": 0},
        # a router's weight, fp32 throughout
        {"name": "orthogonalize_256x1024", "op": "orthogonalize", "L": 1, "M": 256, "N": 1024, "dtype": "f32",
         "out": "f32"},
        # a tall matrix whose sides end inside every tile
        {"name": "orthogonalize_ragged_1000x333", "op": "orthogonalize", "L": 1, "M": 1000, "N": 333,
         "dtype": "bf16", "out": "bf16"},
        # a square projection
        {"name": "orthogonalize_4096x4096", "op": "orthogonalize", "L": 1, "M": 4096, "N": 4096, "dtype": "bf16",
         "out": "bf16"},
        # four experts' fused gate and up projections, from fp32 weight gradients
        {"name": "orthogonalize_4x4096x7168", "op": "orthogonalize", "L": 4, "M": 4096, "N": 7168, "dtype": "f32",
         "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _up(n, m):
    return (n + m - 1) // m * m


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "swiglu", "swiglu_quant", "swiglu_bwd", "orthogonalize", "orthogonalize"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_bwd"):
        K = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            K = _up(K, 8)
        most = 8192 * 7168 // (1 if dtype == "bf16" else 2)
        c = {"op": op, "T": min(_log(rng, 1, 16384), most // K), "K": K, "dtype": dtype,
             "centred": rng.random() < 0.5, "residual": rng.random() < 0.5, "wide": rng.choice([0, 0, 64])}
        c["out" if op == "norm" else "dy"] = rng.choice(["bf16", "f32"]) if dtype == "bf16" else dtype
        return c
    if op != "orthogonalize":
        I = _log(rng, 64, 4096)
        I = _up(I, 128) if op == "swiglu_quant" else _up(I, 8) if rng.random() < 0.6 else I
        most = 65536 * 2048 // (2 if dtype == "bf16" else 4)
        c = {"op": op, "T": min(_log(rng, 1, 65536), most // I), "I": I, "dtype": dtype,
             "G": rng.choice([0, _log(rng, 2, 64)])}
        if op != "swiglu_quant":
            c["out" if op == "swiglu" else "dy"] = rng.choice(["bf16", "f32"]) if dtype == "bf16" else dtype
        return c
    return {"op": op, "L": rng.choice([1, 1, 2, 3]), "M": _log(rng, 16, 4096), "N": _log(rng, 16, 4096),
            "dtype": dtype, "out": rng.choice(["bf16", "bf16", "f32"])}


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


def _blocks(T, G, g):
    """Offsets (int32, G + 1) of T rows shared out between G experts at random, each block padded to whole
    tiles; and the rows that the worst sharing needs."""
    counts = torch.bincount(torch.randint(0, G, (T,), generator=g, device=DEV), minlength=G)
    padded = (counts + TILE - 1) // TILE * TILE
    off = torch.cat([padded.new_zeros(1), padded.cumsum(0)]).to(torch.int32)
    return off, _up(T + (TILE - 1) * G, TILE)


def _gradient(M, N, g):
    """A weight gradient: a few strong directions, a decaying tail, and noise."""
    r = min(64, M, N)
    s = 1.0 / (1.0 + torch.arange(r, device=DEV))
    return (torch.randn(M, r, generator=g, device=DEV) * s) @ torch.randn(r, N, generator=g, device=DEV) \
        + 0.05 * torch.randn(M, N, generator=g, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    op, st = case["op"], {"case": dict(case)}
    if op in ("norm", "norm_bwd"):
        T, K, dt = case["T"], case["K"], DT[case["dtype"]]
        st["x"] = _activations(T, K + case["wide"], g).to(dt)[:, :K]
        st["gamma"] = (1.0 + 0.1 * torch.randn(K, generator=g, device=DEV)).to(torch.bfloat16)
        st["beta"] = (0.05 * torch.randn(K, generator=g, device=DEV)).to(torch.bfloat16) if case["centred"] else None
        st["res"] = torch.randn(T, K, generator=g, device=DEV).to(dt) if case["residual"] else None
        if op == "norm_bwd":
            st["dy"] = torch.randn(T, K, generator=g, device=DEV).to(DT[case["dy"]])
        return st
    if op == "orthogonalize":
        L, M, N, dt = case["L"], case["M"], case["N"], DT[case["dtype"]]
        st["g"] = torch.empty(*([L] if L > 1 else []), M, N, dtype=dt, device=DEV)
        for m in st["g"].view(L, M, N):
            m.copy_(_gradient(M, N, g))
        return st
    T, I, dt, G = case["T"], case["I"], DT[case["dtype"]], case["G"]
    rows = T
    st["off"] = None
    if G:
        st["off"], rows = _blocks(T, G, g)
    st["gu"] = (1.5 * torch.randn(rows, 2 * I, generator=g, device=DEV)).to(dt)
    if op == "swiglu_bwd":
        st["dy"] = torch.randn(rows, I, generator=g, device=DEV).to(DT[case["dy"]])
        st["dgu"] = torch.zeros(rows, 2 * I, dtype=dt, device=DEV) if G else None
    elif op == "swiglu":
        st["y"] = torch.zeros(rows, I, dtype=DT[case["out"]], device=DEV) if G else None
    else:
        st["q"] = torch.zeros(rows, I, dtype=torch.uint8, device=DEV) if G else None
        st["sa"] = torch.zeros(rows, I // TILE, device=DEV) if G else None
    return st


# ---------------------------------------------------------------------------
# the passes
# ---------------------------------------------------------------------------
def run(state):
    c = state["case"]
    return {"norm": _norm, "norm_bwd": _norm_bwd, "swiglu": _swiglu, "swiglu_quant": _swiglu_quant,
            "swiglu_bwd": _swiglu_bwd, "orthogonalize": _orthogonalize}[c["op"]](state, c)


def _hat(x, centred):
    """Rows without their mean, where centred, over their standard deviation; and its inverse. 32 bits."""
    if centred:
        x = x - x.mean(dim=1, keepdim=True)
    r = 1.0 / torch.sqrt((x * x).mean(dim=1, keepdim=True) + EPS)
    return x * r, r


def _norm(st, c):
    x, gamma, beta, res = st["x"], st["gamma"], st["beta"], st["res"]
    if own:
        return _pkg().fp8q_norm(x, gamma, EPS, beta=beta, centred=c["centred"], residual=res, out_dtype=c["out"])
    h = None
    if res is not None:
        x = h = (x.float() + res.float()).to(x.dtype)
    y = _hat(x.float(), c["centred"])[0] * gamma.float()
    if beta is not None:
        y = y + beta.float()
    y = y.to(DT[c["out"]])
    return y if h is None else (y, h)


def _norm_bwd(st, c):
    x, gamma, dy, res = st["x"], st["gamma"], st["dy"], st["res"]
    if own:
        return _pkg().fp8q_norm_bwd(dy, x, gamma, EPS, centred=c["centred"], dres=res)
    xh, r = _hat(x.float(), c["centred"])
    d = dy.float()
    dg = d * gamma.float()
    dx = dg - xh * (dg * xh).mean(dim=1, keepdim=True)
    if c["centred"]:
        dx = dx - dg.mean(dim=1, keepdim=True)
    dx = r * dx
    if res is not None:
        dx = dx + res.float()
    return dx.to(x.dtype), (d * xh).sum(dim=0), d.sum(dim=0) if c["centred"] else None


def _gated(gu):
    """(gate, up, sigmoid of the gate), 32 bits."""
    gate, up = gu.float().chunk(2, dim=1)
    return gate, up, 1.0 / (1.0 + torch.exp(-gate))


def _inside(off, rows):
    """True for the rows before the last block's end."""
    return (torch.arange(rows, device=off.device) < off[-1]).unsqueeze(1)


def _swiglu(st, c):
    gu, off, y = st["gu"], st["off"], st["y"]
    if own:
        return _pkg().fp8q_swiglu(gu, out_dtype=c["out"], m_offsets=off, y=y)
    gate, up, s = _gated(gu)
    v = (gate * s * up).to(DT[c["out"]])
    if off is None:
        return v
    y.copy_(torch.where(_inside(off, gu.shape[0]), v, y))
    return y


def _swiglu_quant(st, c):
    gu, off, q, sa = st["gu"], st["off"], st["q"], st["sa"]
    if own:
        q, sa = _pkg().fp8q_swiglu_quant_act_1x128(gu, m_offsets=off, q=q, sa=sa)
        return q.view(torch.float8_e4m3fn), sa
    gate, up, s = _gated(gu)
    v = (gate * s * up).reshape(gu.shape[0], -1, TILE)
    # (the divisor is a tensor: a division by a number may be done as a product)
    scale = v.abs().amax(dim=2) / torch.full((), FP8_MAX, device=v.device)
    codes = v / torch.where(scale > 0, scale, torch.ones_like(scale)).unsqueeze(2)
    codes = codes.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).reshape(gu.shape[0], -1)
    if off is None:
        return codes, scale
    inside = _inside(off, gu.shape[0])
    q.copy_(torch.where(inside, codes.view(torch.uint8), q))
    sa.copy_(torch.where(inside, scale, sa))
    return q.view(torch.float8_e4m3fn), sa


def _swiglu_bwd(st, c):
    gu, off, dy, dgu = st["gu"], st["off"], st["dy"], st["dgu"]
    if own:
        return _pkg().fp8q_swiglu_bwd(dy, gu, m_offsets=off, dgu=dgu)
    gate, up, s = _gated(gu)
    d = dy.float()
    both = torch.cat([d * up * s * (1.0 + gate * (1.0 - s)), d * gate * s], dim=1).to(gu.dtype)
    if off is None:
        return both
    dgu.copy_(torch.where(_inside(off, gu.shape[0]), both, dgu))
    return dgu


def _orthogonalize(st, c):
    g = st["g"]
    if own:
        return _pkg().fp8q_orthogonalize(g, steps=STEPS, coeffs=COEFFS, out_dtype=c["out"])
    return _newton_schulz(g.float(), c).to(DT[c["out"]])


def _newton_schulz(x, c):
    a, b, d = COEFFS
    tall = c["M"] > c["N"]
    if tall:
        x = x.transpose(-1, -2).contiguous()
    norm = (x * x).sum(dim=(-2, -1), keepdim=True).sqrt()
    x = x / torch.where(norm > 0, norm, torch.ones_like(norm))
    for _ in range(STEPS):
        A = torch.matmul(x, x.transpose(-1, -2).contiguous())
        x = a * x + torch.matmul(b * A + d * torch.matmul(A, A), x)
    return x.transpose(-1, -2).contiguous() if tall else x


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, es = case["op"], 2 if case["dtype"] == "bf16" else 4
    other = case.get("out") or case.get("dy")
    eo = 2 if other == "bf16" else 4
    if op in ("norm", "norm_bwd"):
        n = case["T"] * case["K"]
        extra = n * es if case["residual"] else 0
        if op == "norm":  # x in, y out; with a residual that in and the sum out
            return {"bytes": n * (es + eo) + 2 * extra + case["K"] * 4, "flops": 6 * n}
        return {"bytes": n * (2 * es + eo) + extra + case["K"] * 10, "flops": 14 * n}
    if op == "orthogonalize":
        L, m, n = case["L"], min(case["M"], case["N"]), max(case["M"], case["N"])
        # x x^T and its square are symmetric: one half of each
        return {"bytes": L * m * n * (es + eo), "flops": L * STEPS * (3 * m * m * n + m ** 3)}
    rows = case["T"] + case["G"] * TILE / 2
    n = rows * case["I"]
    if op == "swiglu":
        return {"bytes": n * (2 * es + eo), "flops": 6 * n}
    if op == "swiglu_quant":
        return {"bytes": n * (2 * es + 1 + 4 / TILE), "flops": 9 * n}
    return {"bytes": n * (4 * es + eo), "flops": 12 * n}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "orthogonalize":
        return _exact_orthogonalize(st["g"], case)
    if op in ("norm", "norm_bwd"):
        x = st["x"].double()
        h = None
        if op == "norm" and st["res"] is not None:
            # the sum is kept in x's type, and that is what is normalized
            h = st["x"].double() + st["res"].double()
            x = h.to(st["x"].dtype).double()
        gamma = st["gamma"].double()
        with torch.enable_grad():
            leaf, w = x.clone().requires_grad_(op == "norm_bwd"), gamma.clone().requires_grad_(op == "norm_bwd")
            b = torch.zeros_like(gamma).requires_grad_(op == "norm_bwd")
            if case["centred"]:
                var, mu = torch.var_mean(leaf, dim=1, unbiased=False, keepdim=True)
                y = (leaf - mu) / torch.sqrt(var + EPS) * w + b
            else:
                y = leaf / torch.sqrt(leaf.square().mean(dim=1, keepdim=True) + EPS) * w
            if op == "norm_bwd":
                dx, dw = torch.autograd.grad(y, (leaf, w), st["dy"].double(), retain_graph=True)
                db = torch.autograd.grad(y, b, st["dy"].double())[0] if case["centred"] else None
                return dx if st["res"] is None else dx + st["res"].double(), dw, db
        if st["beta"] is not None:
            y = y + st["beta"].double()
        return y if h is None else (y, h)
    rows, I = st["gu"].shape[0], case["I"]
    last = rows if st["off"] is None else int(st["off"][-1])
    gate, up = st["gu"][:last, :I].double(), st["gu"][:last, I:].double()
    s = torch.sigmoid(gate)
    if op == "swiglu_bwd":
        out = torch.zeros(rows, 2 * I, dtype=torch.float64, device=DEV)
        d = st["dy"][:last].double()
        out[:last, I:] = torch.nn.functional.silu(gate) * d
        out[:last, :I] = (s + gate * s * torch.sigmoid(-gate)) * up * d
        return out
    out = torch.zeros(rows, I, dtype=torch.float64, device=DEV)
    out[:last] = gate * s * up
    if op == "swiglu":
        return out
    # a code is that of a 32-bit quotient: next to a border 64 bits say nothing of it
    return None, out.reshape(rows, -1, TILE).abs().amax(dim=2) / FP8_MAX


def _exact_orthogonalize(g, case):
    a, b, d = COEFFS
    out = torch.empty(g.shape, dtype=torch.float64, device=DEV)
    for m, o in zip(g.view(-1, case["M"], case["N"]), out.view(-1, case["M"], case["N"])):
        x = m.double()
        x = x / torch.linalg.norm(x)
        for _ in range(STEPS):
            if case["M"] <= case["N"]:
                gram = torch.mm(x, x.t())
                x = torch.addmm(x, torch.addmm(gram, gram, gram, beta=b, alpha=d), x, beta=a)
            else:  # the same from the other side: x (b g + d g^2), g = x^T x
                gram = torch.mm(x.t(), x)
                x = torch.addmm(x, x, torch.addmm(gram, gram, gram, beta=b, alpha=d), beta=a)
        o.copy_(x)
    return out
