"""MoE router and its gradient, in float64, token by token.

  p = softmax(l) or 1 / (1 + exp(-l));  z = p + bias; masked experts (logit -inf
  or NaN, or a bias that makes z so) cannot be chosen;
  groups: the score of a group is the sum of its (up to) two largest z; the best
  topk_groups stay;  ids = the topk largest z, ties to the lowest index;
  w_j = scale p_j, or scale p_j / sum_i p_i, a ratio that holds where the p underflow;
  choices that cannot be filled are -1 with weight 0.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""

import numpy as np


def scores(logits, score):
    x = np.asarray(logits, np.float64)
    live = x > -np.inf  # False for NaN
    with np.errstate(over="ignore", under="ignore"):
        if score == "sigmoid":
            v = np.where(live, x, 0.0)
            # (1 + e^v is 1 in float64 below -700, and e^-v would overflow below -709)
            return np.where(live, np.where(v < -700.0, np.exp(np.minimum(v, 0.0)), 1.0 / (1.0 + np.exp(-v))), 0.0)
        p = np.zeros_like(x)
        for t in range(x.shape[0]):
            at = live[t]
            if at.any():
                e = np.exp(x[t, at] - x[t, at].max())
                p[t, at] = e / e.sum()
        return p


def ratios(x, score):
    """p_j / sum_i p_i over the logits x, with the factor e^top that all p share taken out: it holds however small
    the probabilities are. Masked logits count as 0; all masked: all 0."""
    x = np.asarray(x, np.float64)
    live = x > -np.inf
    if not live.any():
        return np.zeros_like(x)
    v = np.where(live, x, 0.0)
    top = v[live].max()
    with np.errstate(under="ignore"):
        if score == "sigmoid":
            n = np.exp(np.minimum(v, 0.0) - min(top, 0.0)) / (1.0 + np.exp(-np.abs(v)))
        else:
            n = np.exp(v - top)
    n = np.where(live, n, 0.0)
    return n / n.sum()


def route(logits, topk, bias=None, score="softmax", renormalize=True, scale=1.0, n_groups=1, topk_groups=1):
    x = np.asarray(logits, np.float64)
    T, G = x.shape
    p = scores(x, score)
    z = p + (0.0 if bias is None else np.asarray(bias, np.float64))
    open_ = (x > -np.inf) & (z > -np.inf)
    ids = np.full((T, topk), -1, np.int32)
    w = np.zeros((T, topk))
    gs = G // n_groups
    for t in range(T):
        can = open_[t].copy()
        if n_groups > 1:
            best = []
            for g in range(n_groups):
                top = sorted((z[t, e] for e in range(g * gs, (g + 1) * gs) if can[e]), reverse=True)[:2]
                if top:
                    best.append((-sum(top), g))
            kept = {g for _, g in sorted(best)[:topk_groups]}
            can &= np.array([e // gs in kept for e in range(G)])
        order = sorted((e for e in range(G) if can[e]), key=lambda e: (-z[t, e], e))[:topk]
        ids[t, :len(order)] = order
        w[t, :len(order)] = scale * (ratios(x[t, order], score) if renormalize else p[t, order])
    return ids, w


def weights_of(logits, ids, score, renormalize, scale):
    """The weights as a function of the logits, the ids held fixed."""
    p = scores(logits, score)
    ids = np.asarray(ids)
    T, G = p.shape
    on = (ids >= 0) & (ids < G)
    if renormalize:
        chosen = np.take_along_axis(np.asarray(logits, np.float64), np.where(on, ids, 0), 1)
        return scale * np.stack([ratios(v, score) for v in np.where(on, chosen, -np.inf)])
    return scale * np.where(on, np.take_along_axis(p, np.where(on, ids, 0), 1), 0.0)


def route_bwd(logits, ids, dweights, score="softmax", renormalize=True, scale=1.0):
    """dlogits[t, e] = sum_j dweights[t, j] d weights[t, j] / d logits[t, e], by the product rule."""
    logits = np.asarray(logits, np.float64)
    p = scores(logits, score)
    ids, g = np.asarray(ids), np.asarray(dweights, np.float64) * scale
    T, G = p.shape
    d = np.zeros((T, G))
    for t in range(T):
        on = [(int(e), g[t, j]) for j, e in enumerate(ids[t]) if 0 <= e < G]
        if renormalize:  # dw_j / dl_e = q_j (delta_je - q_e), times 1 - p_e for sigmoids
            q = ratios([logits[t, e] for e, _ in on], score)
            mean = sum(gj * qj for (_, gj), qj in zip(on, q))
            for (e, gj), qj in zip(on, q):
                d[t, e] += qj * (gj - mean) * (1 - p[t, e] if score == "sigmoid" else 1.0)
            continue
        dp = np.zeros(G)
        for e, gj in on:
            dp[e] += gj
        if score == "sigmoid":
            d[t] = dp * p[t] * (1 - p[t])
        else:
            d[t] = p[t] * (dp - (dp * p[t]).sum())
    return d
