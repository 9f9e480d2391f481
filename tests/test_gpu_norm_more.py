"""More of the normalization and its gradient: many short rows, several rounds of the gradient's row loop in every
shape of row, rows that are not ordinary in them. The bounds are those of test_gpu_norm_rows; u = 2^-24."""

import numpy as np
import pytest

from conftest import gpu_available
from test_gpu_norm_rows import U, check_bwd, check_norm, rows, weights

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.mark.parametrize("K", [64, 128])
@pytest.mark.parametrize("centred", [False, True])
def test_many_short_rows(K, centred):
    """Every head of every token: more than 2^22 rows. Rows of any part of them are the smaller call's, bit for bit;
    the weights' gradients are sums over M / 4096 rows in a thread, 8 in a workgroup, 512 partial rows in 32 runs."""
    import torch
    import fp8_fine_grained_online_amd as F
    M = (1 << 22) + 3
    gen = torch.Generator("cuda").manual_seed(K)
    x, dy = (torch.randn(M, K, device="cuda", generator=gen, dtype=torch.bfloat16) for _ in range(2))
    g, b = weights(K, 5200)
    b = b if centred else None
    y = F.fp8q_norm(x, g, 1e-6, beta=b, centred=centred)
    dx, dgamma, dbeta = F.fp8q_norm_bwd(dy, x, g, 1e-6, centred=centred)
    for part in (slice(0, 40), slice(M // 2, M // 2 + 40), slice(M - 41, M)):
        check_norm(x[part], g, 1e-6, b, centred, y[part], "bf16")
        assert torch.equal(y[part], F.fp8q_norm(x[part], g, 1e-6, beta=b, centred=centred))
        assert torch.equal(dx[part], F.fp8q_norm_bwd(dy[part], x[part], g, 1e-6, centred=centred)[0])
    sums = [torch.zeros(K, dtype=torch.float64, device="cuda") for _ in range(4)]
    for at in range(0, M, 1 << 20):
        h, d = x[at:at + (1 << 20)].double(), dy[at:at + (1 << 20)].double()
        if centred:
            h = h - h.mean(1, keepdim=True)
        h = h / torch.sqrt((h * h).mean(1, keepdim=True) + float(np.float32(1e-6)))
        for s, v in zip(sums, (d * h, (d * h).abs(), d, d.abs())):
            s += v.sum(0)
    n = M / 4096 + 8 + 16 + 32
    assert torch.all((dgamma - sums[0]).abs() <= (n + 80) * U * sums[1])
    if centred:
        assert torch.all((dbeta - sums[2]).abs() <= n * U * sums[3])


@pytest.mark.parametrize("K", [1, 5, 40, 1000, 1100, 2047, 3000, 5000, 9000, 16000])
@pytest.mark.parametrize("centred", [False, True])
def test_bwd_of_the_smallest_rows(K, centred):
    """eps 0 and rows whose 1 / std passes binary32: dx is finite where the formula is, beside ordinary rows."""
    import torch
    import fp8_fine_grained_online_amd as F
    x, dy = rows(7, K, 5210, "f32"), rows(7, K, 5211, "f32")
    g, _ = weights(K, 5212, "f32")
    ordinary = F.fp8q_norm_bwd(dy, x, g, 0.0, centred=centred)[0]
    z, d = x.clone(), dy.clone()
    for m in (2, 5, 6):
        z[m] = (x[m] * 2.0 ** 9).round() * 2.0 ** -139  # whole multiples of 2^-139: subnormal, and centred ones too
        d[m] *= 2.0 ** -16
    if K == 1:
        z[z == 0] = 2.0 ** -139
    dx, dgamma, dbeta = F.fp8q_norm_bwd(d, z, g, 0.0, centred=centred)
    keep = [0, 1, 3, 4]
    assert torch.equal(dx[keep].nan_to_num(7.0), ordinary[keep].nan_to_num(7.0))
    if K > 1 or not centred:  # (a single centred value has no deviation: 0 / 0)
        check_bwd(d, z, g, 0.0, centred, None, (dx, dgamma, dbeta))


# one past two full rounds of the gradient's 512 (beyond 8192 values 256) workgroups, in every shape of row
ROUNDS = [(8201, 64), (8195, 1000), (2051, 1025), (2049, 2047), (1027, 2500), (1031, 5000), (517, 9001), (521, 16383)]


@pytest.mark.parametrize("M,K", ROUNDS)
@pytest.mark.parametrize("centred", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bwd_in_several_rounds(M, K, centred, dtype):
    """Rows whose statistics leave binary32's range in both halves of a workgroup, in the first round, in later ones
    and as the last row, beside ordinary rows, whose gradients keep their bits."""
    import torch
    import fp8_fine_grained_online_amd as F
    x, dy, dres = rows(M, K, 5220, dtype), rows(M, K, 5221, dtype), rows(M, K, 5222, dtype)
    g, _ = weights(K, 5223)
    want = F.fp8q_norm_bwd(dy, x, g, 1e-6, centred=centred, dres=dres)
    check_bwd(dy, x, g, 1e-6, centred, dres, want)
    far = sorted({0, 3, 6, 7, M // 2, M // 2 + 1, M - 2, M - 1})
    z = x.clone()
    z[far] *= 2.0 ** 80
    z[far[2]] *= 2.0 ** -160
    got = F.fp8q_norm_bwd(dy, z, g, 1e-6, centred=centred, dres=dres)
    check_bwd(dy, z, g, 1e-6, centred, dres, got)
    keep = torch.ones(M, dtype=torch.bool)
    keep[far] = False
    assert torch.equal(got[0][keep], want[0][keep])
    z[far[1], K // 2], z[M // 2, 0], z[M - 1, K - 1] = float("nan"), float("inf"), float("nan")
    got = F.fp8q_norm_bwd(dy, z, g, 1e-6, centred=centred, dres=dres)
    assert torch.equal(got[0][keep], want[0][keep])
    assert torch.isnan(got[0][[far[1], M // 2, M - 1]]).any(1).all() and torch.isnan(got[1]).any()


@pytest.mark.parametrize("M,K", [(262147, 8200), (2200000, 1000)])
@pytest.mark.parametrize("centred", [False, True])
def test_more_values_than_32_bits_count(M, K, centred):
    """Rows at either side of 2^31 values, and the last, are the smaller call's, bit for bit."""
    import torch
    import fp8_fine_grained_online_amd as F
    x = torch.empty(M, K, device="cuda", dtype=torch.bfloat16).normal_(generator=torch.Generator("cuda").manual_seed(M))
    g, _ = weights(K, 5230)
    y, h = F.fp8q_norm(x, g, 1e-6, centred=centred, residual=x)
    dx, dgamma, _ = F.fp8q_norm_bwd(y, x, g, 1e-6, centred=centred, dres=x)
    middle = (1 << 31) // K
    for part in (slice(0, 3), slice(middle - 2, middle + 3), slice(M - 3, M)):
        y1, h1 = F.fp8q_norm(x[part], g, 1e-6, centred=centred, residual=x[part])
        assert torch.equal(y[part], y1) and torch.equal(h[part], h1)
        assert torch.equal(dx[part], F.fp8q_norm_bwd(y1, x[part], g, 1e-6, centred=centred, dres=x[part])[0])
    assert torch.isfinite(dgamma).all()
