"""Normalization of rows and its gradient on the GPU, against float64.

u = 2^-24 is the largest relative error of a binary32 rounding. A row's sum over K <= 16384 values
is a chain of at most 32 additions in a thread, 7 over its wavefront and 15 over the row's wavefronts (of 512
threads; of 1024 threads 16 in each): at most 46 roundings, so a sum of nonnegative terms is within 46 u. Hence

* r = 1 / sqrt(var + eps) is within (46 + 3) / 2 u + u < 26 u (1 / K and the product with it are two
  more roundings), centred rows' deviations adding their own rounding, 2 u of var;
* hat = d r is within 28 u |hat|; centred rows are shifted by what the mean is off by, itself a sum
  of deviations of either sign whose mean magnitude times r is at most 1: 50 u more;
* y = hat gamma + beta: two more roundings.

bfloat16 outputs are rounded once more: 2^-8 of their value."""

import numpy as np
import pytest

from conftest import gpu_available
from fp8_fine_grained_online_amd import synthetic as S
from oracle import step

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


def weights(K, seed, dtype="bf16"):
    rng = S.rng_for(seed, K)
    return tensor(1 + 0.3 * rng.standard_normal(K), dtype), tensor(rng.standard_normal(K), dtype)


def rows(M, K, seed, dtype="bf16", wide=0):
    """M x K activations; with `wide`, the first K of K + wide columns."""
    rng = S.rng_for(seed, M + K)
    x = rng.standard_normal((M, K + wide))
    x *= np.where(rng.random(x.shape) < 0.001, 100.0, 1.0)
    return tensor(x, dtype)[:, :K]


def hat_error(hat, centred):
    return 28 * U * np.abs(hat) + (50 * U if centred else 0.0)


def check_norm(x, g, eps, b, centred, got, out):
    want = step.norm(host(x), host(g), eps, None if b is None else host(b), centred)
    hat, _ = step.stats(host(x), eps, centred)
    tol = (hat_error(hat, centred) + U * np.abs(hat)) * np.abs(host(g)) + U * np.abs(want)
    tol += half_step(out) * (np.abs(want) + tol) + 2.0 ** -126
    err = np.abs(host(got) - want)
    assert np.all(err <= tol), float(np.max(err / tol))


# every shape of row that the kernels have (64 to 1024 threads, 1 to 4 chunks each), its limits
# and the sizes around them, odd sizes and the smallest
SIZES = [(1, 1), (3, 7), (5, 8), (2, 9), (7, 512), (3, 513), (6, 1024), (1, 1025), (9, 2048), (4, 2049), (2, 3585), (5, 4095),
         (2, 4097), (1, 7168), (3, 8192), (2, 8193), (3, 12288), (2, 12289), (3, 16383), (2, 16384)]


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("centred", [False, True])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_norm(M, K, centred, dtype, out):
    import torch
    import fp8_fine_grained_online_amd as F
    x = rows(M, K, 3100, dtype)
    g, b = weights(K, 3101, "bf16" if K % 2 else "f32")
    b = b if centred and K % 3 else None
    y = torch.full((M + 1, K), 7.0, dtype=torch_dtype(out), device="cuda")
    got = F.fp8q_norm(x, g, 1e-6, beta=b, centred=centred, out_dtype=out, y=y[:M])
    check_norm(x, g, 1e-6, b, centred, got, out)
    assert torch.all(y[M] == 7.0)  # nothing behind the last row


@pytest.mark.parametrize("M,K,wide", [(5, 512, 64), (3, 513, 1), (300, 1000, 24), (2, 7168, 0), (70, 2050, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("centred", [False, True])
def test_residual_and_rows_apart(M, K, wide, dtype, centred):
    """The sum is torch's, bit for bit, and it is what is normalized; columns of a wider tensor."""
    import torch
    import fp8_fine_grained_online_amd as F
    x, res = rows(M, K, 3110, dtype, wide), rows(M, K, 3111, dtype, 2 * wide)
    assert wide == 0 or not x.is_contiguous()
    g, b = weights(K, 3112)
    y, h = F.fp8q_norm(x, g, 1e-5, beta=b if centred else None, centred=centred, residual=res, out_dtype="f32")
    assert torch.equal(h, (x.float() + res.float()).to(x.dtype))
    check_norm(h, g, 1e-5, b if centred else None, centred, y, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [40, 1000, 5000])
@pytest.mark.parametrize("centred", [False, True])
def test_rows_outside_the_ordinary_range(dtype, K, centred):
    """Zero and constant rows, squares that overflow or underflow binary32, a mean far above the spread."""
    import fp8_fine_grained_online_amd as F
    x = host(rows(8, K, 3120, "f32"))
    x[0] = 0
    x[1] = 3.0
    x[2] *= 2.0 ** 100
    x[3] *= 2.0 ** -110
    x[4] = np.where(np.arange(K) % 2 == 0, 2.0 ** 126, -(2.0 ** 126))
    x[5] *= 2.0 ** 60
    x[6] += 300.0
    x = tensor(x, dtype)
    g, b = weights(K, 3121)
    for eps in (1e-6, 0.0):
        first = 2 if eps == 0 else 0  # a row without spread divides by zero
        y = F.fp8q_norm(x[first:], g, eps, centred=centred, out_dtype="f32")
        check_norm(x[first:], g, eps, None, centred, y, "f32")


@pytest.mark.parametrize("K", [300, 700, 1100, 2047, 3000, 4000, 10000, 16000])
@pytest.mark.parametrize("centred", [False, True])
def test_a_row_outside_the_range_leaves_its_neighbours_alone(K, centred):
    """Also as the last row of an odd number."""
    import torch
    import fp8_fine_grained_online_amd as F
    x = rows(5, K, 5160, "f32")
    g, _ = weights(K, 5161, "f32")
    want = F.fp8q_norm(x, g, 1e-6, centred=centred, out_dtype="f32")
    for far in (1, 4):
        z = x.clone()
        z[far] *= 1e25
        got = F.fp8q_norm(z, g, 1e-6, centred=centred, out_dtype="f32")
        check_norm(z, g, 1e-6, None, centred, got, "f32")
        keep = [i for i in range(5) if i != far]
        assert torch.equal(got[keep], want[keep])


def test_rows_that_are_not_finite():
    import torch
    import fp8_fine_grained_online_amd as F
    for K in (33, 3000):
        for centred in (False, True):
            x = rows(9, K, 3130)
            g, _ = weights(K, 3131)
            want = F.fp8q_norm(x, g, 1e-6, centred=centred)
            dx, _, _ = F.fp8q_norm_bwd(x, x, g, 1e-6, centred=centred)
            bad = x.clone()
            bad[2, K // 2], bad[5, 0], bad[7, K - 1] = float("nan"), float("inf"), -float("inf")
            y = F.fp8q_norm(bad, g, 1e-6, centred=centred)
            d, dg, _ = F.fp8q_norm_bwd(x, bad, g, 1e-6, centred=centred)
            for m in range(9):
                if m in (2, 5, 7):
                    assert torch.isnan(y[m, K // 2 if m == 2 else 0 if m == 5 else K - 1]) and torch.isnan(d[m]).any()
                else:
                    assert torch.equal(y[m], want[m]) and torch.equal(d[m], dx[m])
            assert torch.isnan(dg).any()


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------
def check_bwd(dy, x, g, eps, centred, dres, got):
    import torch
    dx, dgamma, dbeta = got
    M, K = x.shape
    y64, x64, g64 = host(dy), host(x), host(g)
    hat, r = step.stats(x64, eps, centred)
    dg = y64 * g64
    want = step.norm_bwd(y64, x64, g64, eps, centred, None if dres is None else host(dres))
    e_hat = hat_error(hat, centred)
    c, one = (dg * hat).mean(1, keepdims=True), dg.mean(1, keepdims=True) if centred else 0.0
    # the means: 46 roundings of the sum and three more, and the error of what is summed
    e_c = 50 * U * np.abs(dg * hat).mean(1, keepdims=True) + (np.abs(dg) * e_hat).mean(1, keepdims=True)
    e_one = 50 * U * np.abs(dg).mean(1, keepdims=True) if centred else 0.0
    tol = r * (3 * U * (np.abs(dg) + np.abs(one) + np.abs(hat * c)) + e_hat * np.abs(c) + (np.abs(hat) + e_hat) * e_c + e_one)
    tol += 28 * U * np.abs(r * (dg - one - hat * c)) + 2 * U * np.abs(want[0])
    tol += half_step("bf16" if dx.dtype == torch.bfloat16 else "f32") * (np.abs(want[0]) + tol) + 2.0 ** -126
    err = np.abs(host(dx) - want[0])
    assert dx.dtype == x.dtype and np.all(err <= tol), float(np.max(err / tol))
    # over rows: at most M additions in whatever order (far fewer in a chain), with the terms' own errors
    mag = np.abs(y64 * hat).sum(0)
    n = min(M, M / 256 + 80)  # rows of one thread, the workgroup's rows, 256 partial rows in 16 runs
    err = np.abs(host(dgamma) - want[1])
    tol = (n + 1) * U * mag + (np.abs(y64) * e_hat).sum(0) + 2.0 ** -126
    assert np.all(err <= tol), float(np.max(err / tol))
    assert (dbeta is None) == (not centred)
    if centred:
        err = np.abs(host(dbeta) - want[2])
        tol = n * U * np.abs(y64).sum(0) + 2.0 ** -126
        assert np.all(err <= tol), float(np.max(err / tol))


@pytest.mark.parametrize("M,K", SIZES + [(600, 64), (2100, 200), (777, 3001), (523, 9000)])
@pytest.mark.parametrize("centred", [False, True])
@pytest.mark.parametrize("dtype,ddtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_norm_bwd(M, K, centred, dtype, ddtype):
    import torch
    import fp8_fine_grained_online_amd as F
    x, dy = rows(M, K, 3140, dtype), rows(M, K, 3141, ddtype)
    g, _ = weights(K, 3142, "f32" if K % 2 else "bf16")
    dres = rows(M, K, 3143, dtype) if M % 2 else None
    dx = torch.full((M + 1, K), 7.0, dtype=torch_dtype(dtype), device="cuda")
    dgamma = torch.full((K,), float("nan"), device="cuda")
    got = F.fp8q_norm_bwd(dy, x, g, 1e-6, centred=centred, dres=dres, dx=dx[:M], dgamma=dgamma)
    check_bwd(dy, x, g, 1e-6, centred, dres, got)
    assert torch.all(dx[M] == 7.0)
    again = F.fp8q_norm_bwd(dy, x, g, 1e-6, centred=centred, dres=dres)
    for a, b in zip(got, again):  # no order that changes
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("K,wide", [(512, 64), (513, 1), (5000, 8)])
@pytest.mark.parametrize("centred", [False, True])
def test_bwd_rows_apart(K, wide, centred):
    import fp8_fine_grained_online_amd as F
    x, dy, dres = rows(37, K, 3150, "bf16", wide), rows(37, K, 3151, "f32", 3 * wide), rows(37, K, 3152, "bf16", 2 * wide)
    g, _ = weights(K, 3153)
    check_bwd(dy, x, g, 1e-5, centred, dres, F.fp8q_norm_bwd(dy, x, g, 1e-5, centred=centred, dres=dres))


@pytest.mark.parametrize("K", [40, 1000, 5000, 9000])
@pytest.mark.parametrize("centred", [False, True])
def test_bwd_rows_outside_the_ordinary_range(K, centred):
    """Rows whose statistics leave binary32's range, beside ordinary ones of the same workgroup."""
    import fp8_fine_grained_online_amd as F
    x = host(rows(40, K, 3160, "f32"))
    x[0] = 0
    x[1] = 3.0
    x[2] *= 2.0 ** 60
    x[9] *= 2.0 ** 80
    x[6] += 300.0
    x, dy = tensor(x), rows(40, K, 3161, "f32")
    g, _ = weights(K, 3162)
    check_bwd(dy, x, g, 1e-6, centred, None, F.fp8q_norm_bwd(dy, x, g, 1e-6, centred=centred))


def test_bwd_of_no_rows():
    import torch
    import fp8_fine_grained_online_amd as F
    x = torch.empty(0, 100, device="cuda")
    dx, dg, db = F.fp8q_norm_bwd(x, x, torch.ones(100, device="cuda"), 1e-6, centred=True)
    assert dx.shape == (0, 100) and not dg.any() and not db.any()
    assert F.fp8q_norm(x, torch.ones(100, device="cuda"), 1e-6).shape == (0, 100)
    e = torch.empty(4, 0, device="cuda")
    assert F.fp8q_norm(e, torch.ones(0, device="cuda"), 1e-6).shape == (4, 0)


@pytest.mark.parametrize("centred", [False, True])
def test_gradient_is_the_difference_of_the_forward_call(centred):
    """sum(y dy) along a direction: the forward call's own difference against the gradient call's product.
    y's error is at most 80 u of its size (above), so the difference over 2 t of two sums of K such
    terms is off by at most 80 u sum|y dy| / t, and by the third derivative's t^2 term; t = 2^-6 makes
    both small against the sum of magnitudes."""
    import fp8_fine_grained_online_amd as F
    M, K, t = 6, 300, 2.0 ** -6
    rng = S.rng_for(3170, int(centred))
    x, v, dy = (np.round(rng.standard_normal((M, K)) * 256) / 256 for _ in range(3))  # x + t v is exact
    g, b = weights(K, 3171, "f32")
    b = b if centred else None
    up, down = (F.fp8q_norm(tensor(x + s * t * v), g, 1e-5, beta=b, centred=centred, out_dtype="f32") for s in (1, -1))
    slope = ((host(up) - host(down)) * dy).sum(1) / (2 * t)
    dx, _, _ = F.fp8q_norm_bwd(tensor(dy), tensor(x), g, 1e-5, centred=centred)
    got = (host(dx) * v).sum(1)
    exact = ((step.norm(x + t * v, host(g), 1e-5, None, centred) - step.norm(x - t * v, host(g), 1e-5, None, centred))
             * dy).sum(1) / (2 * t)
    third = np.abs(exact - (step.norm_bwd(dy, x, host(g), 1e-5, centred)[0] * v).sum(1))
    noise = 80 * U * (np.abs(host(up)) * np.abs(dy)).sum(1) / t + 100 * U * (np.abs(host(dx)) * np.abs(v)).sum(1)
    assert np.all(np.abs(slope - got) <= third + noise)


def test_the_fused_casts_gradient_and_a_stream():
    """The gradient takes the fused forward's inputs; another stream and the caller's buffers give the same bits."""
    import torch
    import fp8_fine_grained_online_amd as F
    M, K = 130, 1024
    x, dy = rows(M, K, 3180), rows(M, K, 3181)
    g, _ = weights(K, 3182)
    q, sa = F.fp8q_norm_quant_act_1x128(x, g, 1e-6)
    y = F.fp8q_norm(x, g, 1e-6, out_dtype="f32")
    deq = q.view(torch.float8_e4m3fn).float().reshape(M, -1, 128) * sa.unsqueeze(2)
    # half a step of a code: 2^-4 of it, or of the smallest normal code's scale
    assert torch.all((deq.reshape(M, K) - y).abs() <= 2.0 ** -4 * y.abs() + 2.0 ** -10 * sa.repeat_interleave(128, 1) + 1e-5)
    want = F.fp8q_norm_bwd(dy, x, g, 1e-6)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ws = torch.empty(F.lib().fp8q_norm_bwd_workspace_bytes(M, K, 0), dtype=torch.uint8, device="cuda")
    got = F.fp8q_norm_bwd(dy, x, g, 1e-6, workspace=ws, stream=s)
    y2 = F.fp8q_norm(x, g, 1e-6, out_dtype="f32", stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[2] is None and torch.equal(y, y2)


def test_refusals():
    import torch
    import fp8_fine_grained_online_amd as F
    x, g = rows(4, 64, 3190), weights(64, 3191)[0]
    for call in (lambda: F.fp8q_norm(x.t(), g, 1e-6), lambda: F.fp8q_norm(x[:1].expand(4, 64), g, 1e-6),
                 lambda: F.fp8q_norm(x, g[:32], 1e-6), lambda: F.fp8q_norm(x, g, 1e-6, residual=x[:2]),
                 lambda: F.fp8q_norm(x, g, 1e-6, h=x), lambda: F.fp8q_norm(x, g.cpu(), 1e-6),
                 lambda: F.fp8q_norm_bwd(x[:3], x, g, 1e-6), lambda: F.fp8q_norm_bwd(x, x, g, 1e-6, dbeta=g.float())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: F.fp8q_norm(x.half(), g, 1e-6), lambda: F.fp8q_norm(x, g, 1e-6, beta=g.float(), centred=True),
                 lambda: F.fp8q_norm(x, g, 1e-6, residual=x.float())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: F.fp8q_norm(x, g, -1.0), lambda: F.fp8q_norm(x, g, 1e-6, beta=g),
                 lambda: F.fp8q_norm_bwd(x, x, g, 1e-6, workspace=torch.empty(4, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(F.Fp8qError):
            call()
    big = torch.empty(1, 16392, device="cuda")
    with pytest.raises(F.Fp8qError):
        F.fp8q_norm(big, torch.ones(16392, device="cuda"), 1e-6)
