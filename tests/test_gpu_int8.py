"""GPU row quantization and 8-bit integer products against the oracle, bit for bit
(every step is a defined binary32 rounding; bfloat16 outputs are those, rounded once)."""

import numpy as np
import pytest

from conftest import gpu_available
from fp8_fine_grained_online_amd import synthetic as S
from oracle import int8

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def codes(shape, seed):
    """All 256 values, -128 among them."""
    return S.rng_for(seed, 0).integers(-128, 128, shape).astype(np.int8)


def scales(shape, seed):
    return (0.001 + S.rng_for(seed, 1).random(shape)).astype(np.float32)


def dev(a):
    import torch
    return torch.from_numpy(a).cuda()


def rounded(f32, out):
    import torch
    t = torch.from_numpy(f32)
    return t if out == "f32" else t.to(torch.bfloat16)


def same(got, want):
    import torch
    got = got.cpu()
    assert got.dtype == want.dtype and got.shape == want.shape
    bad = (got.double() != want.double()) & ~(torch.isnan(got) & torch.isnan(want))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("M,K", [(1, 16), (1, 7168), (3, 48), (33, 2064), (5, 32768), (2, 65552), (4100, 112),
                                 (4097, 8208), (4096, 16), (7, 131072)])
def test_quant_rows(M, K):
    import torch
    import fp8_fine_grained_online_amd as F
    rng = S.rng_for(2700 + M, K)
    x = torch.from_numpy(rng.standard_normal((M, K), dtype=np.float32)).to(torch.bfloat16)
    x[:, 3] *= 100
    x[M // 2] = 0                                  # a row of nothing
    x[0] *= 2.0 ** -120                            # a subnormal scale
    if M > 2:
        x[1] = torch.where(torch.arange(K) % 2 == 0, 1.0, 0.5)  # 63.5: ties
        x[2] *= 2.0 ** 118
    q = torch.full((M, K), 77, dtype=torch.int8, device="cuda")
    s = torch.full((M,), float("nan"), device="cuda")
    F.fp8q_quant_int8_rows(x.cuda(), q=q, s=s)
    want_q, want_s = int8.quant_rows(x.float().numpy())
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q.cpu().numpy(), want_q)


def test_quant_every_value_under_every_maximum():
    """One binade of maxima (128 significands) by all smaller bfloat16 values down to codes of zero."""
    import torch
    import fp8_fine_grained_online_amd as F
    for field in (127, 1, 0, 254):
        rows = S.exhaustive_tiles(field, depth=10)
        x = torch.from_numpy(rows.view(np.int16)).view(torch.bfloat16)
        q, s = F.fp8q_quant_int8_rows(x.cuda())
        want_q, want_s = int8.quant_rows(x.float().numpy())
        assert np.array_equal(s.cpu().numpy(), want_s)
        assert np.array_equal(q.cpu().numpy(), want_q)


def test_quant_codes_beyond_the_cache():
    """Over 256 MiB of codes (stored another way), against the same formula in torch: the division of two
    tensors and the rounding are IEEE there too."""
    import torch
    import fp8_fine_grained_online_amd as F
    M, K = 40000, 7168
    x = torch.randn(M, K, device="cuda", generator=torch.Generator("cuda").manual_seed(5)).to(torch.bfloat16)
    q, s = F.fp8q_quant_int8_rows(x)
    for m in range(0, M, 8000):
        xf = x[m:m + 8000].float()
        want_s = xf.abs().amax(1) / torch.full((), 127.0, device="cuda")
        assert torch.equal(s[m:m + 8000], want_s)
        assert torch.equal(q[m:m + 8000], torch.round(xf / want_s.unsqueeze(1)).to(torch.int8))


@pytest.mark.parametrize("K", [16, 1040, 4112, 40000])
def test_quant_rows_that_are_not_finite(K):
    """An infinite or NaN row has that as its scale, a product's row from it is not finite, and other rows are exact."""
    import torch
    import fp8_fine_grained_online_amd as F
    M = 21
    x = torch.from_numpy(S.rng_for(2715, K).standard_normal((M, K), dtype=np.float32)).to(torch.bfloat16)
    bad = {2: float("inf"), 5: -float("inf"), 6: float("nan"), 20: float("inf")}
    for row, v in bad.items():
        x[row, (row * 7) % K] = v
    x[20, 3] = float("nan")
    q, s = F.fp8q_quant_int8_rows(x.cuda())
    good = [m for m in range(M) if m not in bad]
    want_q, want_s = int8.quant_rows(x[good].float().numpy())
    assert np.array_equal(s.cpu().numpy()[good], want_s) and np.array_equal(q.cpu().numpy()[good], want_q)
    assert s[[2, 5]].eq(float("inf")).all() and s[[6, 20]].isnan().all()
    b, sb = codes((70, K), 2716), scales(70, 2717)
    c = F.int8_gemm_scaled(q, s, dev(b), dev(sb), "f32").cpu()
    assert not torch.isfinite(c[list(bad)]).any()
    same(c[good], rounded(int8.gemm(want_q, want_s, b, sb), "f32"))


def test_quant_weights_of_experts():
    import torch
    import fp8_fine_grained_online_amd as F
    x = torch.from_numpy(S.rng_for(2710, 0).standard_normal((3, 40, 64), dtype=np.float32)).to(torch.bfloat16).cuda()
    q, s = F.fp8q_quant_int8_rows(x)
    assert q.shape == (3, 40, 64) and s.shape == (3, 40)
    q2, s2 = F.fp8q_quant_int8_rows(x.reshape(120, 64))
    assert torch.equal(q.reshape(120, 64), q2) and torch.equal(s.reshape(-1), s2)


DENSE = [(1, 1, 16), (1, 7168, 1024), (2, 33, 48), (16, 100, 4112), (17, 129, 128), (64, 65, 256), (100, 2050, 272),
         (129, 257, 144), (333, 514, 2064), (1000, 31, 640), (1, 64, 131056), (520, 520, 144), (260, 4100, 96),
         (1500, 3000, 400), (2049, 4097, 128), (4100, 2056, 272), (300, 300, 208), (500, 500, 528),
         (1000, 1900, 272), (1500, 2000, 400), (1000, 1901, 2064),
         (4090, 4080, 272), (4000, 4081, 400), (333, 514, 2192), (200, 1030, 2320), (100, 4097, 4112),
         (500, 1000, 2176)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense(M, N, K, out):
    import torch
    import fp8_fine_grained_online_amd as F
    a, b = codes((M, K), 2720 + M), codes((N, K), 2721 + N)
    sa, sb = scales(M, 2722), scales(N, 2723)
    sa[M // 2] = 0  # a zero row's scale
    c = torch.full((M, N), float("nan"), dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    F.int8_gemm_scaled(dev(a), dev(sa), dev(b), dev(sb), out, c=c)
    same(c, rounded(int8.gemm(a, sa, b, sb), out))


@pytest.mark.parametrize("M,N,K", [(129, 1025, 2320), (1025, 129, 4112), (64, 4097, 6160), (65, 4033, 2576),
                                   (129, 1025, 8208), (1025, 129, 8464), (64, 4097, 16400), (65, 4033, 8272)])
def test_last_rows_alone_in_their_tiles(M, N, K):
    """One row of a, of b or of both in a 64 x 64 tile, and a K that two groups of waves do not halve: the second
    group's last step lies past K, where its copies must read zeros."""
    import torch
    import fp8_fine_grained_online_amd as F
    a, b = codes((M, K), 2760 + M), codes((N, K), 2761 + N)
    sa, sb = scales(M, 2762), scales(N, 2763)
    c = torch.full((M, N), float("nan"), device="cuda")
    F.int8_gemm_scaled(dev(a), dev(sa), dev(b), dev(sb), "f32", c=c)
    same(c, rounded(int8.gemm(a, sa, b, sb), "f32"))


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(333, 514, 1920), (333, 514, 2048), (200, 1030, 2176), (500, 1000, 2432),
                                   (200, 1030, 8176), (200, 1030, 8208), (333, 514, 8320), (100, 4097, 9232)])
def test_one_and_two_groups_of_waves(M, N, K, out):
    """64 x 64 tiles on both sides of the limits of K, with whole 128-byte steps and without, even and odd."""
    import torch
    import fp8_fine_grained_online_amd as F
    a, b = codes((M, K), 2770 + M), codes((N, K), 2771 + N)
    sa, sb = scales(M, 2772), scales(N, 2773)
    c = torch.full((M, N), float("nan"), dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    F.int8_gemm_scaled(dev(a), dev(sa), dev(b), dev(sb), out, c=c)
    same(c, rounded(int8.gemm(a, sa, b, sb), out))


def test_largest_sums():
    """-128 by -128 over the largest K: 2^14 * 131056 < 2^31."""
    import torch
    import fp8_fine_grained_online_amd as F
    K = 131056
    for M, N in ((3, 5), (2100, 4100)):
        a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
        b = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
        c = F.int8_gemm_scaled(a, torch.ones(M, device="cuda"), b, torch.ones(N, device="cuda"), "f32")
        assert (c == float(np.float32(16384 * K))).all()


def test_operands_past_32_bits():
    """Rows whose byte offset does not fit 32 bits: a 40000 x 131056, b 40 x 1024 x 131056 (5.2 and 5.4 GB)."""
    import torch
    import fp8_fine_grained_online_amd as F
    K, N = 131056, 17
    ones = torch.ones(40960, device="cuda")
    k = torch.arange(K, device="cuda")
    row, col = (k % 251 - 125).to(torch.int8), (k % 127 - 63).to(torch.int8)
    sums = float(np.float32(int((row.long() * col.long()).sum())))
    a = torch.zeros((40000, K), dtype=torch.int8, device="cuda")
    a[-1] = row
    b = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    b[-1] = col
    c = F.int8_gemm_scaled(a, ones[:40000], b, ones[:N], "f32")
    assert c[-1, -1] == sums and torch.count_nonzero(c) == 1
    del a
    b = torch.zeros((40, 1024, K), dtype=torch.int8, device="cuda")
    b[-1, -1] = col
    a = torch.zeros((128, K), dtype=torch.int8, device="cuda")
    a[5] = row
    off = torch.zeros(41, dtype=torch.int32, device="cuda")
    off[40] = 128
    c = F.int8_gemm_grouped(a, ones[:128], b, ones.view(40, 1024), off, "f32")
    assert c[5, -1] == sums and torch.count_nonzero(c) == 1


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_outputs_past_32_bits(out):
    import torch
    import fp8_fine_grained_online_amd as F
    M, N, K = 65537, 40001, 16
    sa, sb = scales(M, 2750), scales(N, 2751)
    a, b = codes((M, K), 2752), codes((N, K), 2753)
    c = F.int8_gemm_scaled(dev(a), dev(sa), dev(b), dev(sb), out)
    for rows in (slice(0, 3), slice(M - 3, M)):
        same(c[rows], rounded(int8.gemm(a[rows], sa[rows], b, sb), out))


def test_empty_sizes():
    import torch
    import fp8_fine_grained_online_amd as F

    def z(*shape, dtype=torch.int8):
        return torch.zeros(shape, dtype=dtype, device="cuda")
    f = torch.float32
    assert F.int8_gemm_scaled(z(0, 64), z(0, dtype=f), z(5, 64), z(5, dtype=f)).shape == (0, 5)
    assert F.int8_gemm_scaled(z(4, 64), z(4, dtype=f), z(0, 64), z(0, dtype=f)).shape == (4, 0)
    for M, N in ((4, 5), (3000, 3000)):
        c = torch.full((M, N), float("nan"), device="cuda")
        F.int8_gemm_scaled(z(M, 0), torch.ones(M, device="cuda"), z(N, 0), torch.ones(N, device="cuda"), "f32", c=c)
        assert not c.any()
    q, s = F.fp8q_quant_int8_rows(z(4, 0, dtype=torch.bfloat16))
    assert q.shape == (4, 0) and not s.any()


GROUPED = [([128], 64, 64), ([0, 128, 0], 100, 48), ([128, 384, 256, 0], 257, 272), ([256] * 5, 514, 1040),
           ([128] * 40, 128, 144), ([1024, 128, 2048], 300, 128), ([0, 0], 64, 64), ([128] * 70 + [256], 96, 64),
           ([128] * 40, 514, 144), ([1024, 128, 2048, 384], 1030, 272), ([512, 0, 256] * 30, 300, 1040)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("rows,N,K", GROUPED, ids=[f"{len(r)}x{sum(r)}_{n}_{k}" for r, n, k in GROUPED])
def test_grouped(rows, N, K, out):
    import torch
    import fp8_fine_grained_online_amd as F
    G, M = len(rows), sum(rows) + 256  # rows behind the last block
    off = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    a, b = codes((M, K), 2730 + G), codes((G, N, K), 2731 + G)
    sa, sb = scales(M, 2732), scales((G, N), 2733)
    c = torch.full((M, N), float("nan"), dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    F.int8_gemm_grouped(dev(a), dev(sa), dev(b), dev(sb), dev(off), out, c=c)
    same(c, rounded(int8.gemm_grouped(a, sa, b, sb, off), out))  # NaN where nothing is written


def test_grouped_with_fewer_rows_than_given():
    """M_total below a's rows: offsets are held to it, and c has M_total rows."""
    import torch
    import fp8_fine_grained_online_amd as F
    a, b = codes((640, 96), 2740), codes((3, 70, 96), 2741)
    sa, sb = scales(700, 2742), scales((3, 70), 2743)
    off = np.array([0, 128, 256, 384], np.int32)
    c = F.int8_gemm_grouped(dev(a), dev(sa), dev(b), dev(sb), dev(off), "f32", M_total=384)
    assert c.shape == (384, 70)
    same(c, rounded(int8.gemm_grouped(a[:384], sa[:384], b, sb, off), "f32"))
    with pytest.raises(ValueError):
        F.int8_gemm_grouped(dev(a), dev(sa), dev(b), dev(sb), dev(off), "f32", M_total=768)


def test_grouped_without_k():
    import torch
    import fp8_fine_grained_online_amd as F
    off = torch.tensor([0, 128, 256], dtype=torch.int32, device="cuda")
    c = torch.full((384, 70), 5.0, device="cuda")
    F.int8_gemm_grouped(torch.zeros((384, 0), dtype=torch.int8, device="cuda"), torch.ones(384, device="cuda"),
                        torch.zeros((2, 70, 0), dtype=torch.int8, device="cuda"), torch.ones((2, 70), device="cuda"),
                        off, "f32", c=c)
    assert not c[:256].any() and (c[256:] == 5).all()


def test_refusals():
    import torch
    import fp8_fine_grained_online_amd as F

    def z(*shape, dtype=torch.int8):
        return torch.zeros(shape, dtype=dtype, device="cuda")
    f = torch.float32
    with pytest.raises(F.Fp8qError):
        F.int8_gemm_scaled(z(4, 40), z(4, dtype=f), z(5, 40), z(5, dtype=f))  # K % 16
    with pytest.raises(ValueError):
        F.int8_gemm_scaled(z(4, 64), z(3, dtype=f), z(5, 64), z(5, dtype=f))
    with pytest.raises(ValueError):
        F.int8_gemm_scaled(z(4, 64), z(4, dtype=f), z(5, 32), z(5, dtype=f))
    with pytest.raises(TypeError):
        F.int8_gemm_scaled(z(4, 64, dtype=torch.uint8), z(4, dtype=f), z(5, 64), z(5, dtype=f))
    with pytest.raises(ValueError):
        F.int8_gemm_scaled(z(4, 64), z(4, dtype=f), z(5, 64), z(5, dtype=f), out_dtype="f16")
    with pytest.raises(TypeError):
        F.fp8q_quant_int8_rows(z(4, 64))
    with pytest.raises(ValueError):
        F.int8_gemm_grouped(z(128, 64), z(128, dtype=f), z(2, 5, 64), z(2, 4, dtype=f),
                            torch.zeros(3, dtype=torch.int32, device="cuda"))
