"""GPU permute, combine and combine's gradient against the float64 oracle: rows bit
for bit, sums within the roundings of their terms, unwritten rows untouched."""

import numpy as np
import pytest

from conftest import gpu_available
from fp8_fine_grained_online_amd import synthetic as S
from oracle import tokens

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

EPS32 = 2.0 ** -24   # half a step of binary32, relative
BF16 = 2.0 ** -8     # and of bfloat16


def dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def rounding(name):
    return BF16 if name == "bf16" else 0.0


def routing(T, topk, G, seed, drop=0):
    rng = S.rng_for(seed, 1)
    ids = np.stack([rng.permutation(G)[:topk] if topk <= G else rng.integers(0, G, topk) for _ in range(T)])
    ids = ids.astype(np.int32).reshape(T, topk)
    if drop and T:
        ids[::drop, 0] = -1
        ids[1::drop, topk - 1] = G + 2
    return ids


def randn(shape, name, seed):
    import torch
    return torch.from_numpy(S.rng_for(seed, 2).standard_normal(shape)).to(dtype(name)).cuda()


CASES = [(1, 1, 1, 8), (1, 8, 32, 7168), (3, 2, 4, 16), (33, 6, 64, 2056), (300, 2, 7, 512), (129, 1, 1, 128),
         (50, 8, 256, 1032), (700, 4, 5, 520), (9, 70, 128, 64), (2, 300, 1024, 72), (1500, 8, 600, 8)]


@pytest.mark.parametrize("name", ["bf16", "f32"])
@pytest.mark.parametrize("T,topk,G,K", CASES)
def test_permute(T, topk, G, K, name):
    import torch
    import fp8_fine_grained_online_amd as F
    ids = routing(T, topk, G, 2600 + T, drop=5)
    x = randn((T, K), name, 2601)
    cap = F.lib().fp8q_moe_dispatch_max_rows(T, topk, G)
    xp = torch.full((cap, K), float("nan"), dtype=dtype(name), device="cuda")
    _, off, rows = F.fp8q_moe_permute(x, torch.from_numpy(ids).cuda(), G, xp=xp)
    want, want_off, want_rows = tokens.permute(x.float().cpu().numpy(), ids, G)
    assert np.array_equal(off.cpu().numpy(), want_off)
    assert np.array_equal(rows.cpu().numpy(), want_rows)
    got = xp.float().cpu().numpy()
    assert np.array_equal(got[:len(want)], want)
    assert np.isnan(got[len(want):]).all()  # not written


@pytest.mark.parametrize("T,topk,G", [(2048, 1, 8), (2049, 1, 8), (256, 8, 1024), (257, 8, 1024), (32, 64, 100),
                                      (1024, 1, 8), (1025, 1, 8), (128, 8, 1024), (129, 8, 1024), (16, 64, 100),
                                      (1000, 6, 1024), (1366, 3, 1), (3, 5000, 100), (4096, 16, 40), (4097, 2, 3),
                                      (5, 13200, 64), (65537, 1, 3), (9000, 8, 64)])
def test_permute_where_the_sort_changes_hands(T, topk, G):
    """1024 slots are sorted inside the copy, 65536 of at most 4096 tokens are counted in blocks of 4096 (a token's
    slots may lie in several), more in blocks of 256: the same rows."""
    import torch
    import fp8_fine_grained_online_amd as F
    ids = routing(T, topk, G, 2650 + T, drop=9)
    x = randn((T, 24), "bf16", 2651)
    xp, off, rows = F.fp8q_moe_permute(x, torch.from_numpy(ids).cuda(), G)
    want, want_off, want_rows = tokens.permute(x.float().cpu().numpy(), ids, G)
    assert np.array_equal(off.cpu().numpy(), want_off)
    assert np.array_equal(rows.cpu().numpy(), want_rows)
    assert np.array_equal(xp[:len(want)].float().cpu().numpy(), want)


def test_permute_is_the_dispatch_layout():
    import torch
    import fp8_fine_grained_online_amd as F
    for T, topk, G in ((64, 8, 32), (3000, 6, 100)):
        ids = torch.from_numpy(routing(T, topk, G, 2610, drop=7)).cuda()
        x = randn((T, 256), "bf16", 2611)
        _, _, off, rows = F.fp8q_moe_dispatch_1x128(x, ids, G)
        _, off2, rows2 = F.fp8q_moe_permute(x, ids, G)
        assert torch.equal(off, off2) and torch.equal(rows, rows2)


def test_permute_with_the_callers_buffers():
    """A workspace of exactly the stated size, kept between calls of each of the three sorting paths, and its end
    left alone; one byte less is refused."""
    import torch
    import fp8_fine_grained_online_amd as F
    for T, topk, G in ((200, 2, 9), (2000, 8, 40), (9000, 2, 16)):
        need = F.lib().fp8q_moe_dispatch_workspace_bytes(T, topk, G)
        buffer = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        x = randn((T, 16), "f32", 2613)
        for seed in (1, 2):
            ids = routing(T, topk, G, 2614 + seed, drop=6)
            off = torch.full((G + 1,), -7, dtype=torch.int32, device="cuda")
            rows = torch.full((T, topk), -7, dtype=torch.int32, device="cuda")
            xp, off2, rows2 = F.fp8q_moe_permute(x, torch.from_numpy(ids).cuda(), G, m_offsets=off, row_of_slot=rows,
                                                 workspace=buffer[:need])
            assert off2 is off and rows2 is rows
            want, want_off, want_rows = tokens.permute(x.cpu().numpy(), ids, G)
            assert np.array_equal(off.cpu().numpy(), want_off) and np.array_equal(rows.cpu().numpy(), want_rows)
            assert np.array_equal(xp[:len(want)].cpu().numpy(), want)
            assert (buffer[need:] == 0xA5).all()
        with pytest.raises(F.Fp8qError):
            F.fp8q_moe_permute(x, torch.from_numpy(ids).cuda(), G, workspace=buffer[:need - 1])


def test_permute_without_tokens_or_columns():
    import torch
    import fp8_fine_grained_online_amd as F
    off = torch.full((9,), -7, dtype=torch.int32, device="cuda")
    F.fp8q_moe_permute(torch.empty((0, 64), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda"), 8,
                       m_offsets=off)
    assert not off.any()
    ids = routing(40, 2, 8, 2612)
    _, off, rows = F.fp8q_moe_permute(torch.empty((40, 0), device="cuda"), torch.from_numpy(ids).cuda(), 8)
    want_rows, want_off, _ = tokens.layout(ids, 8)
    assert np.array_equal(off.cpu().numpy(), want_off) and np.array_equal(rows.cpu().numpy(), want_rows)


@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("dst", ["bf16", "f32"])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,topk,G,K", CASES)
def test_combine(T, topk, G, K, src, dst, weighted):
    import torch
    import fp8_fine_grained_online_amd as F
    ids = routing(T, topk, G, 2620 + T, drop=4)
    if T > 2:
        ids[2] = -1  # a token without experts
    rows, off, _ = tokens.layout(ids, G)
    M = int(off[-1])
    c = torch.full((max(M, 1), K), float("nan"), dtype=dtype(src), device="cuda")  # rows that nothing maps: NaN
    used = np.unique(rows[rows >= 0])
    c[torch.from_numpy(used).cuda().long()] = randn((used.size, K), src, 2621)
    w = S.rng_for(2622, T).random((T, topk)).astype(np.float32) if weighted else None
    if weighted:
        w[rows < 0] = np.nan  # nor is a dropped choice's weight used
    y = torch.full((T, K), float("nan"), dtype=dtype(dst), device="cuda")
    F.fp8q_moe_combine(c, torch.from_numpy(rows).cuda(), None if w is None else torch.from_numpy(w).cuda(),
                       out_dtype=dst, y=y)
    want, mag = tokens.combine(c.double().cpu().numpy(), rows, w)
    # one rounding per term of at most the running sum of magnitudes, then the output's
    tol = topk * EPS32 * mag + rounding(dst) * (np.abs(want) + topk * EPS32 * mag)
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol)


def test_rows_beyond_the_cache():
    """More than 256 MiB of rows (read and stored another way), against float64 sums in torch."""
    import torch
    import fp8_fine_grained_online_amd as F
    T, topk, G, K = 2600, 8, 16, 7168
    ids = torch.from_numpy(routing(T, topk, G, 2635, drop=9)).cuda()
    x = randn((T, K), "bf16", 2636)
    xp, off, rows = F.fp8q_moe_permute(x, ids, G)
    want_rows, want_off, _ = tokens.layout(ids.cpu().numpy(), G)
    assert np.array_equal(rows.cpu().numpy(), want_rows) and np.array_equal(off.cpu().numpy(), want_off)
    on = rows >= 0
    assert torch.equal(xp[rows[on].long()], x.unsqueeze(1).expand(T, topk, K)[on])
    w = torch.rand(T, topk, device="cuda", generator=torch.Generator("cuda").manual_seed(6))
    y = F.fp8q_moe_combine(xp, rows, w, out_dtype="f32")
    for t in range(0, T, 650):
        s = slice(t, t + 650)
        terms = torch.where(on[s].unsqueeze(2), xp[rows[s].clamp(min=0).long()].double() * w[s].double().unsqueeze(2), 0.0)
        assert torch.all((y[s].double() - terms.sum(1)).abs() <= topk * EPS32 * terms.abs().sum(1))
    dc, dw = F.fp8q_moe_combine_bwd(x, xp, rows, w, off)
    # dc = w x: one product rounded to binary32, then to bfloat16; c's rows are x's, so dw is |x|^2
    want = (w.unsqueeze(2) * x.float().unsqueeze(1))[on].to(torch.bfloat16)
    assert torch.equal(dc[rows[on].long()], want)
    norm = x.double().square().sum(1, keepdim=True)
    assert torch.all((dw.double() - torch.where(on, norm, 0.0)).abs() <= (K / 64 + 24) * EPS32 * norm)


def padding_of(rows, off, M):
    """(rows below off[G] that nothing maps, rows from off[G] on), as masks over M rows."""
    import torch
    mapped = torch.zeros(M, dtype=torch.bool, device="cuda")
    mapped[rows[rows >= 0].long()] = True
    behind = torch.arange(M, device="cuda") >= off[-1]
    return ~mapped & ~behind, behind


@pytest.mark.parametrize("name", ["bf16", "f32"])
@pytest.mark.parametrize("T,topk,G,K", [(2600, 8, 16, 7168), (5600, 3, 300, 64), (16385, 1, 7, 200), (2048, 8, 40, 4096),
                                        (300, 8, 256, 4096), (9000, 2, 1024, 24)])
def test_padding_rows_are_zero_and_rows_behind_stay(T, topk, G, K, name):
    """Sixteen and four zeroing workgroups per expert (up to 16384 slots, and more), rows that fit the cache and that
    do not (stored another way), blocks without a row: padding is zero in every element, rows behind are not written."""
    import torch
    import fp8_fine_grained_online_amd as F
    ids = routing(T, topk, G, 2660 + T, drop=5)
    ids[ids == G - 2] = G - 1  # an expert without rows
    ids = torch.from_numpy(ids).cuda()
    x, dy = randn((T, K), name, 2661), randn((T, K), name, 2662)
    cap = F.lib().fp8q_moe_dispatch_max_rows(T, topk, G)
    xp = torch.full((cap, K), float("nan"), dtype=dtype(name), device="cuda")
    _, off, rows = F.fp8q_moe_permute(x, ids, G, xp=xp)
    padding, behind = padding_of(rows, off, cap)
    assert padding.any() and behind.any()
    assert torch.count_nonzero(xp[padding]) == 0 and torch.isnan(xp[behind]).all()
    w = torch.rand(T, topk, device="cuda", generator=torch.Generator("cuda").manual_seed(8))
    c = torch.where(padding.unsqueeze(1), float("nan"), xp.float()).to(dtype(name))  # padding is never read
    want = (w.unsqueeze(2) * dy.float().unsqueeze(1)).to(dtype(name)) if T * topk * K < 1 << 28 else None
    for with_dw in (True, False):
        dc = torch.full((cap, K), float("nan"), dtype=dtype(name), device="cuda")
        _, dw = F.fp8q_moe_combine_bwd(dy, c, rows, w, off, dc=dc, with_dw=with_dw)
        assert torch.count_nonzero(dc[padding]) == 0 and torch.isnan(dc[behind]).all()
        on = rows >= 0
        if want is not None:
            assert torch.equal(dc[rows[on].long()], want[on])
        if with_dw:
            assert torch.isfinite(dw).all() and torch.count_nonzero(dw[~on]) == 0


def test_combine_skips_rows_outside():
    import torch
    import fp8_fine_grained_online_amd as F
    c = randn((128, 64), "bf16", 2630)
    rows = torch.tensor([[0, 128], [-5, 127], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device="cuda")
    y = F.fp8q_moe_combine(c, rows, out_dtype="f32")
    assert torch.equal(y, torch.stack([c[0], c[127], torch.zeros_like(c[0])]).float())


@pytest.mark.parametrize("gy", ["bf16", "f32"])
@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,topk,G,K", CASES)
def test_combine_gradient(T, topk, G, K, gy, src, weighted):
    import torch
    import fp8_fine_grained_online_amd as F
    ids = routing(T, topk, G, 2640 + T, drop=3)
    rows, off, _ = tokens.layout(ids, G)
    M = int(off[-1]) + 128  # rows behind the last block
    c = randn((M, K), src, 2641)
    dy = randn((T, K), gy, 2642)
    w = S.rng_for(2643, T).random((T, topk)).astype(np.float32) if weighted else None
    wd = None if w is None else torch.from_numpy(w).cuda()
    dc = torch.full((M, K), float("nan"), dtype=dtype(src), device="cuda")
    rd, od = torch.from_numpy(rows).cuda(), torch.from_numpy(off).cuda()
    _, dw = F.fp8q_moe_combine_bwd(dy, c, rd, wd, od, dc=dc)
    want, want_dw, mag = tokens.combine_bwd(dy.double().cpu().numpy(), c.double().cpu().numpy(), rows, w, off)
    got = dc.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))  # padding written, rows behind not
    ok = ~np.isnan(want)
    # one product rounded to binary32 and to c's type
    assert np.all(np.abs(got - want)[ok] <= (EPS32 + rounding(src) * (1 + EPS32)) * np.abs(want[ok]))
    # a lane's chain is at most K / 64 terms long here; the tree over lanes and waves adds under 16
    assert np.all(np.abs(dw.double().cpu().numpy() - want_dw) <= (K / 64 + 24) * EPS32 * mag)
    dc2 = torch.full_like(dc, float("nan"))
    _, none = F.fp8q_moe_combine_bwd(dy, c, rd, wd, od, dc=dc2, with_dw=False)
    assert none is None and torch.equal(torch.nan_to_num(dc2), torch.nan_to_num(dc))


def test_gradient_without_tokens_zeroes_the_blocks():
    import torch
    import fp8_fine_grained_online_amd as F
    off = torch.tensor([0, 128, 128, 256], dtype=torch.int32, device="cuda")
    c = torch.ones(384, 16, device="cuda")
    dc = torch.full_like(c, 3.0)
    dw = F.fp8q_moe_combine_bwd(torch.empty((0, 16), device="cuda"), c,
                                torch.empty((0, 2), dtype=torch.int32, device="cuda"), None, off, dc=dc)[1]
    assert dw.shape == (0, 2) and not dc[:256].any() and (dc[256:] == 3).all()


def test_offsets_past_32_bits():
    """Rows whose byte offset does not fit 32 bits: 9000 x 131072 float32 is 4.7 GB."""
    import torch
    import fp8_fine_grained_online_amd as F
    K, M = 131072, 8960
    c = torch.zeros(M, K, device="cuda")
    c[M - 1] = torch.arange(K, device="cuda")
    rows = torch.tensor([[M - 1, 0]], dtype=torch.int32, device="cuda")
    y = F.fp8q_moe_combine(c, rows, out_dtype="f32")
    assert torch.equal(y[0], c[M - 1])
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    dc = torch.zeros_like(c)
    F.fp8q_moe_combine_bwd(y, c, rows, None, off, dc=dc)
    assert torch.equal(dc[M - 1], y[0]) and torch.equal(dc[0], y[0])
    assert not dc[1:M - 1:997].any()


def test_permuted_rows_past_32_bits():
    """70 experts' blocks of 128 rows of 262144 bfloat16: 4.7 GB, the last token's row and its padding at its end."""
    import torch
    import fp8_fine_grained_online_amd as F
    K, G = 262144, 70
    x = torch.arange(1, G + 1, device="cuda").to(torch.bfloat16).unsqueeze(1).expand(G, K).contiguous()
    ids = torch.arange(G, dtype=torch.int32, device="cuda").unsqueeze(1)
    xp, off, rows = F.fp8q_moe_permute(x, ids, G, xp=torch.full((F.lib().fp8q_moe_dispatch_max_rows(G, 1, G), K), 3.0,
                                                                dtype=torch.bfloat16, device="cuda"))
    assert off[G] == 128 * G and torch.equal(rows[:, 0], 128 * torch.arange(G, dtype=torch.int32, device="cuda"))
    for e in (0, G - 1):
        assert (xp[128 * e] == e + 1).all() and not xp[128 * e + 1:128 * e + 128].any()


def test_refusals():
    import torch
    import fp8_fine_grained_online_amd as F
    x = torch.zeros(4, 64, device="cuda")
    rows = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(F.Fp8qError):
        F.fp8q_moe_permute(torch.zeros(4, 60, device="cuda"), rows, 4)
    with pytest.raises(ValueError):
        F.fp8q_moe_permute(x, rows, 0)
    with pytest.raises(TypeError):
        F.fp8q_moe_permute(x.half(), rows, 4)
    with pytest.raises(ValueError):
        F.fp8q_moe_permute(x, rows[:3], 4)
    with pytest.raises(ValueError):
        F.fp8q_moe_combine(x, rows.cpu())
    with pytest.raises(ValueError):
        F.fp8q_moe_combine(x, rows, torch.ones(4, 3, device="cuda"))
    with pytest.raises(ValueError):
        F.fp8q_moe_combine(x[:, ::2], rows)
    with pytest.raises(ValueError):
        F.fp8q_moe_combine_bwd(x[:3], x, rows, None, off)
    with pytest.raises(TypeError):
        F.fp8q_moe_combine_bwd(x, x, rows.long(), None, off)
