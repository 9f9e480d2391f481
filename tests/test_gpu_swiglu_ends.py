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
