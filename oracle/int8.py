"""8-bit row quantization and the 8-bit integer product.

  s = fl32(amax / 127), q = clamp(RNE(fl32(x / s)), -127, 127)
  c = fl32(fl32(fl32(sum_k a b) sa) sb), the sum exact

Every step is one correctly rounded binary32 operation, so the results are
defined bit for bit.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""

import numpy as np


def quant_rows(x):
    """x float32 (bfloat16 values) M x K -> (q int8 M x K, s float32 M)."""
    x = np.asarray(x, np.float32)
    amax = np.abs(x).max(axis=1) if x.shape[1] else np.zeros(x.shape[0], np.float32)
    s = (amax / np.float32(127)).astype(np.float32)
    d = np.where(amax > 0, s, np.float32(1))
    q = np.clip(np.rint(x / d[:, None]), -127, 127)
    return q.astype(np.int8), s


def gemm(a, sa, b, sb):
    """float32 M x N. float64 products are exact here: |sum| < 2^31."""
    acc = np.asarray(a, np.float64) @ np.asarray(b, np.float64).T
    with np.errstate(over="ignore", under="ignore"):
        return (acc.astype(np.float32) * np.asarray(sa, np.float32)[:, None]) * np.asarray(sb, np.float32)[None, :]


def gemm_grouped(a, sa, b, sb, m_offsets):
    off = np.asarray(m_offsets, np.int64)
    out = np.full((a.shape[0], b.shape[1]), np.nan, np.float32)
    for e in range(b.shape[0]):
        r = slice(int(off[e]), int(off[e + 1]))
        out[r] = gemm(a[r], sa[r], b[e], sb[e])
    return out
