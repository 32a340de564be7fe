"""The root-mean-square limit of the paged attention's fp16 tests, on the CPU: it
lets the kernels' roundings pass and rejects a lost low part."""
import numpy as np
import pytest

import paged_bounds
from oracle.paged import PagedOracle

HALF = 2.0 ** -11                                            # half a step of fp16


def setup(dim, n, before, seed):
    g = np.random.default_rng(seed)
    total, page = n + before, 64
    pages = (total + page - 1) // page
    o = PagedOracle(2, dim, pages, page, (dim,))
    table = np.arange(pages, dtype=np.int32)[None]
    x = lambda rows, heads: g.standard_normal((rows, heads, dim)).astype(np.float16).astype(np.float32)
    pos = np.arange(total, dtype=np.int32)[:, None]
    o.append(x(total, 2), x(total, 2), pos, [0, total], [total], table)
    return o, x(n, 16), pos[before:], [0, n], [total], table


@pytest.mark.parametrize("dim,n,before", [(64, 3, 300), (128, 3, 300), (128, 2, 2000), (64, 2, 3000), (128, 60, 200), (64, 60, 200)])
def test_the_limit_rejects_a_lost_low_part(dim, n, before):
    args, kw = setup(dim, n, before, 0), dict(scale=0.3)
    g = np.random.default_rng(1)
    want = paged_bounds.outputs(*args, **kw)
    rms = lambda out: np.sqrt(((out - want) ** 2).mean())
    fp16 = lambda x: x.astype(np.float16).astype(np.float64)
    rounded_weights = np.zeros(want.shape)
    for rows, h, p, v, _ in paged_bounds.pieces(*args, **kw):
        w = p / p.max(axis=1, keepdims=True) * 2.0 ** g.uniform(6, 14, (len(p), 1))
        rounded_weights[rows, h] = (fp16(w) @ v) / w.sum(axis=1, keepdims=True)
    lost = paged_bounds.outputs(*args, change=paged_bounds.to_fp16_of_row, **kw) - want
    if n > 32:                                               # the kernel of many rows: weights in one fp16 number
        limit = paged_bounds.rms_limit(HALF, HALF, *args, **kw)
        assert rms(fp16(rounded_weights)) < limit < rms(fp16(rounded_weights) + lost) / 1.2
    else:
        limit = paged_bounds.rms_limit(2.0 ** -21, HALF, *args, **kw)
        assert rms(fp16(want)) < limit < rms(fp16(want) + lost) / 1.3
        assert limit < rms(fp16(rounded_weights)) / 1.05
