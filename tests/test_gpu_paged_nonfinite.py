"""NaN in the paged cache: whatever else a page holds, a NaN token is stored as
one and reaches the outputs that see it."""
import numpy as np
import pytest
import torch

from test_gpu_paged import BF, HF, Case, cu

pytestmark = pytest.mark.gpu

NAN = float("nan")


def append(c, seqs, k, v):
    """Rows of k and v (whole sequences, in order) into the cache and the oracle."""
    start, ln, pos = c.batch(seqs)
    c.kv.append(k.cuda(), v.cuda(), cu(pos), cu(start), cu(ln), cu(c.table))
    c.oracle.append(k.float().numpy(), v.float().numpy(), pos, start, ln, c.table)


def attended(c):
    """Every token's queries over the cache, against the formula with NaN."""
    start, ln, pos = c.batch(c.seqs)
    q = c.draw(c.n, c.q_heads)
    out = c.kv.attend(q.cuda(), cu(pos), cu(start), cu(ln), cu(c.table)).float().cpu().numpy()
    with np.errstate(invalid="ignore"):
        want = c.oracle.attend(q.float().numpy(), pos, start, ln, c.table)[0]
    return out, want


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 32), (128, 64), (64, 128)])
@pytest.mark.parametrize("n", [1, 3, 70])
def test_blocks_of_nan(dtype, dim, page, n):
    """n new tokens per sequence whose key head 1 is all NaN: in fresh pages,
    behind rows of scale 0, behind ordinary rows; head 0 is ordinary.  Then
    ordinary rows behind the NaN ones, which grow the scales."""
    befores = [0, page, 5, page + 7]
    c = Case([(0, b + n + 9) for b in befores], kv_heads=2, group=2, dim=dim, page=page, dtype=dtype)
    total = sum(befores)
    k, v = c.draw(total, 2), c.draw(total, 2)
    k[page:page + 5], v[page:page + 5] = 0, 0                 # the third sequence: scale 0
    append(c, [(b, 0) for b in befores], k, v)
    k, v = c.draw(4 * n, 2), c.draw(4 * n, 2)
    k[:, 1], v[:, 1] = NAN, NAN
    append(c, [(n, b) for b in befores], k, v)
    c.check_cache()
    k, v = c.draw(4 * 9, 2).float() * 8, c.draw(4 * 9, 2).float() * 8
    append(c, [(9, b + n) for b in befores], k.to(dtype), v.to(dtype))
    c.check_cache()
    assert c.kv.debug_state() == 0
    c.seqs, c.n, c.rows = [(9, b + n) for b in befores], 36, 36
    out, want = attended(c)
    assert np.isnan(want[:, 2:]).all() and np.isnan(out[:, 2:]).all()       # key head 1
    assert np.isfinite(out[:, :2]).all()
    assert c.kv.debug_state() == 0


@pytest.mark.parametrize("few", [True, False])
def test_nan_beside_rows_that_are_zero(few):
    """One NaN row among rows below 2^-100, with either kernel; values only, keys
    only, one channel only."""
    n = 2 if few else 40
    c = Case([(n, 0)] * 4, kv_heads=1, group=3, page=16)
    k, v = (c.draw(4 * n, 1).float() * 2.0 ** -110 for _ in range(2))
    k[:n] = c.draw(n, 1).float()
    k[n - 1] = NAN                                            # beside ordinary keys
    k[n + n // 2] = NAN                                       # beside keys of nothing
    v[2 * n + n // 2, 0, 37] = NAN
    append(c, [(n, 0)] * 4, k.to(BF), v.to(BF))
    c.check_cache()
    out, _ = attended(c)
    sees = np.zeros(4 * n, bool)                              # rows that see a NaN
    sees[n - 1] = sees[n + n // 2:2 * n] = True
    assert np.isnan(out[sees]).all()
    sees[2 * n + n // 2:3 * n] = True                         # a value's NaN: its channel, or the whole row
    assert np.isnan(out[2 * n + n // 2:3 * n, :, 37]).all()
    assert np.isfinite(out[~sees]).all()
    assert c.kv.debug_state() == 0
