"""Pages of the paged cache whose V scales lie far apart: an output channel keeps
its precision whatever the other pages hold, seen or not."""
import numpy as np
import pytest
import torch

from oracle import rope
from test_gpu_paged import BF, HF, Case, cu

pytestmark = pytest.mark.gpu


def fill(c, k, v):
    start, ln, pos = c.batch([(n, 0) for n in c.len])
    k, v = k.to(c.dtype), v.to(c.dtype)
    c.kv.append(k.cuda(), v.cuda(), cu(pos), cu(start), cu(ln), cu(c.table))
    c.oracle.append(k.float().numpy(), v.float().numpy(), pos, start, ln, c.table)
    c.check_cache()


ROWS, TILES = 2.0 ** -19, 2.0 ** -17


def largest_weight_times_values(c, q, causal, window):
    """Per row the largest softmax weight, times the sum of |v| over the keys seen."""
    start, ln, pos = c.batch(c.seqs)
    x = rope.rope_f64(q.float().numpy(), pos, c.axis_dims, 10000.0)
    out = np.zeros(x.shape)
    for b, n in enumerate(ln):
        rows = slice(start[b], start[b + 1])
        at = n - (start[b + 1] - start[b]) + np.arange(start[b + 1] - start[b])
        t = np.arange(n)
        seen = (t <= at[:, None]) | (not causal)
        seen &= (t > at[:, None] - window) if window else True
        for h in range(c.q_heads):
            k, v = (c.oracle.rows(name, c.table[b], n, h * c.kv_heads // c.q_heads) for name in "kv")
            z = np.where(seen, x[rows, h] @ k.T / np.sqrt(c.dim), -np.inf)
            p = 1 / np.exp(z - z.max(axis=1, keepdims=True)).sum(axis=1)
            out[rows, h] = p[:, None] * (seen @ np.abs(v))
    return out


def check(c, small, skip=None, **how):
    """Per element, as the other attention tests, and for every key that is seen
    ``small`` times the row's largest weight: half of fp16's smallest number, 2^-25,
    where a weight may lie 2^14 below its equal on the page with the largest scale
    and that one at 2^8 (2^6 in the kernel of many rows): 2^-19 and 2^-17.  Scales
    further apart are worked on in fp32.  skip: channels left out."""
    q = c.draw(c.n, c.q_heads)
    start, ln, pos = c.batch(c.seqs)
    out = c.kv.attend(q.cuda(), cu(pos), cu(start), cu(ln), cu(c.table), **how).double().cpu().numpy()
    assert c.kv.debug_state() == 0
    causal, window = how.get("causal", True), how.get("window") or 0
    want, spread, logit = c.oracle.attend(q.float().numpy(), pos, start, ln, c.table, causal, window)
    half = torch.finfo(c.dtype).eps / 2
    bound = spread * (np.expm1(2 * (2.0 ** -11 + 2.0 ** -18) * logit)[..., None] + 2.0 ** -11 + 2.0 ** -16)
    bound = bound + small * largest_weight_times_values(c, q, causal, window)
    bound = bound * (1 + half) + np.abs(want) * half + 2.0 ** -24 * (c.dtype is HF) + 1e-30
    ok = np.ones(out.shape, bool)
    if skip is not None:
        ok[..., skip] = False
    err = np.abs(out - want)[ok]
    assert np.isfinite(err).all() and (err <= bound[ok]).all(), f"{(err / bound[ok]).max():.2f} of its bound"
    return out


CHUNKS = [(1, ROWS), (4, ROWS), (50, TILES)]                # 2 to 8 query rows a key head, and 100


@pytest.mark.parametrize("e", [9, 15, 20, 26, 30, 40, 100])
@pytest.mark.parametrize("n,small", CHUNKS, ids=[1, 4, 50])
@pytest.mark.parametrize("where", ["front", "middle", "last"])
def test_one_large_value(where, n, small, e):
    """4,096 keys, one value of one channel 2^e times the others: before all
    others, behind 2,000 of them, and as the last token's, which most of a
    chunk's queries do not see."""
    c = Case([(n, 4096 - n), (n, 100)], kv_heads=2, group=2, page=16 if n == 4 else 64)
    total = sum(c.len)
    k, v = c.draw(total, 2), c.draw(total, 2).float()
    for s, ln in ((0, c.len[0]), (c.len[0], c.len[1])):
        v[s + {"front": 3, "middle": ln // 2, "last": ln - 1}[where], :, 5] = 2.0 ** e
    fill(c, k, v)
    check(c, small)
    check(c, small, max_new=n, window=2050)


@pytest.mark.parametrize("n,small", CHUNKS, ids=[1, 4, 50])
@pytest.mark.parametrize("e", [12, 24])
def test_one_large_value_f16(e, n, small):
    c = Case([(n, 3000)], kv_heads=2, group=2, dim=64, page=32, dtype=HF)
    v = c.draw(c.len[0], 2).float() * 2.0 ** (12 - e)
    v[1500, :, 9] = 2.0 ** 12
    fill(c, c.draw(c.len[0], 2), v)
    check(c, small)


@pytest.mark.parametrize("n,small", CHUNKS, ids=[1, 4, 50])
@pytest.mark.parametrize("step", [11, -11, 3])
@pytest.mark.parametrize("dim,page", [(128, 16), (64, 64)])
def test_scales_that_climb_and_fall(dim, page, step, n, small):
    """Every page's values 2^step times those of the page before, each in a
    channel of its own besides; pages of zeros between and in front."""
    pages = 13
    c = Case([(n, page * pages - n), (n, 7)], kv_heads=1, group=2, dim=dim, page=page)
    total = sum(c.len)
    k, v = c.draw(total, 1), c.draw(total, 1).float() / 4
    for j in range(pages):
        at = v[j * page:(j + 1) * page]
        own = at[..., 4 * j:4 * j + 4].clone()
        at.zero_()
        at[..., 4 * j:4 * j + 4] = own * 2.0 ** (step * (j - 6))
    v[:page] = 0
    v[4 * page:5 * page] = 0
    fill(c, k, v)
    check(c, small)
    check(c, small, causal=False)


@pytest.mark.parametrize("n,small", CHUNKS, ids=[1, 4, 50])
@pytest.mark.parametrize("at", [40, 2999])
def test_an_infinity_in_v(at, n, small):
    """Its page's other values become zeros in that head (the scale is 2^120); the
    rest of the cache and the queries in front of it are as they were."""
    c = Case([(n, 3000 - n)], kv_heads=2, group=2)
    k, v = c.draw(3000, 2), c.draw(3000, 2).float()
    v[at, 1, 77] = float("inf")
    fill(c, k, v)
    out = check(c, small, skip=77)
    front = [i for i in range(n) if 3000 - n + i < at]
    assert np.isfinite(out[front]).all()
    check(c, small, skip=77, window=500)


@pytest.mark.parametrize("n,small", CHUNKS, ids=[1, 4, 50])
@pytest.mark.parametrize("spread", [0, 30])
def test_queries_as_large_as_keys_are_small(spread, n, small):
    """Scores of ordinary size from queries near 2^98 and keys near 2^-96."""
    c = Case([(n, 900), (n, 40)], kv_heads=2, group=2)
    k, v = c.draw(sum(c.len), 2).float() * 2.0 ** -96, c.draw(sum(c.len), 2).float()
    v[17, :, 3] = 2.0 ** spread
    fill(c, k, v)
    draw = c.draw
    c.draw = lambda rows, heads: (draw(rows, heads).float() * 2.0 ** 96).to(BF)
    check(c, small)
