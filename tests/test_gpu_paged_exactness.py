"""What a generous bound per element would hide: the low parts of fp16 queries and
weights, and keys left out of a long sum or counted twice."""
import numpy as np
import pytest
import torch

import paged_bounds
from test_gpu_paged import BF, HF, Case, cu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("seqs,group", [
    ([(1, 300)] * 12, 4),                                     # high and low parts in one column tile
    ([(1, 500), (1, 3000)] * 4, 8),                           # in two
    ([(3, 300), (4, 900), (2, 5000)], 8),                     # several row tiles
    ([(100, 200), (60, 900), (40, 5000)], 4),                 # the kernel of many rows
], ids=range(4))
def test_fp16_keeps_its_low_parts(seqs, group, dim, page):
    """The error's root mean square below that of the stated roundings (queries to
    22 bits, weights too in the kernel of few rows, the output to 11)."""
    c = Case(seqs, kv_heads=2, group=group, dim=dim, page=page, dtype=HF)
    x = lambda n, heads: torch.from_numpy(c.g.standard_normal((n, heads, dim)).astype(np.float32)).half()
    start, ln, pos = c.batch([(n, 0) for n in c.len])
    k, v = x(int(start[-1]), 2), x(int(start[-1]), 2)
    c.kv.append(k.cuda(), v.cuda(), cu(pos), cu(start), cu(ln), cu(c.table))
    c.oracle.append(k.float().numpy(), v.float().numpy(), pos, start, ln, c.table)
    c.check_cache()
    start, ln, pos = c.batch(c.seqs)
    q = x(c.n, c.q_heads)
    out = c.kv.attend(q.cuda(), cu(pos), cu(start), cu(ln), cu(c.table), scale=0.3, max_new=max(c.new))
    assert c.kv.debug_state() == 0
    args = (c.oracle, q.float().numpy(), pos, start, ln, c.table)
    weight_step = 2.0 ** -11 if max(c.new) * group > 32 else 2.0 ** -21
    limit = paged_bounds.rms_limit(weight_step, 2.0 ** -11, *args, scale=0.3)
    err = out.double().cpu().numpy() - paged_bounds.outputs(*args, scale=0.3)
    assert np.sqrt((err ** 2).mean()) <= limit, np.sqrt((err ** 2).mean()) / limit


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("seqs,heads,group,dim,page,how", [
    ([(1, 30000)], 1, 1, 128, 64, {}),
    ([(1, 30001), (1, 77), (1, 4000)], 2, 4, 64, 16, {}),
    ([(1, 20000)], 1, 8, 128, 128, dict(window=15001)),
    ([(3, 9000), (2, 100), (4, 12345)], 1, 8, 128, 32, {}),
    ([(200, 20000)], 1, 2, 128, 128, {}),
    ([(64, 9000), (1, 500), (130, 300)], 2, 4, 64, 64, {}),
    ([(300, 7000)], 1, 3, 128, 16, dict(window=5003)),
    ([(50, 8000), (50, 3)], 1, 7, 64, 32, dict(causal=False)),
], ids=range(8))
def test_every_key_counts_once(seqs, heads, group, dim, page, how, dtype):
    """Queries of zeros weigh all keys alike, and the values of every 16 keys are
    ones in a channel of their own (modulo D): each channel is the share of its
    keys among those that the row sees.  16 keys more or less are several steps of
    the bound: the weights' and the output's rounding."""
    c = Case(seqs, kv_heads=heads, group=group, dim=dim, page=page, dtype=dtype)
    start, ln, pos = c.batch([(n, 0) for n in c.len])
    index = np.concatenate([np.arange(n) for n in c.len])
    v = np.zeros((len(index), heads, dim), np.float32)
    for h in range(heads):
        v[np.arange(len(index)), h, (index // 16 + 5 * h) % dim] = 1
    v = torch.from_numpy(v).to(dtype)
    c.kv.append(c.draw(len(index), heads).cuda(), v.cuda(), cu(pos), cu(start), cu(ln), cu(c.table))
    start, ln, pos = c.batch(c.seqs)
    q = torch.zeros((c.n, c.q_heads, dim), dtype=dtype, device="cuda")
    out = c.kv.attend(q, cu(pos), cu(start), cu(ln), cu(c.table), max_new=max(c.new), **how).double().cpu().numpy()
    assert c.kv.debug_state() == 0
    half = torch.finfo(dtype).eps / 2
    bound = (1 + 2.0 ** -11 + 2.0 ** -16) * (1 + half) - 1
    for b, (n, before) in enumerate(seqs):
        total = before + n
        tile = np.zeros((total, dim))
        tile[np.arange(total), np.arange(total) // 16 % dim] = 1
        counts = np.concatenate([np.zeros((1, dim)), np.cumsum(tile, axis=0)])
        for i in range(n):
            hi = before + i + 1 if how.get("causal", True) else total
            lo = max(0, before + i - how["window"] + 1) if "window" in how else 0
            share = counts[hi] - counts[lo]
            if share.min() > 0:
                assert 16 / share.max() > 4 * bound
            for h in range(c.q_heads):
                want = np.roll(share, 5 * (h // group)) / (hi - lo)
                got = out[start[b] + i, h]
                assert (np.abs(got - want) <= bound * want + 2.0 ** -24).all(), (b, i, h)
