"""The paged cache on the GPU against its numpy oracle: the appended codes and
scales bit for bit, the attention within a bound derived from its roundings,
over types, head layouts, page sizes, ragged lengths, masks, strides, streams
and graphs."""
import numpy as np
import pytest
import torch

import synth
from oracle.paged import PagedOracle

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def paged(*args, **kw):
    from fp8_ring_kv_gb300.paged import PagedKV
    return PagedKV(*args, **kw)


class Case:
    """A cache with its oracle, and one batch of sequences (new, before)."""

    def __init__(self, seqs, kv_heads=2, group=2, dim=128, page=64, axes=1, dtype=BF, seed=0, extra_rows=0, width=None,
                 layers=1, big=1.0):
        self.seqs, self.kv_heads, self.q_heads, self.dim, self.page, self.dtype = seqs, kv_heads, kv_heads * group, dim, page, dtype
        self.axis_dims = (dim,) if axes == 1 else (dim // 4, dim * 3 // 8, dim * 3 // 8)
        self.g = np.random.default_rng(seed)
        self.new = [a for a, _ in seqs]
        self.len = [a + c for a, c in seqs]
        held = [(n + page - 1) // page for n in self.len]
        self.n_pages = sum(held) + 2
        order = self.g.permutation(self.n_pages)
        width = width or max(1, max(held))
        self.table = np.full((len(seqs), width), -1, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.n = int(self.start[-1])
        self.rows = self.n + extra_rows
        top = max([1] + self.len) + 1
        self.pos_count = (top,) if axes == 1 else (top // 12 + 1, 3, 4)
        self.kv = paged(kv_heads, self.q_heads, dim, self.n_pages, page, self.axis_dims, (0,) * axes, self.pos_count,
                        dtype=dtype, layers=layers)
        self.oracle = PagedOracle(kv_heads, dim, self.n_pages, page, self.axis_dims)
        self.big = big

    def positions(self, index):
        index = np.maximum(np.asarray(index), 0)
        if len(self.axis_dims) == 1:
            return index[:, None].astype(np.int32)
        return np.stack([index // 12, index // 4 % 3, index % 4], 1).astype(np.int32)

    def draw(self, n, heads):
        """n tokens' heads in the cache's type, a few channels louder."""
        x = self.g.standard_normal((n, heads, self.dim)).astype(np.float32) * np.float32(self.big)
        x[..., ::37] *= 4
        return torch.from_numpy(x).to(self.dtype)

    def batch(self, seqs):
        start = np.concatenate([[0], np.cumsum([a for a, _ in seqs])]).astype(np.int32)
        ln = np.array([a + c for a, c in seqs], np.int32)
        index = np.concatenate([np.arange(c, c + a) for a, c in seqs] + [np.zeros(0, int)])
        return start, ln, self.positions(index)

    def append(self, seqs, k=None, v=None, layer=0, oracle=True):
        start, ln, pos = self.batch(seqs)
        n = int(start[-1])
        k = self.draw(n, self.kv_heads) if k is None else k
        v = self.draw(n, self.kv_heads) if v is None else v
        self.kv.append(k.cuda(), v.cuda(), cu(pos), cu(start), cu(ln), cu(self.table), layer=layer)
        if oracle:
            self.oracle.append(k.float().numpy(), v.float().numpy(), pos, start, ln, self.table)

    def fill(self, pieces=1):
        """Everything before the batch, and the batch's own tokens, in so many calls."""
        cuts = [[n * i // pieces for n in self.len] for i in range(pieces + 1)]
        for lo, hi in zip(cuts, cuts[1:]):
            self.append([(b - a, a) for a, b in zip(lo, hi)])

    def check_cache(self, layer=0):
        torch.cuda.synchronize()
        for name in "kv":
            codes = getattr(self.kv, name + "_codes")[layer].cpu().numpy()
            scales = getattr(self.kv, name + "_scales")[layer].cpu().numpy()
            assert np.array_equal(scales.view(np.uint32), self.oracle.scales[name].view(np.uint32)), name
            bad = np.argwhere(codes != self.oracle.codes[name])
            assert bad.size == 0, f"{name}: {len(bad)} codes differ, first {bad[:4].tolist()}"

    def attend(self, causal=True, window=None, scale=None, max_new=None, q=None):
        q = self.draw(self.rows, self.q_heads) if q is None else q
        start, ln, pos = self.batch(self.seqs)
        pos = np.concatenate([pos, np.zeros((self.rows - self.n, pos.shape[1]), np.int32)])
        out = torch.full((self.rows, self.q_heads, self.dim), 7.0, dtype=self.dtype, device="cuda")
        got = self.kv.attend(q.cuda(), cu(pos), cu(start), cu(ln), cu(self.table), out=out, causal=causal,
                             window=window, scale=scale, max_new=max_new)
        assert got is out
        want = self.oracle.attend(q[:self.n].float().numpy(), pos[:self.n], start, ln, self.table, causal, window or 0, scale)
        self.check_out(out, *want)
        assert bool((out[self.n:] == 7.0).all())         # rows past the last sequence stay as they were
        return out

    def check_out(self, out, want, spread, logit):
        """Per element, with u = 2^-11 (fp16 rounding, half a step): the query
        in fp16 moves a logit by at most u * scale * sum |q_d k_d| (logit * u),
        so a weight by the factor exp(2 u logit) with its sum; a weight's own
        fp16 rounding is another u.  fp32 sums over D and the keys: 2^-16 is
        generous for D = 128 products and a few thousand keys.  Then the
        output's rounding, half a step of its type."""
        u = 2.0 ** -11
        half = torch.finfo(self.dtype).eps / 2
        bound = spread * (np.expm1(2 * (u + 2.0 ** -18) * logit)[..., None] + u + 2.0 ** -16)
        bound = bound * (1 + half) + np.abs(want) * half + 2.0 ** -24 * (1 if self.dtype is HF else 0) + 1e-30
        err = np.abs(out[:self.n].double().cpu().numpy() - want)
        worst = float((err / bound).max()) if err.size else 0.0
        assert np.isfinite(err).all() and worst <= 1.0, f"error {err.max():.3e}, {worst:.2f} of its bound"


def cu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


APPENDS = [
    dict(seqs=[(1, 0)]),
    dict(seqs=[(1, 63), (1, 64), (1, 65), (5, 0)], page=64),
    dict(seqs=[(200, 0), (3, 77), (0, 40), (129, 15)], page=16, dim=64, kv_heads=3, group=1, dtype=HF),
    dict(seqs=[(131, 130), (64, 64), (2, 31)], page=32, axes=3, kv_heads=1, group=4),
    dict(seqs=[(300, 1), (128, 128), (127, 1), (1, 127)], page=128, kv_heads=5, group=3),
    dict(seqs=[(260, 100), (17, 0)], page=128, dim=64, axes=3, kv_heads=2, dtype=HF),
    dict(seqs=[(1, i) for i in range(150)], page=16, kv_heads=1, group=1),
    dict(seqs=[(1, 10)], kv_heads=128, group=1, dim=64, page=16),
]


@pytest.mark.parametrize("pieces", [1, 2, 5])
@pytest.mark.parametrize("case", APPENDS, ids=range(len(APPENDS)))
def test_append_bit_for_bit(case, pieces):
    c = Case(**case)
    c.fill(pieces)
    c.check_cache()
    assert c.kv.debug_state() == 0


ATTENDS = [
    (dict(seqs=[(1, 0)]), {}),
    (dict(seqs=[(1, 776)], kv_heads=8, group=4), {}),
    (dict(seqs=[(1, 5), (1, 0), (1, 63), (1, 64), (1, 1500), (1, 31)], group=4), {}),
    (dict(seqs=[(1, 300)] * 40, kv_heads=1, group=1, dim=64, page=16, dtype=HF), {}),
    (dict(seqs=[(3, 100), (1, 7), (0, 9), (5, 0)], group=3, page=32), {}),
    (dict(seqs=[(2, 900), (16, 200)], kv_heads=1, group=8, page=128), dict(window=100)),
    (dict(seqs=[(70, 0), (1, 400), (33, 65)], kv_heads=2, group=1, page=16), dict(window=33)),
    (dict(seqs=[(257, 0), (40, 300)], group=4), {}),
    (dict(seqs=[(300, 11)], kv_heads=3, group=1, dim=64, axes=3, dtype=HF), dict(causal=False)),
    (dict(seqs=[(129, 0), (128, 0), (127, 0)], kv_heads=1, group=2, page=128), {}),
    (dict(seqs=[(9, 0), (1, 250)], kv_heads=1, group=16, page=64), dict(scale=0.3)),
    (dict(seqs=[(600, 700)], kv_heads=1, group=7, page=32, dtype=HF), {}),
    (dict(seqs=[(520, 0), (64, 1000)], kv_heads=2, group=8, page=64), dict(window=200)),
    (dict(seqs=[(757, 500)], kv_heads=2, group=1, axes=3), dict(causal=False)),
    (dict(seqs=[(150, 0)], kv_heads=1, group=2, big=20.0), {}),
    (dict(seqs=[(1, 9000)], kv_heads=2, group=4), {}),
]


@pytest.mark.parametrize("case,how", ATTENDS, ids=range(len(ATTENDS)))
def test_attend(case, how):
    c = Case(extra_rows=3, **case)
    c.fill(2)
    c.check_cache()
    c.attend(**how)
    if max(c.new) > 0:
        c.attend(max_new=max(c.new), **how)
    assert c.kv.debug_state() == 0


# ---------------------------------------------------------------- long and split
SPLITS = [
    (dict(seqs=[(200, 20000)], kv_heads=1, group=2, page=128), {}),            # one item over the whole GPU
    (dict(seqs=[(1, 30000)], kv_heads=1, group=16, page=64), {}),
    (dict(seqs=[(1, 30000)], kv_heads=2, group=4, page=16, dim=64, dtype=HF), {}),
    (dict(seqs=[(1, 12000)], kv_heads=1, group=8, page=32, dtype=HF), dict(window=5000)),
    (dict(seqs=[(40, 9000)], kv_heads=2, group=7, page=64, dtype=HF), {}),
    (dict(seqs=[(100, 6000)], kv_heads=1, group=3, dim=64, page=16), dict(window=700)),
    (dict(seqs=[(3, 17), (130, 1), (1, 4000), (64, 64), (2, 0), (300, 2000), (1, 1)], kv_heads=2, group=4), {}),
]


@pytest.mark.parametrize("case,how", SPLITS, ids=range(len(SPLITS)))
def test_attend_split_items(case, how):
    c = Case(**case)
    c.fill(3)
    c.check_cache()
    out = c.attend(**how)
    assert c.kv.debug_state() == 0
    # the same call gives the same bits, whoever finishes first
    q = c.draw(c.rows, c.q_heads)
    a = [c.attend(q=q, **how).clone() for _ in range(3)]
    assert bool((a[0] == a[1]).all()) and bool((a[0] == a[2]).all())
    del out


def test_query_heads_and_sequences_at_their_limits():
    c = Case([(1, i % 40) for i in range(2048)], kv_heads=1, group=2, dim=64, page=16)
    c.fill(1)
    c.check_cache()
    c.attend(max_new=1)
    c = Case([(2, 30)], kv_heads=128, group=8, dim=64, page=32)
    c.fill(2)
    c.attend()
    assert c.kv.debug_state() == 0


def test_offsets_past_32_bits():
    """Pages whose codes lie more than 2^32 bytes into the pool."""
    c = Case([(3, 200), (90, 100)], kv_heads=8, group=2, page=128)
    pages = 34000                                            # x 128 KiB of K codes: 4.45e9 bytes
    c.kv = paged(8, 16, 128, pages, 128, (128,), (0,), c.pos_count)
    c.oracle = PagedOracle(8, 128, c.n_pages, 128, (128,))
    small = c.table.copy()
    c.table = np.where(small >= 0, pages - 1 - small, -1).astype(np.int32)
    assert int(c.table.max()) * 128 * 8 * 128 > 2 ** 32

    start, ln, pos = c.batch([(n, 0) for n in c.len])
    k, v = c.draw(int(start[-1]), 8), c.draw(int(start[-1]), 8)
    c.kv.append(k.cuda(), v.cuda(), cu(pos), cu(start), cu(ln), cu(c.table))
    c.oracle.append(k.float().numpy(), v.float().numpy(), pos, start, ln, small)
    torch.cuda.synchronize()
    for name in "kv":
        got = getattr(c.kv, name + "_codes")[0][pages - c.n_pages:].flip(0).cpu().numpy()
        assert np.array_equal(got, c.oracle.codes[name])
    start, ln, pos = c.batch(c.seqs)
    q = c.draw(c.n, 16)
    out = c.kv.attend(q.cuda(), cu(pos), cu(start), cu(ln), cu(c.table))
    c.check_out(out, *c.oracle.attend(q.float().numpy(), pos, start, ln, small))


# ---------------------------------------------------------------- masks and what lies behind them
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (128, 16), (64, 128)])
def test_stale_pages_stay_behind_the_mask(dim, page, dtype):
    """A pool full of NaN codes and non-finite scales, as freed pages may be:
    what no query sees never reaches an output, and pages that a window has
    left behind need not be in the table."""
    for window in (None, 70):
        c = Case([(1, 100), (50, 75), (3, 200), (1, page - 1)], group=4, dim=dim, page=page, dtype=dtype)
        for name in "kv":
            getattr(c.kv, name + "_codes").fill_(0x7F)
            getattr(c.kv, name + "_scales").fill_(float("nan"))
        c.fill(2)
        table = c.table.copy()
        if window:
            for b, (n, before) in enumerate(c.seqs):
                gone = max(0, before + 1 - window) // page
                c.table[b, :gone] = -7
        q = c.draw(c.rows, c.q_heads)
        start, ln, pos = c.batch(c.seqs)
        out = c.kv.attend(q.cuda(), cu(pos), cu(start), cu(ln), cu(c.table), window=window)
        c.check_out(out, *c.oracle.attend(q.float().numpy(), pos, start, ln, table, True, window or 0))
        assert c.kv.debug_state() == 0


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("seqs", [[(4, 60)], [(100, 30), (3, 90)], [(1, 9000), (4, 9000)], [(70, 9000)]])
def test_nan_reaches_only_the_queries_that_see_it(seqs, dim, dtype):
    """NaN values and keys in some of the tokens: queries in front of them (or
    behind the window) are untouched, the others have NaN where the formula has."""
    c = Case(seqs, kv_heads=2, group=2, dim=dim, page=16, dtype=dtype)
    start, ln, pos = c.batch([(n, 0) for n in c.len])
    k, v = c.draw(int(start[-1]), 2), c.draw(int(start[-1]), 2)
    nan_k, nan_v = [], []                                    # (sequence, cache index), key head 0 or 1
    for b, (n, before) in enumerate(seqs):
        if n > 1:
            v[start[b] + before + n // 2, 0, 5] = float("nan")
            nan_v.append((b, before + n // 2))
        k[start[b] + before + n - 1, 1, 8] = float("nan")
        nan_k.append((b, before + n - 1))
        v[start[b] + 3, 1, 7] = float("nan")                 # left behind by the window
    c.kv.append(k.cuda(), v.cuda(), cu(pos), cu(start), cu(ln), cu(c.table))
    c.oracle.append(k.float().numpy(), v.float().numpy(), pos, start, ln, c.table)
    c.check_cache()
    clean = PagedOracle(2, dim, c.n_pages, 16, c.axis_dims)
    for name in "kv":
        clean.codes[name] = np.where(c.oracle.codes[name] == 0x7F, 0, c.oracle.codes[name]).astype(np.uint8)
        clean.scales[name] = c.oracle.scales[name]
    q = c.draw(c.n, c.q_heads)
    start, ln, pos = c.batch(seqs)
    for window in (20, 8990 if max(c.len) > 9000 else 33):
        out = c.kv.attend(q.cuda(), cu(pos), cu(start), cu(ln), cu(c.table), window=window).cpu()
        want, spread, logit = clean.attend(q.float().numpy(), pos, start, ln, c.table, True, window)
        for b, (n, before) in enumerate(seqs):
            for i in range(n):
                at, row = before + i, start[b] + i
                sees = lambda j: at - window < j <= at
                for h in range(4):
                    vd = [j for s, j in nan_v if s == b and h < 2 and sees(j)] + ([3] if h >= 2 and sees(3) else [])
                    kd = [j for s, j in nan_k if s == b and h >= 2 and sees(j)]
                    got = out[row, h]
                    if kd:
                        assert bool(torch.isnan(got).all()), (b, i, h)
                    elif vd:
                        assert bool(torch.isnan(got[7 if h >= 2 else 5])), (b, i, h)
                    else:
                        one, c.n = c.n, 1
                        c.check_out(got[None, None], want[row:row + 1, h:h + 1], spread[row:row + 1, h:h + 1],
                                    logit[row:row + 1, h:h + 1])
                        c.n = one
    # a NaN query
    q[0, 1, 3] = float("nan")
    out = c.kv.attend(q.cuda(), cu(pos), cu(start), cu(ln), cu(c.table), window=20).cpu()
    assert bool(torch.isnan(out[0, 1]).all()) and not bool(torch.isnan(out[0, 0]).any())
    assert c.kv.debug_state() == 0


def test_rows_that_see_nothing_are_zero():
    c = Case([(4, 0), (40, 0), (2, 30)], group=4)
    c.fill(1)
    # causal, with more queries than cached tokens: the first ones see nothing
    start = np.array([0, 4, 44, 46], np.int32)
    ln = np.array([2, 13, 0], np.int32)
    pos = np.zeros((46, 1), np.int32)
    q = c.draw(46, c.q_heads)
    for causal in (True, False):
        out = c.kv.attend(q.cuda(), cu(pos), cu(start), cu(ln), cu(c.table), causal=causal)
        want, spread, logit = c.oracle.attend(q.float().numpy(), pos, start, ln, c.table, causal)
        c.n = 46
        c.check_out(out, want, spread, logit)
        assert bool((out[44:] == 0).all())                  # an empty cache
        if causal:
            assert bool((out[:2] == 0).all()) and bool((out[4:31] == 0).all())
    assert c.kv.debug_state() == 0


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_pages_of_very_different_size(dtype, n):
    """Zero pages, tiny and huge ones side by side: each page's scale is an
    offset of the weights' exponents."""
    c = Case([(n, 700), (n, 64)], group=4, page=16, dtype=dtype)
    g = np.random.default_rng(5)
    total = sum(c.len)
    k, v = c.draw(total, c.kv_heads), c.draw(total, c.kv_heads).float()
    start, ln, pos = c.batch([(m, 0) for m in c.len])
    size = np.concatenate([np.repeat(np.exp2(g.integers(-8, 9, m // 16 + 1)), 16)[:m] for m in c.len])
    v = v * torch.from_numpy(size.astype(np.float32))[:, None, None]
    v[32:200] = 0                                            # pages of zeros among the first
    v[start[1]:start[1] + 48] = 0                            # and in front
    k[64:96] = 0
    k, v = k.to(dtype), v.to(dtype)
    c.kv.append(k.cuda(), v.cuda(), cu(pos), cu(start), cu(ln), cu(c.table))
    c.oracle.append(k.float().numpy(), v.float().numpy(), pos, start, ln, c.table)
    c.check_cache()
    c.attend()
    c.attend(window=100)


def test_block_scale_limits():
    """Blocks below 2^-100 are zero blocks; values near the type's end, which
    the rotation may carry to infinity; a scale that grows re-rounds the older
    codes only."""
    c = Case([(1, 3), (2, 0), (1, 63), (1, 0)], kv_heads=2, group=1, page=64)
    start, ln, pos = c.batch([(n, 0) for n in c.len])
    k = c.draw(int(start[-1]), 2).float()
    k[start[0]:start[1]] *= 2.0 ** -110
    k[start[1]:start[2]] = 3e38
    k[start[2]:start[3]] *= torch.from_numpy(np.exp2(np.arange(64) - 30).astype(np.float32))[:, None, None]
    k[start[3]:] = 0
    k = k.to(BF)
    for cut in (0, 40):
        seqs = [(n if not cut or n < 64 else cut, 0) for n in c.len]
        s2, l2, p2 = c.batch(seqs)
        idx = np.concatenate([np.arange(start[b], start[b] + n) for b, (n, _) in enumerate(seqs)])
        c.kv.append(k[idx].cuda(), k[idx].cuda(), cu(p2), cu(s2), cu(l2), cu(c.table))
        c.oracle.append(k[idx].float().numpy(), k[idx].float().numpy(), p2, s2, l2, c.table)
        c.check_cache()
    # the third sequence's other tokens, each larger than the last: the scale grows at every call
    for i in range(40, 64):
        one = [(0, 4), (0, 2), (1, i), (0, 1)]
        s2, l2, p2 = c.batch(one)
        row = k[start[2] + i:start[2] + i + 1]
        c.kv.append(row.cuda(), row.cuda(), cu(p2), cu(s2), cu(l2), cu(c.table))
        c.oracle.append(row.float().numpy(), row.float().numpy(), p2, s2, l2, c.table)
    c.check_cache()
    assert c.kv.debug_state() == 0


# ---------------------------------------------------------------- layouts
def test_slices_strides_layers_and_shared_pages():
    c = Case([(5, 60), (1, 130), (70, 3)], kv_heads=2, group=3, layers=3, extra_rows=4)
    c.fill(1)
    h, qh, d = 2, 6, 128
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn((c.rows, qh + 2 * h + 1, d), generator=g).to(BF)
    start, ln, pos = c.batch(c.seqs)
    pos = np.concatenate([pos, np.zeros((4, 1), np.int32)])
    # the rows that follow the last sequence hold anything, a wide table has other columns beside it
    qkv[c.n:] = float("nan")
    dev = qkv.cuda()
    wide = torch.full((3, c.table.shape[1] + 5), -3, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + c.table.shape[1]] = cu(c.table)
    table = wide[:, 2:2 + c.table.shape[1]]
    before = [c.kv.k_codes[layer].clone() for layer in (0, 2)]
    filled = c.kv.k_codes[0].clone(), c.kv.v_codes[0].clone(), c.kv.k_scales[0].clone(), c.kv.v_scales[0].clone()
    c.kv.k_codes[1].copy_(filled[0]), c.kv.v_codes[1].copy_(filled[1])
    c.kv.k_scales[1].copy_(filled[2]), c.kv.v_scales[1].copy_(filled[3])
    c.kv.append(dev[:, qh:qh + h], dev[:, qh + h:qh + 2 * h], cu(pos), cu(start), cu(ln), table, layer=1)
    c.oracle.append(qkv[:c.n, qh:qh + h].float().numpy(), qkv[:c.n, qh + h:qh + 2 * h].float().numpy(), pos[:c.n], start, ln,
                    c.table)
    c.check_cache(layer=1)
    assert bool((c.kv.k_codes[0] == before[0]).all()) and bool((c.kv.k_codes[2] == before[1]).all())
    out = torch.full((c.rows, qh + 2, d), 5.0, dtype=BF, device="cuda")
    got = c.kv.attend(dev[:, :qh], cu(pos), cu(start), cu(ln), table, out=out[:, 1:1 + qh], layer=1)
    assert got.data_ptr() == out[:, 1:].data_ptr()
    c.check_out(out[:, 1:1 + qh], *c.oracle.attend(qkv[:c.n, :qh].float().numpy(), pos[:c.n], start, ln, c.table))
    assert bool((out[:, 0] == 5).all()) and bool((out[:, qh + 1] == 5).all()) and bool((out[c.n:] == 5).all())
    assert c.kv.debug_state() == 0


def test_sequences_that_share_a_prefix():
    c = Case([(1, 200), (30, 140)], kv_heads=2, group=4, page=32)
    c.fill(1)
    c.table[1, :4] = c.table[0, :4]                          # 128 tokens read by both
    c.attend()


def test_one_token_at_a_time():
    """A prompt, then single tokens, append and attend in turn, three sequences
    that start and end at different times."""
    c = Case([(0, 90), (0, 70), (0, 33)], kv_heads=2, group=4, page=32)
    have = [0, 0, 0]
    joins, first = [0, 3, 9], [50, 64, 1]
    for step in range(30):
        seqs = []
        for b in range(3):
            new = 0 if step < joins[b] else first[b] if step == joins[b] else 1
            new = min(new, c.len[b] - have[b])
            seqs.append((new, have[b]))
            have[b] += new
        n = sum(a for a, _ in seqs)
        if n == 0:
            continue
        c.append(seqs)
        c.seqs, c.n, c.rows = seqs, n, n
        c.attend(max_new=max(a for a, _ in seqs) if step % 2 else None)
    c.check_cache()
    assert c.kv.debug_state() == 0


# ---------------------------------------------------------------- streams and graphs
def test_captured_calls_follow_the_lengths():
    """One graph of append and attend for a decoding batch, replayed while the
    host moves the lengths, the table and the inputs on; a second graph of the
    same cache in between."""
    steps = 70
    c = Case([(0, 40 + steps), (0, 3 + steps), (0, 200 + steps)], kv_heads=2, group=4, page=64)
    have = [40, 3, 200]
    c.append([(n, 0) for n in have])
    start, ln, pos = c.batch([(1, n) for n in have])
    k, v, q = (torch.zeros((3, h, 128), dtype=BF, device="cuda") for h in (2, 2, 8))
    ln_d, pos_d, start_d, table = cu(ln), cu(pos), cu(start), cu(c.table)
    out = torch.zeros((3, 8, 128), dtype=BF, device="cuda")
    out2 = torch.zeros_like(out)

    def work(o, **kw):
        c.kv.append(k, v, pos_d, start_d, ln_d, table)
        c.kv.attend(q, pos_d, start_d, ln_d, table, out=o, **kw)

    graphs = []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for o, kw in ((out, dict(max_new=1)), (out2, dict(window=20))):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=side):
                work(o, **kw)
            graphs.append(gr)
    torch.cuda.synchronize()
    for step in range(steps):
        kk, vv, qq = c.draw(3, 2), c.draw(3, 2), c.draw(3, 8)
        start, ln, pos = c.batch([(1, n) for n in have])
        for d, h in ((k, kk), (v, vv), (q, qq), (ln_d, torch.from_numpy(ln)), (pos_d, torch.from_numpy(pos))):
            d.copy_(h)
        graphs[0].replay()
        graphs[1].replay()
        c.oracle.append(kk.float().numpy(), vv.float().numpy(), pos, start, ln, c.table)
        if step % 23 == 0 or step == steps - 1:
            c.n = 3
            c.check_out(out, *c.oracle.attend(qq.float().numpy(), pos, start, ln, c.table))
            c.check_out(out2, *c.oracle.attend(qq.float().numpy(), pos, start, ln, c.table, True, 20))
        have = [n + 1 for n in have]
    c.check_cache()
    assert c.kv.debug_state() == 0


def test_another_stream():
    c = Case([(40, 100), (1, 500)], group=4)
    side = torch.cuda.Stream()
    start, ln, pos = c.batch([(n, 0) for n in c.len])
    k, v = c.draw(int(start[-1]), 2), c.draw(int(start[-1]), 2)
    args = [cu(x) for x in (pos, start, ln, c.table)]
    kd, vd = k.cuda(), v.cuda()
    side.wait_stream(torch.cuda.current_stream())
    c.kv.append(kd, vd, *args, stream=side)
    c.oracle.append(k.float().numpy(), v.float().numpy(), pos, start, ln, c.table)
    start, ln, pos = c.batch(c.seqs)
    q = c.draw(c.n, c.q_heads)
    qd, args = q.cuda(), [cu(x) for x in (pos, start, ln, c.table)]
    side.wait_stream(torch.cuda.current_stream())
    out = c.kv.attend(qd, *args, stream=side)
    raw = c.kv.attend(qd, *args, stream=side.cuda_stream)
    side.synchronize()
    c.check_out(out, *c.oracle.attend(q.float().numpy(), pos, start, ln, c.table))
    assert bool((out == raw).all())


def test_two_caches_at_once():
    """Calls on two handles may overlap: each has its own scratch."""
    pair = [Case([(60, 900), (1, 3000)], kv_heads=2, group=4, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in pair]
    for c in pair:
        c.fill(1)
    torch.cuda.synchronize()
    qs, outs, args = [], [], []
    for c in pair:
        start, ln, pos = c.batch(c.seqs)
        qs.append(c.draw(c.n, c.q_heads))
        args.append((pos, start, ln))
    dev = [(q.cuda(), *[cu(x) for x in a], cu(c.table)) for q, a, c in zip(qs, args, pair)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, c in enumerate(pair):
            out = c.kv.attend(*dev[i], stream=streams[i])
            if _ == 19:
                outs.append(out)
    torch.cuda.synchronize()
    for c, q, (pos, start, ln), out in zip(pair, qs, args, outs):
        c.check_out(out, *c.oracle.attend(q.float().numpy(), pos, start, ln, c.table))


@pytest.mark.parametrize("seqs", [[(2, 50), (300, 0), (1, 4000), (17, 9)], [(130, 10)] * 5, [(1, 100)] * 3])
def test_many_calls_in_a_row(seqs):
    """The kernels of consecutive calls overlap at their ends (dependent launch):
    the outputs are those of single calls."""
    c = Case(seqs, kv_heads=2, group=4, page=32)
    c.fill(1)
    start, ln, pos = c.batch(c.seqs)
    qs = [c.draw(c.n, c.q_heads).cuda() for _ in range(3)]
    args = [cu(x) for x in (pos, start, ln, c.table)]
    want = []
    for q in qs:
        want.append(c.kv.attend(q, *args).clone())
        torch.cuda.synchronize()
    outs = [c.kv.attend(qs[i % 3], *args) for i in range(60)]
    torch.cuda.synchronize()
    assert all(bool((o == want[i % 3]).all()) for i, o in enumerate(outs))
    assert c.kv.debug_state() == 0


# ---------------------------------------------------------------- refusals
def test_numbers_that_contradict_are_left_out():
    from fp8_ring_kv_gb300 import kvring as K
    c = Case([(3, 60), (5, 5), (40, 100), (2, 20)], group=4)
    c.fill(1)
    q = c.draw(c.n, c.q_heads)
    start, ln, pos = c.batch(c.seqs)
    good, spread, logit = c.oracle.attend(q.float().numpy(), pos, start, ln, c.table)
    codes = c.kv.k_codes.clone()

    def attend(start, ln, table=c.table, **kw):
        out = torch.full((c.n, c.q_heads, c.dim), 7.0, dtype=BF, device="cuda")
        c.kv.attend(q.cuda(), cu(pos), cu(start), cu(ln), cu(table), out=out, **kw)
        torch.cuda.synchronize()
        err = c.kv.debug_state()
        c.kv.workspace[:4].zero_()                           # the error word
        return out, err

    def same(out, rows):
        all_n, c.n = c.n, len(range(*rows))
        c.check_out(out[rows[0]:rows[1]], good[rows[0]:rows[1]], spread[rows[0]:rows[1]], logit[rows[0]:rows[1]])
        c.n = all_n

    for bad_len in (-1, c.table.shape[1] * c.page + 1, 2 ** 31 - 1):
        l2 = ln.copy()
        l2[1] = bad_len
        out, err = attend(start, l2)
        assert err == K.KVRING_DEVERR_SEQ
        assert bool((out[3:8] == 7).all())                   # left out
        same(out, (0, 3)), same(out, (8, c.n))
    for s1 in (-5, 2 ** 30, 60):                             # decreasing or past the rows
        s2 = start.copy()
        s2[1] = s1
        out, err = attend(s2, ln)
        assert err == K.KVRING_DEVERR_SEQ
        same(out, (8, c.n))
    out, err = attend(start, ln, max_new=5)                  # the third sequence has 40
    assert err == K.KVRING_DEVERR_SEQ and bool((out[8:48] == 7).all())
    same(out, (0, 8)), same(out, (48, c.n))
    # append: more new tokens than the sequence has with them
    k = c.draw(c.n, c.kv_heads).cuda()
    l2 = np.array([2, 4, 39, 1], np.int32)
    c.kv.append(k, k, cu(pos), cu(start), cu(l2), cu(c.table))
    assert c.kv.debug_state() == K.KVRING_DEVERR_SEQ
    assert bool((c.kv.k_codes == codes).all())
    c.kv.workspace[:4].zero_()
    # page ids outside the pool
    for pg in (-1, c.n_pages, 2 ** 31 - 1, -2 ** 31):
        t2 = c.table.copy()
        t2[2, 1] = pg
        out, err = attend(start, ln, t2)
        assert err == K.KVRING_DEVERR_PAGE
        assert bool(torch.isfinite(out.float()).all())
        same(out, (0, 8)), same(out, (48, c.n))
        t2 = np.where(c.table >= 0, pg, -1).astype(np.int32)
        c.kv.append(k, k, cu(pos), cu(start), cu(ln), cu(t2))
        assert c.kv.debug_state() == K.KVRING_DEVERR_PAGE
        assert bool((c.kv.k_codes == codes).all())
        c.kv.workspace[:4].zero_()
    # positions outside the table are clamped
    p2 = pos.copy()
    p2[0] = 10 ** 6
    p2[1] = -4
    c.kv.append(k, k, cu(p2), cu(start), cu(ln), cu(c.table))
    assert c.kv.debug_state() == K.KVRING_DEVERR_POS_RANGE


def test_host_refusals():
    from fp8_ring_kv_gb300 import kvring as K
    from fp8_ring_kv_gb300.kvring import KVRingError
    c = Case([(3, 60), (2, 5)], group=4, layers=2)
    c.fill(1)
    start, ln, pos = c.batch(c.seqs)
    q, k = c.draw(c.n, 8).cuda(), c.draw(c.n, 2).cuda()
    a = dict(pos=cu(pos), seq_start=cu(start), kv_len=cu(ln), page_table=cu(c.table))
    out = torch.empty_like(q)

    def bad(match, what="attend", **kw):
        args = dict(a, **kw)
        with pytest.raises(KVRingError, match=match):
            if what == "append":
                c.kv.append(args.pop("k", k), args.pop("v", k), **args)
            else:
                args["q_pos"] = args.pop("pos")
                c.kv.attend(args.pop("q", q), **args)

    for what in ("append", "attend"):
        bad("layer", what, layer=2)
        bad("layer", what, layer=-1)
        bad("int64", what, kv_len=cu(ln).long())
        bad("shape", what, kv_len=cu(ln)[:1])
        bad("shape", what, seq_start=cu(start)[:2])
        bad("shape", what, pos=cu(pos)[:2])
        bad("cpu", what, seq_start=torch.from_numpy(start))
        bad("shape", what, page_table=cu(c.table)[0])
        bad("strides", what, page_table=cu(c.table).t().contiguous().t().expand(2, -1) if c.table.shape[1] > 1
            else cu(np.zeros((4, 2), np.int32)).t()[:2])
        bad("more than", what, page_table=torch.zeros((2, 70000), dtype=torch.int32, device="cuda"))
    bad("float32", "append", k=k.float())
    bad("shape", "append", v=k[:, :1])
    bad("strides", "append", k=torch.zeros((c.n, 128, 2), dtype=BF, device="cuda").transpose(1, 2))
    bad("strides", "append", k=torch.zeros((c.n, 2 * 128 + 4), dtype=BF, device="cuda")[:, :256].unflatten(1, (2, 128)))
    bad("float16", q=q.half())
    bad("window", window=4, causal=False)
    bad("window", window=0)
    bad("scale", scale=-1.0)
    bad("scale", scale=float("inf"))
    bad("max_new", max_new=0)
    bad("max_new", max_new=c.n + 1)
    bad("shape", out=out[:2])
    bad("misaligned", q=torch.zeros(q.numel() + 4, dtype=BF, device="cuda")[4:].view_as(q))
    with pytest.raises(KVRingError, match="sequences"):
        many = torch.zeros((2049, 1), dtype=torch.int32, device="cuda")
        c.kv.append(k, k, a["pos"], torch.zeros(2050, dtype=torch.int32, device="cuda"), many[:, 0].contiguous(), many)
    lib, h, p = K.load(), c.kv.handle, q.data_ptr()
    good = [h, 0, p, 1024, p, 5, p, 2, c.n, c.n, p, 4, 2, 1, 0, 0.0, p, 1024, None]
    names = "h layer q q_stride q_pos start len n_seqs n_tokens max_new table t_stride width causal window scale out o_stride st"
    base = dict(zip(names.split(), [h, 0, p, 1024, p, p, p, 2, c.n, c.n, p, 4, 2, 1, 0, 0.0, p, 1024, None]))
    del good
    for key, value, status in (("layer", 2, -1), ("q", None, -1), ("q_stride", 1016, -1), ("q_stride", 1028, -1),
                               ("q", p + 8, -2), ("start", None, -1), ("start", p + 2, -2), ("n_seqs", -1, -1),
                               ("n_seqs", 2049, -1), ("n_tokens", -1, -1), ("max_new", 0, -1), ("max_new", c.n + 1, -1),
                               ("width", 0, -1), ("t_stride", 1, -1), ("width", 1 << 20, -1), ("causal", 2, -1),
                               ("window", -1, -1), ("scale", -1.0, -1), ("scale", float("nan"), -1), ("out", p + 4, -2),
                               ("o_stride", 8, -1)):
        assert lib.kvring_paged_attend(*dict(base, **{key: value}).values()) == status, (key, value)
    # nothing to do is fine
    empty = q[:0]
    r = c.kv.attend(empty, a["pos"][:0], a["seq_start"] * 0, a["kv_len"], a["page_table"])
    assert r.shape == (0, 8, 128)
    c.kv.append(k[:0], k[:0], a["pos"][:0], a["seq_start"] * 0, a["kv_len"], a["page_table"])
    assert c.kv.debug_state() == 0
    c.check_cache()
    c.kv.close()
    with pytest.raises(KVRingError, match="closed"):
        c.kv.append(k, k, **a)


def test_append_leaves_out_only_the_contradicting_sequence():
    from fp8_ring_kv_gb300 import kvring as K
    c = Case([(3, 60), (5, 5), (40, 100), (2, 20)], kv_heads=1)
    start, ln, pos = c.batch(c.seqs)
    k, v = c.draw(c.n, 1), c.draw(c.n, 1)
    for bad in (2 ** 31 - 1, 2 ** 30, -2 ** 31, -1):         # the end of sequence 0, the start of sequence 1
        s2 = start.copy()
        s2[1] = bad
        c.kv.append(k.cuda(), v.cuda(), cu(pos), cu(s2), cu(ln), cu(c.table))
        assert c.kv.debug_state() == K.KVRING_DEVERR_SEQ
        c.kv.workspace[:4].zero_()
    rest = start[2:] - start[2]
    at = start[2]
    c.oracle.append(k[at:].float().numpy(), v[at:].float().numpy(), pos[at:], rest, ln[2:], c.table[2:])
    c.check_cache()
    # one that counts more new tokens than it has, beside whole ones
    l2 = ln.copy()
    l2[2] = 39
    c.kv.append(k.cuda(), v.cuda(), cu(pos), cu(start), cu(l2), cu(c.table))
    assert c.kv.debug_state() == K.KVRING_DEVERR_SEQ
    c.oracle.append(k[:8].float().numpy(), v[:8].float().numpy(), pos[:8], start[:3], ln[:2], c.table[:2])
    c.oracle.append(k[48:].float().numpy(), v[48:].float().numpy(), pos[48:], [0, 2], ln[3:], c.table[3:])
    c.check_cache()


def test_a_window_wider_than_everything():
    c = Case([(4, 0), (40, 0), (3, 30)], group=4)
    c.fill(1)
    q = c.draw(c.n, c.q_heads).cuda()
    start, ln, pos = c.batch(c.seqs)
    for ln in (ln, np.array([2, 13, 33], np.int32)):         # also with queries that see nothing
        args = [cu(x) for x in (pos, start, ln, c.table)]
        want = c.kv.attend(q, *args)
        for window in (64, 2 ** 22, 2 ** 31 - 1, 2 ** 40):
            assert bool((c.kv.attend(q, *args, window=window) == want).all()), window


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("case,how", [
    (dict(seqs=[(1, 900), (2, 300), (3, 5000), (4, 40), (5, 700), (4, 0)], group=8), {}),
    (dict(seqs=[(3, 5000), (4, 900), (2, 33)], group=8, page=16, dim=64), dict(window=130)),
    (dict(seqs=[(1, 2000), (1, 3), (2, 70)], kv_heads=1, group=16), dict(max_new=2)),
    (dict(seqs=[(31, 2), (32, 500), (33, 500), (9, 100), (17, 100), (25, 1000)], group=1, page=32), {}),
    (dict(seqs=[(31, 2), (32, 500), (8, 100), (16, 100), (24, 3000)], group=1, dim=64, page=128), dict(causal=False)),
    (dict(seqs=[(3, 600), (1, 10)], kv_heads=3, group=11), dict(max_new=3)),
], ids=range(6))
def test_several_row_tiles_of_a_few_tokens(case, how, dtype):
    """Sequences whose query rows fill one to four of the register tiles, or one more."""
    c = Case(dtype=dtype, **case)
    c.fill(2)
    c.attend(**how)
    assert c.kv.debug_state() == 0


@pytest.mark.parametrize("dtype,n,dim,page", [(BF, 1, 64, 128), (HF, 3, 128, 64), (BF, 50, 128, 64), (HF, 40, 64, 128)])
def test_the_longest_sequence(dtype, n, dim, page):
    """2^22 tokens whose table names the same few pages again and again: the
    attention over those pages once."""
    c = Case([(0, 4 * page)], kv_heads=1, group=2, dim=dim, page=page, dtype=dtype)
    c.fill(1)
    times = 2 ** 22 // (4 * page)
    table = np.tile(c.table[:, :4], (1, times))
    q = c.draw(n, 2)
    pos = np.zeros((n, 1), np.int32)
    start = np.array([0, n], np.int32)
    # not causal: every query sees every page equally often
    out = c.kv.attend(q.cuda(), cu(pos), cu(start), cu(np.array([2 ** 22], np.int32)), cu(table), causal=False)
    c.n = n
    c.check_out(out, *c.oracle.attend(q.float().numpy(), pos, start, [4 * page], c.table, False))
    # a window that reaches back over whole rounds of the pages
    if n == 1:
        out = c.kv.attend(q.cuda(), cu(pos), cu(start), cu(np.array([2 ** 22], np.int32)), cu(table), window=4 * page * 1000)
        c.check_out(out, *c.oracle.attend(q.float().numpy(), pos, start, [4 * page], c.table, False))
    assert c.kv.debug_state() == 0


def test_many_sequences_of_both_kinds():
    """2,048 sequences, some without new tokens, some with prompts' worth of rows."""
    seqs = [(0 if i % 5 == 3 else 300 if i % 401 == 7 else 40 if i % 97 == 0 else 1 + i % 2, i % 50) for i in range(2048)]
    c = Case(seqs, kv_heads=1, group=3, dim=64, page=32)
    c.fill(2)
    c.check_cache()
    c.attend()
    c.attend(window=9)
    assert c.kv.debug_state() == 0


def test_rows_are_32_bit_numbers():
    from fp8_ring_kv_gb300 import kvring as K
    kv = paged(1, 1024, 64, 2, 16, (64,), (0,), (8,))
    p = kv.workspace.data_ptr()                              # never read: the call is refused
    args = [kv.handle, 0, p, 65536, p, p, p, 1, 1 << 21, 1, p, 2, 2, 1, 0, 0.0, p, 65536, None]
    assert K.load().kvring_paged_attend(*args) == K.KVRING_ERR_INVALID_ARG
    args[8] = (1 << 24) + 1
    assert K.load().kvring_paged_attend(*args) == K.KVRING_ERR_INVALID_ARG
    assert kv.debug_state() == 0


def test_a_captured_fork_and_join():
    """The append on a second stream of the capture, the attention after both;
    memory copies in front, so that edges of either kind meet."""
    c = Case([(1, 300), (40, 64), (3, 10)], group=4)
    c.append([(0, 0)] * 3)                                   # nothing
    c.append([(b, 0) for _, b in c.seqs])
    start, ln, pos = c.batch(c.seqs)
    k, v, q = c.draw(c.n, 2), c.draw(c.n, 2), c.draw(c.n, 8)
    args = [cu(x) for x in (pos, start, ln, c.table)]
    src = [t.cuda() for t in (k, v, q)]
    kd, vd, qd = (torch.zeros_like(t) for t in src)
    out = torch.full_like(qd, 7.0)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=one):
        kd.copy_(src[0]), vd.copy_(src[1])
        two.wait_stream(one)
        with torch.cuda.stream(two):
            c.kv.append(kd, vd, *args)
        qd.copy_(src[2])
        one.wait_stream(two)
        c.kv.attend(qd, *args, out=out)
    c.oracle.append(k.float().numpy(), v.float().numpy(), pos, start, ln, c.table)
    for _ in range(3):
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        c.check_cache()
        c.check_out(out, *c.oracle.attend(q.float().numpy(), pos, start, ln, c.table))
    assert c.kv.debug_state() == 0
