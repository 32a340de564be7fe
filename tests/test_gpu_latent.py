"""The latent cache on the GPU against its numpy oracle: appended codes and scales
and read rows bit for bit, the attention of both forms within bounds derived
from its roundings, over types, sizes, page sizes, ragged lengths, masks,
strides, streams and graphs."""
import numpy as np
import pytest
import torch

import latent_bounds
from oracle.latent import ROPE, LatentOracle, attend_expanded

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
KIND = {BF: "bf16", HF: "f16"}
SCALE = 192 ** -0.5


def cu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def num(t):
    return t.float().numpy()


class Case:
    """A cache with its oracle, and one batch of sequences (new, before)."""

    def __init__(self, seqs, heads=4, latent=256, page=64, axes=1, dtype=BF, seed=0, extra_rows=0, width=None, layers=1, big=1.0):
        from fp8_ring_kv_gb300 import LatentKV
        self.seqs, self.heads, self.C, self.page, self.dtype, self.big = seqs, heads, latent, page, dtype, big
        self.axis_dims = (ROPE,) if axes == 1 else (16, 24, 24)
        self.g = np.random.default_rng(seed)
        self.new, self.len = [a for a, _ in seqs], [a + c for a, c in seqs]
        held = [(n + page - 1) // page for n in self.len]
        self.n_pages = sum(held) + 2
        order = self.g.permutation(self.n_pages)
        self.table = np.full((len(seqs), width or max(1, max(held))), -1, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.n = sum(self.new)
        self.rows = self.n + extra_rows
        top = max([1] + self.len) + 1
        self.kv = LatentKV(heads, latent, self.n_pages, page, self.axis_dims, (0,) * axes,
                           (top,) if axes == 1 else (top // 12 + 1, 3, 4), dtype=dtype, layers=layers)
        self.oracle = LatentOracle(latent, self.n_pages, page, self.axis_dims)

    def draw(self, *shape):
        """Numbers in the cache's type, a few channels louder."""
        x = self.g.standard_normal(shape).astype(np.float32) * np.float32(self.big)
        x[..., ::37] *= 4
        return torch.from_numpy(x).to(self.dtype)

    def positions(self, index):
        index = np.maximum(np.asarray(index), 0)
        if len(self.axis_dims) == 1:
            return index[:, None].astype(np.int32)
        return np.stack([index // 12, index // 4 % 3, index % 4], 1).astype(np.int32)

    def batch(self, seqs):
        start = np.concatenate([[0], np.cumsum([a for a, _ in seqs])]).astype(np.int32)
        ln = np.array([a + c for a, c in seqs], np.int32)
        index = np.concatenate([np.arange(c, c + a) for a, c in seqs] + [np.zeros(0, int)])
        return start, ln, self.positions(index)

    def append(self, seqs, latent=None, rope=None, layer=0):
        start, ln, pos = self.batch(seqs)
        n = int(start[-1])
        x = self.draw(n, self.C) if latent is None else latent
        r = self.draw(n, ROPE) if rope is None else rope
        self.kv.append(x.cuda(), r.cuda(), cu(pos), cu(start), cu(ln), cu(self.table), layer=layer)
        self.oracle.append(num(x), num(r), pos, start, ln, self.table)

    def fill(self, pieces=1):
        cuts = [[n * i // pieces for n in self.len] for i in range(pieces + 1)]
        for lo, hi in zip(cuts, cuts[1:]):
            self.append([(b - a, a) for a, b in zip(lo, hi)])

    def check_cache(self, layer=0):
        torch.cuda.synchronize()
        codes, scales = self.kv.codes[layer].cpu().numpy(), self.kv.scales[layer].cpu().numpy()
        assert np.array_equal(np.isnan(scales), np.isnan(self.oracle.scales))
        assert np.array_equal(np.nan_to_num(scales, nan=-1), np.nan_to_num(self.oracle.scales, nan=-1))
        bad = np.argwhere(codes != self.oracle.codes)
        assert bad.size == 0, f"{len(bad)} codes differ, first {bad[:4].tolist()}"

    def attend(self, causal=True, window=None, scale=SCALE, max_new=None, q=None, qr=None):
        q = self.draw(self.rows, self.heads, self.C) * 0.5 if q is None else q
        qr = self.draw(self.rows, self.heads, ROPE) if qr is None else qr
        start, ln, pos = self.batch(self.seqs)
        pos = np.concatenate([pos, np.zeros((self.rows - self.n, pos.shape[1]), np.int32)])
        out = torch.full((self.rows, self.heads, self.C), 7.0, dtype=self.dtype, device="cuda")
        got = self.kv.attend(q.cuda(), qr.cuda(), cu(pos), cu(start), cu(ln), cu(self.table), scale, out=out, causal=causal,
                             window=window, max_new=max_new)
        assert got is out
        r = self.oracle.attend(num(q[:self.n]), num(qr[:self.n]), pos[:self.n], start, ln, self.table, scale, causal, window or 0)
        check(out[:self.n], r, latent_bounds.absorbed(r, KIND[self.dtype]))
        rms = float(np.sqrt(np.mean((out[:self.n].double().cpu().numpy() - r.out) ** 2))) if self.n else 0.0
        assert rms <= latent_bounds.absorbed_rms(r, KIND[self.dtype]) if self.n else True
        assert bool((out[self.n:] == 7.0).all())             # rows past the last sequence stay as they were
        return out


def check(out, r, bound):
    err = np.abs(out.double().cpu().numpy() - r.out)
    worst = float((err / bound).max()) if err.size else 0.0
    assert bool(np.isfinite(err).all()) and worst <= 1.0, f"error {err.max():.3e}, {worst:.2f} of its bound"


APPENDS = [
    dict(seqs=[(1, 0)], latent=512),
    dict(seqs=[(1, 63), (1, 64), (1, 65), (5, 0)], page=64),
    dict(seqs=[(200, 0), (3, 77), (0, 40), (129, 15)], page=16, latent=128, dtype=HF),
    dict(seqs=[(131, 130), (64, 64), (2, 31)], page=32, axes=3, latent=384),
    dict(seqs=[(300, 1), (128, 128), (127, 1), (1, 127)], page=128, latent=512, dtype=HF),
    dict(seqs=[(i % 3, i) for i in range(150)], page=16, latent=128),
    # more rows than go one to a warp; sequences without tokens between them
    dict(seqs=[(700, 0), (0, 5), (1, 3000), (2, 0)] + [(0, 0)] * 40 + [(1, i) for i in range(43)], page=16, latent=256),
    dict(seqs=[(2999, 4), (1, 6), (0, 0), (3, 1)], page=128, latent=512, axes=3, dtype=HF),
]


@pytest.mark.parametrize("pieces", [1, 3])
@pytest.mark.parametrize("case", APPENDS, ids=range(len(APPENDS)))
def test_append_and_read_bit_for_bit(case, pieces):
    c = Case(**case)
    c.fill(pieces)
    c.check_cache()
    # all rows, and the last ones of each sequence
    for new in (c.len, c.new):
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        ln = np.array(c.len, np.int32)
        want = torch.from_numpy(c.oracle.read(start, ln, c.table)).to(c.dtype)
        got = c.kv.read(cu(start), cu(ln), cu(c.table), int(start[-1]))
        assert bool((got.cpu() == want).all())
        out = torch.full((int(start[-1]) + 3, c.C + ROPE + 8), 7.0, dtype=c.dtype, device="cuda")
        c.kv.read(cu(start), cu(ln), cu(c.table), out=out[:, :c.C + ROPE])
        assert bool((out[:int(start[-1]), :c.C + ROPE].cpu() == want).all())
        assert bool((out[int(start[-1]):] == 7).all()) and bool((out[:, c.C + ROPE:] == 7).all())
    assert c.kv.debug_state() == 0


def test_bad_pages_and_lengths_among_many_rows():
    """Rows of several sequences in one warp, some of them nowhere."""
    from fp8_ring_kv_gb300 import kvring as K
    c = Case([(3, 0)] * 900 + [(0, 0)] * 5 + [(50, 0)] * 6, latent=128, page=16)
    start, ln, pos = c.batch(c.seqs)
    x, r = c.draw(c.n, 128), c.draw(c.n, ROPE)
    x[2500, 3] = float("nan")
    table, bad_len = c.table.copy(), ln.copy()
    table[7, 0], table[300, 0], table[907, 1] = -1, c.n_pages, 2 ** 31 - 1
    bad_len[5], bad_len[899] = 2, -1                       # fewer than the new tokens
    lost = np.zeros(c.n, bool)
    for b in (5, 7, 300, 899):
        lost[start[b]:start[b + 1]] = True
    lost[start[907] + 16:start[907] + 32] = True
    keep = [b for b in range(len(ln)) if b not in (5, 7, 300, 899)]
    c.kv.append(x.cuda(), r.cuda(), cu(pos), cu(start), cu(bad_len), cu(table))
    assert c.kv.debug_state() == K.KVRING_DEVERR_SEQ | K.KVRING_DEVERR_PAGE
    c.oracle.append(num(x), num(r), pos, start, ln, c.table)
    want = torch.from_numpy(c.oracle.read(start, ln, c.table)).to(c.dtype)
    for b in (5, 7, 300, 899):
        c.oracle.codes[c.table[b, 0]], c.oracle.scales[c.table[b, 0]] = 0, 0
    c.oracle.codes[c.table[907, 1]], c.oracle.scales[c.table[907, 1]] = 0, 0
    c.check_cache()
    out = torch.full((c.n + 2, c.C + ROPE), 7.0, dtype=c.dtype, device="cuda")
    c.kv.read(cu(start), cu(bad_len), cu(table), out=out)
    out = out.cpu()
    assert bool((out[c.n:] == 7).all()) and bool((out[:c.n][lost] == 7).all()) and len(keep) == 907
    good = out[:c.n][~lost]
    assert bool(torch.isnan(out[2500]).all()) and bool(((good == want[~lost]) | torch.isnan(want[~lost])).all())


def test_sizes_of_rows():
    """Tiny, huge and zero rows; rows that are no numbers are marked, alone."""
    c = Case([(40, 0), (24, 0)], latent=128, page=16)
    x, r = c.draw(64, 128).float(), c.draw(64, ROPE).float()
    size = np.exp2(np.arange(64) * 1.5 - 48).astype(np.float32)
    x, r = x * torch.from_numpy(size)[:, None], r * torch.from_numpy(size)[:, None]
    x[5], r[5] = 0, 0
    x[7, 3], r[9, 1], x[11, 0], r[41, 63] = float("nan"), float("inf"), 3e38, float("-inf")
    c.append([(40, 0), (24, 0)], x.to(BF), r.to(BF))
    c.check_cache()
    marked = np.isnan(c.oracle.scales).sum()
    assert marked >= 4 and c.kv.debug_state() == 0
    rows = c.kv.read(cu(np.array([0, 40, 64], np.int32)), cu(np.array([40, 24], np.int32)), cu(c.table), 64)
    assert bool(torch.isnan(rows[7]).all()) and not bool(torch.isnan(rows[8]).any())


ATTENDS = [
    (dict(seqs=[(1, 0)], latent=512), {}),
    (dict(seqs=[(1, 776)], heads=32, latent=512), {}),
    (dict(seqs=[(1, 5), (1, 0), (1, 63), (1, 64), (1, 127), (1, 128), (1, 1500), (1, 31)], heads=20), {}),
    (dict(seqs=[(1, 300)] * 40, heads=1, latent=128, page=16, dtype=HF), {}),
    (dict(seqs=[(3, 100), (1, 7), (0, 9), (5, 0)], heads=3, page=32, latent=384), {}),
    (dict(seqs=[(1, 130), (1, 500)], heads=128, latent=512, page=128), {}),
    (dict(seqs=[(2, 900), (16, 200)], heads=8, page=128, dtype=HF), dict(window=100)),
    (dict(seqs=[(70, 0), (1, 400), (33, 65)], heads=2, page=16), dict(window=33)),
    (dict(seqs=[(2, 300)], heads=33, latent=128, dtype=HF), dict(window=1)),
    (dict(seqs=[(60, 11)], heads=5, latent=512, axes=3), dict(causal=False)),
    (dict(seqs=[(129, 0), (128, 0), (1, 0)], heads=1, page=128, latent=128), {}),
    (dict(seqs=[(9, 0), (1, 250)], heads=16, latent=384), dict(scale=0.3)),
    (dict(seqs=[(40, 300)], heads=7, page=32, dtype=HF, latent=512, axes=3), {}),
    (dict(seqs=[(30, 200)], heads=12, big=6.0), {}),
    (dict(seqs=[(1, 9000)], heads=40, latent=512), {}),
    (dict(seqs=[(1, 200)], heads=256, latent=128), {}),
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


@pytest.mark.parametrize("case,how", [
    (dict(seqs=[(1, 30000)], heads=16, latent=256, page=128), {}),                 # one item over the whole GPU
    (dict(seqs=[(1, 20000), (2, 10)], heads=64, latent=128, page=16, dtype=HF), dict(window=9000)),
    (dict(seqs=[(3, 17), (30, 1), (1, 4000), (64, 64), (2, 0), (50, 2000), (1, 1)], heads=4), {}),
], ids=range(3))
def test_split_items_give_the_same_bits(case, how):
    c = Case(**case)
    c.fill(3)
    c.attend(**how)
    q, qr = c.draw(c.rows, c.heads, c.C) * 0.5, c.draw(c.rows, c.heads, ROPE)
    a = [c.attend(q=q, qr=qr, **how).clone() for _ in range(3)]
    assert bool((a[0] == a[1]).all()) and bool((a[0] == a[2]).all())
    assert c.kv.debug_state() == 0


def test_many_sequences():
    seqs = [(0 if i % 5 == 3 else 40 if i % 97 == 0 else 1 + i % 2, i % 50) for i in range(2048)]
    c = Case(seqs, heads=3, latent=128, page=16)
    c.fill(2)
    c.check_cache()
    c.attend(window=9)
    assert c.kv.debug_state() == 0


@pytest.mark.parametrize("dtype,n,heads", [(BF, 1, 40), (HF, 3, 2)])
def test_the_longest_sequence(dtype, n, heads):
    """2^22 tokens whose table names the same few pages again and again: the
    attention over those pages once."""
    c = Case([(0, 512)], heads=heads, latent=128, page=128, dtype=dtype)
    c.fill(1)
    table = np.tile(c.table[:, :4], (1, 2 ** 22 // 512))
    q, qr = c.draw(n, heads, 128), c.draw(n, heads, ROPE)
    pos, start = np.zeros((n, 1), np.int32), np.array([0, n], np.int32)
    out = c.kv.attend(q.cuda(), qr.cuda(), cu(pos), cu(start), cu(np.array([2 ** 22], np.int32)), cu(table), SCALE, causal=False)
    r = c.oracle.attend(num(q), num(qr), pos, start, [512], c.table, SCALE, False)
    r.floor *= 2 ** 22 / 512                                 # as many keys
    check(out, r, latent_bounds.absorbed(r, KIND[dtype]))
    assert c.kv.debug_state() == 0


def test_offsets_past_32_bits():
    """Pages whose codes lie more than 2^32 bytes into the pool."""
    from fp8_ring_kv_gb300 import LatentKV
    c = Case([(3, 200), (20, 100)], heads=8, latent=512, page=128)
    pages = 60000                                            # x 73,728 bytes
    c.kv = LatentKV(8, 512, pages, 128, (ROPE,), (0,), (400,))
    small = c.table.copy()
    c.table = np.where(small >= 0, pages - 1 - small, -1).astype(np.int32)
    assert int(c.table[c.table >= 0].min()) * 128 * 576 > 2 ** 32
    start, ln, pos = c.batch([(n, 0) for n in c.len])
    x, r = c.draw(int(start[-1]), 512), c.draw(int(start[-1]), ROPE)
    c.kv.append(x.cuda(), r.cuda(), cu(pos), cu(start), cu(ln), cu(c.table))
    c.oracle.append(num(x), num(r), pos, start, ln, small)
    assert np.array_equal(c.kv.codes[0][pages - c.n_pages:].flip(0).cpu().numpy(), c.oracle.codes)
    got = c.kv.read(cu(start), cu(ln), cu(c.table), int(start[-1]))
    assert bool((got.cpu() == torch.from_numpy(c.oracle.read(start, ln, small)).to(BF)).all())
    start, ln, pos = c.batch(c.seqs)
    q, qr = c.draw(c.n, 8, 512), c.draw(c.n, 8, ROPE)
    out = c.kv.attend(q.cuda(), qr.cuda(), cu(pos), cu(start), cu(ln), cu(c.table), SCALE)
    res = c.oracle.attend(num(q), num(qr), pos, start, ln, small, SCALE)
    check(out, res, latent_bounds.absorbed(res, "bf16"))


# ---------------------------------------------------------------- masks and what lies behind them
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("latent,page", [(128, 16), (512, 64), (256, 128)])
def test_stale_pages_stay_behind_the_mask(latent, page, dtype):
    """A pool full of NaN codes and non-finite scales, as freed pages may be:
    what no query sees never reaches an output, and pages that a window has
    left behind need not be in the table."""
    for window in (None, 70):
        c = Case([(1, 100), (50, 75), (3, 200), (1, page - 1)], heads=6, latent=latent, page=page, dtype=dtype)
        c.kv.codes.fill_(0x7F)
        c.kv.scales.fill_(float("nan"))
        c.fill(2)
        if window:
            for b, (n, before) in enumerate(c.seqs):
                c.table[b, :max(0, before + 1 - window) // page] = -7
        q, qr = c.draw(c.rows, c.heads, c.C), c.draw(c.rows, c.heads, ROPE)
        start, ln, pos = c.batch(c.seqs)
        out = c.kv.attend(q.cuda(), qr.cuda(), cu(pos), cu(start), cu(ln), cu(c.table), SCALE, window=window)
        r = c.oracle.attend(num(q), num(qr), pos, start, ln, np.maximum(c.table, 0), SCALE, True, window or 0)
        check(out, r, latent_bounds.absorbed(r, KIND[dtype]))
        assert c.kv.debug_state() == 0


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("seqs", [[(4, 60)], [(100, 30), (3, 90)], [(1, 9000), (4, 9000)]])
def test_a_marked_token_reaches_only_the_queries_that_see_it(seqs, dtype):
    c = Case(seqs, heads=5, latent=128, page=16, dtype=dtype)
    start, ln, pos = c.batch([(n, 0) for n in c.len])
    x, r = c.draw(int(start[-1]), 128), c.draw(int(start[-1]), ROPE)
    clean = LatentOracle(128, c.n_pages, 16)
    clean.append(num(x), num(r), pos, start, ln, c.table)
    marked = []
    for b, (n, before) in enumerate(seqs):
        for j, t in ((before + n // 2, x), (before + n - 1, r), (3, x)):
            t[start[b] + j, 5] = float("nan" if j % 2 else "inf")
            marked.append((b, j))
    c.kv.append(x.cuda(), r.cuda(), cu(pos), cu(start), cu(ln), cu(c.table))
    start, ln, pos = c.batch(seqs)
    q, qr = c.draw(c.n, 5, 128), c.draw(c.n, 5, ROPE)
    for window in (20, 8990 if max(c.len) > 9000 else 33):
        out = c.kv.attend(q.cuda(), qr.cuda(), cu(pos), cu(start), cu(ln), cu(c.table), SCALE, window=window).cpu()
        want = clean.attend(num(q), num(qr), pos, start, ln, c.table, SCALE, True, window)
        bound = latent_bounds.absorbed(want, KIND[dtype])
        for b, (n, before) in enumerate(seqs):
            for i in range(n):
                at, row = before + i, start[b] + i
                if any(s == b and at - window < j <= at for s, j in marked):
                    assert bool(torch.isnan(out[row]).all()), (b, i)
                else:
                    err = np.abs(out[row].double().numpy() - want.out[row])
                    assert np.all(err <= bound[row]), (b, i)
    q[0, 1, 3], qr[c.n - 1, 2, 9] = float("nan"), float("inf")
    out = c.kv.attend(q.cuda(), qr.cuda(), cu(pos), cu(start), cu(ln), cu(c.table), SCALE, window=1).cpu()
    bad = [b for b in range(len(seqs)) for s, j in marked if s == b and j == seqs[b][1]]
    assert bool(torch.isnan(out[0, 1]).all()) and bool(torch.isnan(out[c.n - 1, 2]).all())
    assert bad or not bool(torch.isnan(out[0, 0]).any())
    assert c.kv.debug_state() == 0


def test_rows_that_see_nothing_are_zero():
    c = Case([(4, 0), (40, 0), (2, 30)], heads=6)
    c.fill(1)
    start, ln = np.array([0, 4, 44, 46], np.int32), np.array([2, 13, 0], np.int32)
    pos = np.zeros((46, 1), np.int32)
    q, qr = c.draw(46, 6, c.C), c.draw(46, 6, ROPE)
    for causal in (True, False):
        out = c.kv.attend(q.cuda(), qr.cuda(), cu(pos), cu(start), cu(ln), cu(c.table), SCALE, causal=causal)
        r = c.oracle.attend(num(q), num(qr), pos, start, ln, c.table, SCALE, causal)
        check(out, r, latent_bounds.absorbed(r, "bf16"))
        assert bool((out[44:] == 0).all())                  # an empty cache
        if causal:
            assert bool((out[:2] == 0).all()) and bool((out[4:31] == 0).all())
    assert c.kv.debug_state() == 0


@pytest.mark.parametrize("heads", [4, 60])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_tokens_of_very_different_size(dtype, heads):
    """Zero tokens, tiny and huge ones side by side: a token's scale is an offset of
    its logits and a weight of its codes."""
    c = Case([(2, 700), (1, 64)], heads=heads, latent=128, page=16, dtype=dtype)
    total = sum(c.len)
    x, r = c.draw(total, 128).float(), c.draw(total, ROPE).float()
    size = np.exp2(c.g.integers(-10, 5, total)).astype(np.float32)
    size[100:140] = 0
    size[:20] = 2.0 ** -20 if dtype is BF else 2.0 ** -9
    x, r = x * torch.from_numpy(size)[:, None], r * torch.from_numpy(size)[:, None]
    c.append([(n, 0) for n in c.len], x.to(dtype), r.to(dtype))
    c.check_cache()
    c.attend(scale=0.02)
    c.attend(scale=0.02, window=100)
    assert c.kv.debug_state() == 0


@pytest.mark.parametrize("dtype", [BF, HF])
def test_maxima_that_rise_late(dtype):
    """Keys whose logits grow from tile to tile: the reference is raised again and
    again, by a little and by much."""
    c = Case([(2, 1500)], heads=40, latent=128, dtype=dtype)
    total = c.len[0]
    x = (c.g.standard_normal((total, 128)) * 0.3).astype(np.float32)
    way = c.g.standard_normal(128).astype(np.float32)
    grow = np.repeat(np.cumsum(c.g.choice([0, 0.5, 3.0], total // 100 + 1)), 100)[:total]
    x += grow[:, None].astype(np.float32) * way / np.linalg.norm(way)
    c.append([(total, 0)], torch.from_numpy(x).to(dtype), c.draw(total, ROPE) * 0.1)
    q = torch.from_numpy((c.g.uniform(0, 12, (2, 40, 1)) * way).astype(np.float32)).to(dtype)
    c.attend(q=q, qr=c.draw(2, 40, ROPE) * 0.1)
    assert c.kv.debug_state() == 0


# ---------------------------------------------------------------- the expanded form
class Expanded:
    """Keys and values of every head, as slices of one product's output."""

    def __init__(self, seqs, heads=4, dtype=BF, axes=1, seed=0, extra_rows=0, gap=0, big=1.0):
        self.c = Case(seqs, heads=heads, latent=128, axes=axes, dtype=dtype, seed=seed)
        c = self.c
        self.first = np.concatenate([[0], np.cumsum([n + gap for n in c.len])]).astype(np.int32)[:len(seqs)]
        self.T = sum(c.len) + gap * len(seqs)
        self.q = c.draw(c.n + extra_rows, heads, 192) * 0.6
        self.kv = c.draw(self.T, heads, 256) * big
        self.k, self.v = self.kv[..., :128], self.kv[..., 128:]
        self.rows = c.draw(self.T, c.C + ROPE)
        self.kr = self.rows[:, c.C:]
        self.extra = extra_rows

    def run(self, **how):
        c = self.c
        start, ln, pos = c.batch(c.seqs)
        self.args = pos, start, ln
        pos = np.concatenate([pos, np.zeros((self.extra, pos.shape[1]), np.int32)])
        kv, rows = self.kv.cuda(), self.rows.cuda()
        out = torch.full((c.n + self.extra, c.heads, 128), 7.0, dtype=c.dtype, device="cuda")
        got = c.kv.attend_expanded(self.q.cuda(), kv[..., :128], rows[:, c.C:], kv[..., 128:], cu(pos), cu(start), cu(self.first),
                                   cu(ln), out=out, **how)
        assert got is out
        return out

    def want(self, causal=True, window=None, scale=None, **_):
        pos, start, ln = self.args
        return attend_expanded(num(self.q[:self.c.n]), num(self.k), num(self.kr), num(self.v), pos, start, self.first, ln,
                               self.c.axis_dims, causal=causal, window=window or 0, scale=scale)

    def check(self, **how):
        out = self.run(**how)
        r = self.want(**how)
        check(out[:self.c.n], r, latent_bounds.expanded(r, KIND[self.c.dtype]))
        assert bool((out[self.c.n:] == 7.0).all())
        assert self.c.kv.debug_state() == 0
        return out


@pytest.mark.parametrize("case,how", [
    (dict(seqs=[(1, 0)]), {}),
    (dict(seqs=[(90, 0)], heads=5, dtype=HF), {}),
    (dict(seqs=[(1, 5), (1, 0), (3, 126), (1, 127), (0, 9), (2, 128), (5, 700)], heads=3), {}),
    (dict(seqs=[(257, 0), (128, 0), (129, 1), (255, 300)], heads=2), {}),
    (dict(seqs=[(300, 40)], heads=2, axes=3, dtype=HF), dict(causal=False)),
    (dict(seqs=[(300, 200), (20, 400)], heads=3, gap=5), dict(window=33)),
    (dict(seqs=[(130, 500)], heads=2, dtype=HF, gap=130), dict(window=1)),
    (dict(seqs=[(600, 0)], heads=1, big=20.0), dict(scale=0.2)),
    (dict(seqs=[(100, 9000)], heads=2), {}),                 # items cut over many blocks
    (dict(seqs=[(2, 6000), (300, 6000)], heads=3, dtype=HF), dict(window=4000)),
], ids=range(10))
def test_expanded(case, how):
    e = Expanded(extra_rows=3, **case)
    e.check(**how)
    if max(e.c.new) > 0:
        a = e.check(max_new=max(e.c.new), **how)
        b = e.run(max_new=max(e.c.new), **how)
        assert bool((a == b).all())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("window", [None, 50])
def test_expanded_values_that_are_no_numbers(dtype, window):
    """Non-finite keys and values in front of some queries, behind others, between
    the sequences and past the last: only the queries that see one change."""
    e = Expanded([(200, 30), (3, 140), (150, 0)], heads=2, dtype=dtype, gap=9)
    e.run(window=window)
    clean = e.want(window=window)
    bound = latent_bounds.expanded(clean, KIND[dtype])
    marked = []                                              # (sequence, index, heads)
    for b, j, h, t in ((0, 100, 0, e.v), (0, 229, 1, e.v), (1, 142, 0, e.v), (2, 70, 1, e.k), (2, 149, 0, e.v)):
        t[e.first[b] + j, h, 17] = float("nan" if j % 2 else "inf")
        marked.append((b, j, h))
    for b in range(3):
        e.kv[e.first[b] + e.c.len[b]:e.first[b] + e.c.len[b] + 9] = float("nan")
        e.rows[e.first[b] + e.c.len[b]:e.first[b] + e.c.len[b] + 9] = float("inf")
    out = e.run(window=window).cpu()
    pos, start, ln = e.args
    # an infinite key against a negative query number has the score -inf, and the weight 0
    k = e.k.clone()
    k[e.first[2] + 70, 1, 17] = 1e30
    k[k.isnan()] = 0
    less = attend_expanded(num(e.q), num(k), *(num(x.nan_to_num(0, 0, 0)) for x in (e.kr, e.v)), pos, start, e.first, ln,
                           window=window or 0)
    less.all = clean.all                                    # without that key's 1e30
    less_bound = latent_bounds.expanded(less, KIND[dtype])
    for b, (n, before) in enumerate(e.c.seqs):
        for i in range(n):
            at, row = before + i, start[b] + i
            for h in range(2):
                hit = [j for s, j, g in marked if s == b and g == h and j <= at and (window is None or j > at - window)]
                if hit == [70] and (b, h) == (2, 1) and e.q[row, 1, 17] < 0:
                    assert np.all(np.abs(out[row, h].double().numpy() - less.out[row, h]) <= less_bound[row, h]), (b, i, h)
                elif hit:
                    assert not bool(torch.isfinite(out[row, h, 17])), (b, i, h)
                else:
                    err = np.abs(out[row, h].double().numpy() - clean.out[row, h])
                    assert np.all(err <= bound[row, h]), (b, i, h)
    assert e.c.kv.debug_state() == 0


def test_expanded_rows_that_see_nothing_and_bad_numbers():
    from fp8_ring_kv_gb300 import kvring as K
    e = Expanded([(40, 0), (7, 20)], heads=2)
    good = e.check()
    c = e.c
    start, ln, pos = c.batch(c.seqs)
    kv, rows, q = e.kv.cuda(), e.rows.cuda(), e.q.cuda()

    def call(first=e.first, ln=ln, n_keys=None, **how):
        out = torch.full((c.n, 2, 128), 7.0, dtype=BF, device="cuda")
        t = kv.shape[0] if n_keys is None else n_keys
        c.kv.attend_expanded(q, kv[:t, :, :128], rows[:t, c.C:], kv[:t, :, 128:], cu(pos), cu(start), cu(first), cu(ln), out=out, **how)
        err = c.kv.debug_state()
        c.kv.workspace[:4].zero_()
        return out, err

    out, err = call(ln=np.array([10, 0], np.int32))
    assert err == 0 and bool((out[:30] == 0).all()) and bool((out[40:] == 0).all()) and not bool((out[30:40] == 0).all())
    for first in (-1, 41, 2 ** 31 - 1, -2 ** 31):            # keys of the second sequence outside the tensor
        out, err = call(first=np.array([0, first], np.int32))
        assert err == K.KVRING_DEVERR_SEQ and bool((out[40:] == 7).all()) and bool((out[:40] == good[:40]).all())
    out, err = call(n_keys=66)
    assert err == K.KVRING_DEVERR_SEQ and bool((out[40:] == 7).all()) and bool((out[:40] == good[:40]).all())
    out, err = call(ln=np.array([-1, 27], np.int32))
    assert err == K.KVRING_DEVERR_SEQ and bool((out[:40] == 7).all()) and bool((out[40:] == good[40:]).all())
    out, err = call(max_new=7)
    assert err == K.KVRING_DEVERR_SEQ and bool((out[:40] == 7).all()) and bool((out[40:] == good[40:]).all())
    out, err = call(first=np.array([0, 0], np.int32), ln=np.array([0, 0], np.int32), n_keys=0)
    assert err == 0 and bool((out == 0).all())
    out, err = call(ln=np.array([0, 0], np.int32), n_keys=0)             # its 40 are not in the tensor, keys or none
    assert err == K.KVRING_DEVERR_SEQ and bool((out[:40] == 0).all()) and bool((out[40:] == 7).all())


# ---------------------------------------------------------------- together, layouts, streams, graphs
@pytest.mark.parametrize("dtype", [BF, HF])
def test_prompt_and_decode_together(dtype):
    """As a server runs it: prompts written, read back and attended in the expanded
    form, then single tokens in the absorbed form; both forms of one step agree."""
    heads, C, d = 4, 256, 128
    c = Case([(0, 90), (0, 61), (0, 210)], heads=heads, latent=C, page=32, dtype=dtype)
    w = c.g.standard_normal((2, heads, d, C)) * C ** -0.5
    wk, wv = (torch.from_numpy(x).cuda() for x in w)
    have = [70, 33, 180]
    c.append([(n, 0) for n in have])
    for step in range(6):
        new = [7, 0, 20] if step == 0 else [1, 1, 1]
        seqs = [(a, b) for a, b in zip(new, have)]
        c.append(seqs)
        have = [a + b for a, b in seqs]
        start, ln, pos = c.batch(seqs)
        n = int(start[-1])
        q = c.draw(n, heads, d + ROPE).cuda()
        dev = [cu(x) for x in (pos, start, ln, c.table)]
        # absorbed: queries into the latent space, outputs out of it
        ql = torch.einsum("nhd,hdc->hnc", q[..., :d].double(), wk).to(dtype).transpose(0, 1)
        got = c.kv.attend(ql, q[..., d:], *dev, SCALE, max_new=max(new))
        r = c.oracle.attend(num(ql.cpu()), num(q[..., d:].cpu()), pos, start, ln, c.table, SCALE)
        check(got, r, latent_bounds.absorbed(r, KIND[dtype]))
        # expanded: rows read back, keys and values made from them
        kv_start = np.concatenate([[0], np.cumsum(ln)]).astype(np.int32)
        rows = c.kv.read(cu(kv_start), dev[2], dev[3], int(kv_start[-1]))
        k, v = (torch.einsum("tc,hdc->thd", rows[:, :C].double(), x).to(dtype) for x in (wk, wv))
        out = c.kv.attend_expanded(q, k, rows[:, C:], v, dev[0], dev[1], cu(kv_start[:-1]), dev[2], max_new=max(new))
        r = attend_expanded(num(q.cpu()), num(k.cpu()), num(rows[:, C:].cpu()), num(v.cpu()), pos, start, kv_start[:-1], ln)
        check(out, r, latent_bounds.expanded(r, KIND[dtype]))
        # the two forms: they differ by the roundings of ql, k, v and the outputs, each half a
        # step of numbers around 1 that enter logits of size 1 and outputs of size 1
        absorbed = torch.einsum("nhc,hdc->nhd", got.double(), wv)
        diff = (absorbed - out.double()).square().mean().sqrt() / out.double().square().mean().sqrt()
        assert float(diff) < 16 * latent_bounds.U[KIND[dtype]]
    c.check_cache()
    assert c.kv.debug_state() == 0


@pytest.mark.parametrize("dtype,heads", [(BF, 6), (BF, 40), (HF, 6)])
def test_strides_layers_and_shared_pages(dtype, heads):
    c = Case([(5, 60), (1, 130), (30, 3)], heads=heads, layers=3, extra_rows=4, dtype=dtype)
    c.fill(1)
    c.table[1, 0] = c.table[0, 0]                            # 64 tokens read by both
    c.kv.codes[1].copy_(c.kv.codes[0])
    c.kv.scales[1].copy_(c.kv.scales[0])
    c.kv.codes[0].zero_()
    start, ln, pos = c.batch(c.seqs)
    pos = np.concatenate([pos, np.zeros((4, 1), np.int32)])
    wide = torch.full((3, c.table.shape[1] + 5), -3, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + c.table.shape[1]] = cu(c.table)
    table = wide[:, 2:2 + c.table.shape[1]]
    q, qr = c.draw(c.rows, heads, c.C), c.draw(c.rows, heads, ROPE)
    q[c.n:], qr[c.n:] = float("nan"), float("nan")
    r = c.oracle.attend(num(q[:c.n]), num(qr[:c.n]), pos[:c.n], start, ln, c.table, SCALE)
    layouts = {
        "heads outside": lambda t: t.transpose(0, 1).contiguous().transpose(0, 1),
        "slices": lambda t: torch.cat([t, t[..., :8]], 2)[..., :t.shape[2]],
        "as they come": lambda t: t,
    }
    for name, lay in layouts.items():
        out = lay(torch.full((c.rows, heads, c.C), 5.0, dtype=dtype, device="cuda"))
        got = c.kv.attend(lay(q.cuda()), lay(qr.cuda()), cu(pos), cu(start), cu(ln), table, SCALE, out=out, layer=1)
        assert got.data_ptr() == out.data_ptr()
        check(out[:c.n], r, latent_bounds.absorbed(r, KIND[dtype]))
        assert bool((out[c.n:] == 5).all()), name
    # appends from slices, into one layer only
    x, rp = c.draw(c.n, c.C + ROPE + 8), c.draw(c.n, ROPE)
    before = [c.kv.codes[i].clone() for i in (0, 1)]
    c.table[1, 0] = c.table[1, 1] if c.table[1, 0] == c.table[0, 0] and c.seqs[1][1] < 64 else c.table[1, 0]
    c.kv.append(x.cuda()[:, :c.C], rp.cuda(), cu(pos[:c.n]), cu(start), cu(ln), table, layer=2)
    assert bool((c.kv.codes[0] == before[0]).all()) and bool((c.kv.codes[1] == before[1]).all())
    rows = c.kv.read(cu(start), cu(ln), table, c.n, layer=2).float().cpu()
    assert float((rows[:, :c.C] - x[:, :c.C].float()).abs().max()) <= 2.0 ** -4 * float(x.float().abs().max())
    assert c.kv.debug_state() == 0


def test_expanded_strides():
    e = Expanded([(60, 30), (5, 200)], heads=3)
    want = e.check()
    c = e.c
    pos, start, ln = e.args
    outside = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)
    out = outside(torch.full((c.n, 3, 128), 5.0, dtype=BF, device="cuda"))
    c.kv.attend_expanded(outside(e.q.cuda()), outside(e.k.cuda()), e.kr.cuda().contiguous(), outside(e.v.cuda()), cu(pos), cu(start),
                         cu(e.first), cu(ln), out=out)
    assert bool((out == want).all())


def test_captured_calls_follow_the_lengths():
    """One graph of append, read and both attentions, replayed while the host moves
    the lengths and inputs on; another graph of the same cache in between."""
    steps, heads, C = 40, 6, 128
    c = Case([(0, 40 + steps), (0, 3 + steps), (0, 200 + steps)], heads=heads, latent=C, page=16)
    have = [40, 3, 200]
    c.append([(n, 0) for n in have])
    start, ln, pos = c.batch([(1, n) for n in have])
    dt = dict(dtype=BF, device="cuda")
    x, r, q, qr = (torch.zeros(s, **dt) for s in ((3, C), (3, ROPE), (3, heads, C), (3, heads, ROPE)))
    ln_d, pos_d, start_d, table = cu(ln), cu(pos), cu(start), cu(c.table)
    out, out2, rows = torch.zeros((3, heads, C), **dt), torch.zeros((3, heads, C), **dt), torch.zeros((3, C + ROPE), **dt)
    graphs, side = [], torch.cuda.Stream()
    with torch.cuda.stream(side):
        for o, kw in ((out, dict(max_new=1)), (out2, dict(window=20))):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=side):
                c.kv.append(x, r, pos_d, start_d, ln_d, table)
                c.kv.read(start_d, ln_d, table, out=rows)
                c.kv.attend(q, qr, pos_d, start_d, ln_d, table, SCALE, out=o, **kw)
            graphs.append(gr)
    torch.cuda.synchronize()
    for step in range(steps):
        fresh = [c.draw(*t.shape) for t in (x, r, q, qr)]
        start, ln, pos = c.batch([(1, n) for n in have])
        for d, h in zip((x, r, q, qr, ln_d, pos_d), fresh + [torch.from_numpy(ln), torch.from_numpy(pos)]):
            d.copy_(h)
        graphs[0].replay()
        graphs[1].replay()
        c.oracle.append(num(fresh[0]), num(fresh[1]), pos, start, ln, c.table)
        if step % 13 == 0 or step == steps - 1:
            for o, w in ((out, 0), (out2, 20)):
                res = c.oracle.attend(num(fresh[2]), num(fresh[3]), pos, start, ln, c.table, SCALE, True, w)
                check(o, res, latent_bounds.absorbed(res, "bf16"))
            assert bool((rows.cpu() == torch.from_numpy(c.oracle.read(start, ln, c.table)).to(BF)).all())
        have = [n + 1 for n in have]
    c.check_cache()
    assert c.kv.debug_state() == 0


def test_a_captured_expanded_call():
    e = Expanded([(60, 30), (5, 200), (200, 0)], heads=3)
    want = e.check()
    c = e.c
    pos, start, ln = e.args
    args = [e.q.cuda(), *(t.cuda() for t in (e.k, e.kr, e.v)), cu(pos), cu(start), cu(e.first), cu(ln)]
    out = torch.zeros_like(want)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        c.kv.attend_expanded(*args, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert bool((out == want).all())
    args[7].copy_(torch.tensor([90, 0, 200]))                # the middle sequence has no keys any more
    graph.replay()
    torch.cuda.synchronize()
    assert bool((out[60:65] == 0).all()) and bool((out[:60] == want[:60]).all()) and bool((out[65:] == want[65:]).all())


def test_another_stream_and_two_caches_at_once():
    pair = [Case([(10, 900), (1, 3000)], heads=8, latent=256, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in pair]
    work = []
    for c, st in zip(pair, streams):
        start, ln, pos = c.batch([(n, 0) for n in c.len])
        x, r = c.draw(int(start[-1]), c.C), c.draw(int(start[-1]), ROPE)
        dev = [t.cuda() for t in (x, r)] + [cu(t) for t in (pos, start, ln, c.table)]
        c.oracle.append(num(x), num(r), pos, start, ln, c.table)
        start, ln, pos = c.batch(c.seqs)
        q, qr = c.draw(c.n, 8, c.C), c.draw(c.n, 8, ROPE)
        work.append((c, st, dev, q, qr, pos, start, ln, [q.cuda(), qr.cuda()] + [cu(t) for t in (pos, start, ln, c.table)]))
    torch.cuda.synchronize()
    outs = [None, None]
    for c, st, dev, *_ in work:
        c.kv.append(*dev, stream=st)
    for _ in range(10):
        for i, w in enumerate(work):
            outs[i] = w[0].kv.attend(*w[-1], SCALE, stream=w[1] if _ % 2 else w[1].cuda_stream)
    torch.cuda.synchronize()
    for (c, st, dev, q, qr, pos, start, ln, _), out in zip(work, outs):
        r = c.oracle.attend(num(q), num(qr), pos, start, ln, c.table, SCALE)
        check(out, r, latent_bounds.absorbed(r, "bf16"))
        c.check_cache()


def test_many_calls_in_a_row():
    """The kernels of consecutive calls overlap at their ends (dependent launch): the
    outputs are those of single calls."""
    c = Case([(2, 50), (30, 0), (1, 4000), (17, 9)], heads=5, page=32)
    c.fill(1)
    e = Expanded([(60, 30), (300, 0)], heads=5)
    e.run()
    pos, start, ln = e.args
    xa = [e.q.cuda(), *(t.cuda() for t in (e.k, e.kr, e.v)), cu(pos), cu(start), cu(e.first), cu(ln)]
    start, ln, pos = c.batch(c.seqs)
    args = [cu(x) for x in (pos, start, ln, c.table)]
    qs = [(c.draw(c.n, 5, c.C).cuda(), c.draw(c.n, 5, ROPE).cuda()) for _ in range(3)]
    calls = [lambda q=q: c.kv.attend(*q, *args, SCALE) for q in qs] + [lambda: e.c.kv.attend_expanded(*xa),
                                                                        lambda: c.kv.read(args[1], args[2], args[3], c.n)]
    want = []
    for f in calls:
        want.append(f().clone())
        torch.cuda.synchronize()
    outs = [calls[i % 5]() for i in range(60)]
    torch.cuda.synchronize()
    assert all(bool((o == want[i % 5]).all()) for i, o in enumerate(outs))


def test_first_calls_on_a_workspace_that_held_something_else():
    from fp8_ring_kv_gb300 import LatentKV
    from fp8_ring_kv_gb300.latent import kvring_latent_workspace_bytes, make_latent_config
    c = Case([(3, 70), (1, 300)], heads=40, latent=128)
    c.fill(1)
    start, ln, pos = c.batch([(n, 0) for n in c.len])
    x, r = c.draw(int(start[-1]), 128).cuda(), c.draw(int(start[-1]), ROPE).cuda()
    shape = (40, 128, c.n_pages, 64, (ROPE,), (0,), (400,))
    ws = torch.empty(kvring_latent_workspace_bytes(make_latent_config(*shape)), dtype=torch.uint8, device="cuda")
    q, qr = c.draw(c.n, 40, 128).cuda(), c.draw(c.n, 40, ROPE).cuda()
    first = None
    for byte in (0, 0xFF, 0x7F, 0x80):
        ws.fill_(byte)
        kv = LatentKV(*shape, workspace=ws)
        kv.append(x, r, cu(pos), cu(start), cu(ln), cu(c.table))
        s2, l2, p2 = c.batch(c.seqs)
        out = kv.attend(q, qr, cu(p2), cu(s2), cu(l2), cu(c.table), SCALE)
        assert kv.debug_state() == 0
        first = out.clone() if first is None else first
        assert bool((out == first).all())


# ---------------------------------------------------------------- refusals
def test_numbers_that_contradict_are_left_out():
    from fp8_ring_kv_gb300 import kvring as K
    c = Case([(3, 60), (5, 5), (40, 100), (2, 20)], heads=6)
    c.fill(1)
    q, qr = c.draw(c.n, 6, c.C), c.draw(c.n, 6, ROPE)
    start, ln, pos = c.batch(c.seqs)
    args = [q.cuda(), qr.cuda(), cu(pos)]
    good = c.kv.attend(*args, cu(start), cu(ln), cu(c.table), SCALE)
    rows = c.kv.read(cu(start), cu(ln), cu(c.table), c.n)
    codes = c.kv.codes.clone()

    def state():
        err = c.kv.debug_state()
        c.kv.workspace[:4].zero_()
        return err

    def attend(start, ln, table=c.table, **kw):
        out = torch.full((c.n, 6, c.C), 7.0, dtype=BF, device="cuda")
        c.kv.attend(*args, cu(start), cu(ln), cu(table), SCALE, out=out, **kw)
        err = state()
        back = torch.full((c.n, c.C + ROPE), 7.0, dtype=BF, device="cuda")
        c.kv.read(cu(start), cu(ln), cu(table), out=back)
        return out, err, back, state()

    for bad_len in (-1, c.table.shape[1] * c.page + 1, 2 ** 31 - 1):
        l2 = ln.copy()
        l2[1] = bad_len
        out, err, back, err2 = attend(start, l2)
        assert err == err2 == K.KVRING_DEVERR_SEQ
        assert bool((out[3:8] == 7).all()) and bool((back[3:8] == 7).all())
        assert bool((out[:3] == good[:3]).all()) and bool((out[8:] == good[8:]).all()) and bool((back[8:] == rows[8:]).all())
    for s1 in (-5, 2 ** 30, 60):                             # decreasing or past the rows
        s2 = start.copy()
        s2[1] = s1
        out, err, _, err2 = attend(s2, ln)
        assert err == err2 == K.KVRING_DEVERR_SEQ and bool((out[8:] == good[8:]).all())
    out, err, _, _ = attend(start, ln, max_new=5)            # the third sequence has 40
    assert err == K.KVRING_DEVERR_SEQ and bool((out[8:48] == 7).all()) and bool((out[48:] == good[48:]).all())
    # append and read: more new tokens than the sequence has with them
    x, r = c.draw(c.n, c.C).cuda(), c.draw(c.n, ROPE).cuda()
    l2 = np.array([2, 4, 39, 1], np.int32)
    c.kv.append(x, r, cu(pos), cu(start), cu(l2), cu(c.table))
    assert state() == K.KVRING_DEVERR_SEQ and bool((c.kv.codes == codes).all())
    back = torch.full_like(rows, 7.0)
    c.kv.read(cu(start), cu(l2), cu(c.table), out=back)
    assert state() == K.KVRING_DEVERR_SEQ and bool((back == 7).all())
    # page ids outside the pool
    for pg in (-1, c.n_pages, 2 ** 31 - 1, -2 ** 31):
        t2 = c.table.copy()
        t2[2, 1] = pg
        out, err, back, err2 = attend(start, ln, t2)
        assert err == err2 == K.KVRING_DEVERR_PAGE and bool(torch.isfinite(out.float()).all())
        assert bool((out[:8] == good[:8]).all()) and bool((out[48:] == good[48:]).all())
        assert bool(((back == rows) | (back == 7)).all()) and bool((back[:8] == rows[:8]).all())
        c.kv.append(x, r, cu(pos), cu(start), cu(ln), cu(np.where(c.table >= 0, pg, -1).astype(np.int32)))
        assert state() == K.KVRING_DEVERR_PAGE and bool((c.kv.codes == codes).all())
    # positions outside the table are clamped
    p2 = pos.copy()
    p2[0], p2[1] = 10 ** 6, -4
    c.kv.append(x, r, cu(p2), cu(start), cu(ln), cu(c.table))
    assert state() == K.KVRING_DEVERR_POS_RANGE


def test_host_refusals():
    from fp8_ring_kv_gb300 import kvring as K
    from fp8_ring_kv_gb300.kvring import KVRingError
    e = Expanded([(3, 60), (2, 5)], heads=4)
    c = e.c
    c.fill(1)
    start, ln, pos = c.batch(c.seqs)
    dev = dict(dtype=BF, device="cuda")
    good = {
        "append": dict(latent=torch.zeros(5, 128, **dev), k_rope=torch.zeros(5, 64, **dev), pos=cu(pos), seq_start=cu(start), kv_len=cu(ln),
                       page_table=cu(c.table)),
        "read": dict(seq_start=cu(start), kv_len=cu(ln), page_table=cu(c.table), n_rows=5),
        "attend": dict(q_latent=torch.zeros(5, 4, 128, **dev), q_rope=torch.zeros(5, 4, 64, **dev), q_pos=cu(pos), seq_start=cu(start),
                       kv_len=cu(ln), page_table=cu(c.table), scale=1.0),
        "attend_expanded": dict(q=torch.zeros(5, 4, 192, **dev), k=e.k.cuda(), k_rope=e.kr.cuda(), v=e.v.cuda(), q_pos=cu(pos),
                                seq_start=cu(start), kv_start=cu(e.first), kv_len=cu(ln)),
    }
    for name, kw in good.items():
        getattr(c.kv, name)(**kw)

    def bad(match, what, **kw):
        with pytest.raises(KVRingError, match=match):
            getattr(c.kv, what)(**dict(good[what], **kw))

    for what in ("append", "read", "attend"):
        bad("layer", what, layer=1)
        bad("layer", what, layer=-1)
        bad("shape", what, page_table=cu(c.table)[0])
        bad("more than", what, page_table=torch.zeros((2, 70000), dtype=torch.int32, device="cuda"))
    for what in good:
        bad("int64", what, kv_len=cu(ln).long())
        bad("shape", what, seq_start=cu(start)[:2])
        bad("cpu", what, seq_start=torch.from_numpy(start))
    for what, name in (("append", "pos"), ("attend", "q_pos"), ("attend_expanded", "q_pos"), ("attend_expanded", "kv_start")):
        bad("shape", what, **{name: good[what][name][:1]})
    for what, names in (("append", ("latent", "k_rope")), ("attend", ("q_latent", "q_rope")), ("attend_expanded", ("q", "k", "k_rope", "v"))):
        for name in names:
            t = good[what][name]
            bad("float16", what, **{name: t.half()})
            bad("shape", what, **{name: t[..., :-8]})
            bad("cpu", what, **{name: t.cpu()})
            bad("strides", what, **{name: t.transpose(0, -1).contiguous().transpose(0, -1)})
            flat = torch.zeros(t.numel() + 4, **dev)[4:].view_as(t)
            bad("misaligned", what, **{name: flat})
            bad("strides", what, **{name: t[:1].expand_as(t)})
    for what in ("attend", "attend_expanded"):
        bad("window", what, window=4, causal=False)
        bad("window", what, window=0)
        bad("max_new", what, max_new=0)
        bad("max_new", what, max_new=6)
        for scale in (-1.0, float("inf"), float("nan"), 1e-40):
            bad("scale", what, scale=scale)
        bad("shape", what, out=torch.zeros(4, 4, 128, **dev))
        bad("strides", what, out=torch.zeros(5, 4, 128, 2, **dev)[..., 0])
        bad("strides", what, out=torch.zeros(1, 4, 128, **dev).expand(5, -1, -1))
    bad("scale", "attend", scale=0.0)
    bad("n_rows", "read", n_rows=None)
    bad("n_rows", "read", n_rows=4, out=torch.zeros(5, 192, **dev))
    bad("strides", "read", out=torch.zeros(5, 196, **dev)[:, :192])
    bad("shape", "read", out=torch.zeros(5, 128, **dev))
    many = torch.zeros((2049, 1), dtype=torch.int32, device="cuda")
    bad("sequences", "read", page_table=many, kv_len=many[:, 0].contiguous(), seq_start=torch.zeros(2050, dtype=torch.int32, device="cuda"))
    assert c.kv.debug_state() == 0
    # the C entry points by themselves
    lib, h, p = K.load(), c.kv.handle, c.kv.workspace.data_ptr()
    names = "h layer q qt qh r rt rh pos start len n_seqs n max_new table t_stride width causal window scale out ot oh st"
    base = dict(zip(names.split(), [h, 0, p, 512, 128, p, 256, 64, p, p, p, 2, 5, 5, p, 4, 2, 1, 0, 1.0, p, 512, 128, None]))
    for key, value, status in (("layer", 1, -1), ("q", None, -1), ("qt", 504, -1), ("qt", 514, -1), ("qh", 120, -1), ("qh", -128, -1),
                               ("r", p + 8, -2), ("start", None, -1), ("start", p + 2, -2), ("n_seqs", -1, -1), ("n_seqs", 2049, -1),
                               ("n", -1, -1), ("n", 1 << 25, -1), ("max_new", 0, -1), ("max_new", 6, -1), ("width", 0, -1),
                               ("t_stride", 1, -1), ("width", 1 << 20, -1), ("causal", 2, -1), ("window", -1, -1), ("scale", 0.0, -1),
                               ("scale", float("nan"), -1), ("scale", 3e38, -1), ("out", p + 4, -2), ("ot", 8, -1), ("oh", 64, -1)):
        assert lib.kvring_latent_attend(*dict(base, **{key: value}).values()) == status, (key, value)
    # nothing to do is fine
    none = good["attend"]
    out = c.kv.attend(none["q_latent"][:0], none["q_rope"][:0], none["q_pos"][:0], none["seq_start"] * 0, none["kv_len"], none["page_table"], 1.0)
    assert out.shape == (0, 4, 128)
    assert c.kv.read(none["seq_start"] * 0, none["kv_len"], none["page_table"], 0).shape == (0, 192)
    c.kv.close()
    for what, kw in good.items():
        bad("closed", what)
