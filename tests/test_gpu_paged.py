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
