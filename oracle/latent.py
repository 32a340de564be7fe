"""The latent cache in numpy: a row (latent, rotated part) per token with one
power-of-two e4m3 scale, and latent attention over it in fp64, in its absorbed
and expanded forms.

Scale of a row whose largest magnitude is a: the smallest power of two s with
a <= 448 s, at least 2^-40.  Codes are e4m3_rn(fl32(x / s)), the division
exact.  A row with anything that is no number, or beyond 448 * 2^40, has the
scale NaN and codes of zeros.
"""
import numpy as np

from . import e4m3, rope

ROPE = 64
LEAST, MOST = -40, 40


def row_scale(amax):
    """fp32 amax [...] -> fp32 scale [...]."""
    amax = np.asarray(amax, dtype=np.float32)
    with np.errstate(invalid="ignore"):
        good = amax <= np.float32(448 * 2.0 ** MOST)                 # false for a NaN
    m, e = np.frexp(np.where(good, amax, 1).astype(np.float32))      # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    k = np.where(m <= 0.875, e - 9, e - 8)
    k = np.where(amax == 0, LEAST, np.maximum(k, LEAST))
    return np.where(good, np.ldexp(np.float32(1), k), np.float32(np.nan)).astype(np.float32)


def encode(x, scale):
    """fp32 rows x [..., W] at scale [...] -> codes."""
    s = np.asarray(scale, np.float32)[..., None]
    good = np.isfinite(s)
    y = (np.where(good, x, 0) / np.where(good, s, 1)).astype(np.float32)
    return np.where(good, e4m3.encode_rn_satfinite(y), np.uint8(0)).astype(np.uint8)


class LatentOracle:
    def __init__(self, latent_dim, n_pages, page_tokens, axis_dims=(ROPE,), base=10000.0):
        self.C, self.P, self.axis_dims, self.base = latent_dim, page_tokens, axis_dims, base
        self.codes = np.zeros((n_pages, page_tokens, latent_dim + ROPE), np.uint8)
        self.scales = np.zeros((n_pages, page_tokens), np.float32)

    def append(self, latent, k_rope, pos, seq_start, kv_len, table):
        """latent, k_rope: fp32 [N, C] and [N, 64] (values of the 16-bit inputs)."""
        with np.errstate(invalid="ignore", over="ignore"):
            turned = rope.rope_f32(k_rope[:, None], pos, self.axis_dims, self.base)[:, 0]
        x = np.concatenate([latent, turned], 1).astype(np.float32)
        for b, ln in enumerate(kv_len):
            n = seq_start[b + 1] - seq_start[b]
            t = np.arange(ln - n, ln)
            page, off = np.asarray(table[b])[t // self.P], t % self.P
            rows = x[seq_start[b]:seq_start[b + 1]]
            scale = row_scale(np.abs(rows).max(axis=1, initial=0.0))
            self.codes[page, off] = encode(rows, scale)
            self.scales[page, off] = scale

    def places(self, table_row, n):
        t = np.arange(n)
        return np.asarray(table_row)[t // self.P], t % self.P

    def rows(self, table_row, n):
        """fp64 values of a sequence's first n cached rows, [n, C + 64]."""
        page, off = self.places(table_row, n)
        return e4m3.decode(self.codes[page, off]) * self.scales[page, off].astype(np.float64)[:, None]

    def read(self, seq_start, kv_len, table):
        out = []
        for b, ln in enumerate(kv_len):
            n = seq_start[b + 1] - seq_start[b]
            out.append(self.rows(table[b], ln)[ln - n:])
        return np.concatenate(out) if out else np.zeros((0, self.C + ROPE))

    def attend(self, q_latent, q_rope, pos, seq_start, kv_len, table, scale, causal=True, window=0):
        """q_latent [N, H, C], q_rope [N, H, 64] -> Result in fp64."""
        turned = rope.rope_f64(q_rope, pos, self.axis_dims, self.base)
        out = Result(q_latent.shape)
        for b, ln in enumerate(kv_len):
            rows = slice(seq_start[b], seq_start[b + 1])
            if rows.stop <= rows.start or ln == 0:
                continue
            kv = self.rows(table[b], ln)
            page, off = self.places(table[b], ln)
            out.add(rows, q_latent[rows], turned[rows], kv[:, None, :self.C], kv[:, self.C:], kv[:, None, :self.C], scale,
                    ln, causal, window, self.scales[page, off].astype(np.float64))
        return out


def attend_expanded(q, k, k_rope, v, pos, seq_start, kv_start, kv_len, axis_dims=(ROPE,), base=10000.0, causal=True, window=0,
                    scale=None):
    """q [N, H, 128 + 64], k, v [T, H, 128], k_rope [T, 64] (rotated) -> Result."""
    scale = (q.shape[2]) ** -0.5 if scale is None else scale
    own = q.shape[2] - ROPE
    turned = rope.rope_f64(q[..., own:], pos, axis_dims, base)
    out = Result(q.shape[:2] + (v.shape[2],))
    for b, ln in enumerate(kv_len):
        rows = slice(seq_start[b], seq_start[b + 1])
        if rows.stop <= rows.start or ln == 0:
            continue
        keys = slice(kv_start[b], kv_start[b] + ln)
        out.add(rows, q[rows][..., :own], turned[rows], k[keys], k_rope[keys], v[keys], scale, ln, causal, window, None)
    return out


class Result:
    """Per element: ``out``; ``spread`` = sum_t p_t |v_t|; ``square`` = sum_t p_t^2
    v_t^2; ``floor`` = max_t(p_t s_t) sum_t |v_t| / s_t (s_t: the token's scale).  Per
    row, the largest over the keys it sees: ``turned`` = scale sum |q k| of the
    rotated part, ``all`` of both, ``ones`` = scale max |q| sum |k|."""

    def __init__(self, shape):
        self.out, self.spread, self.square, self.floor = (np.zeros(shape) for _ in range(4))
        self.turned, self.all, self.ones = (np.zeros(shape[:2]) for _ in range(3))

    def add(self, rows, q, qr, k, kr, v, scale, ln, causal, window, s):
        n, heads = q.shape[:2]
        at, t = ln - n + np.arange(n)[:, None], np.arange(ln)
        seen = np.ones((n, ln), bool)
        if causal:
            seen &= t <= at
        if window:
            seen &= t > at - window
        some = seen.any(axis=1)
        for h in range(heads):
            kh, vh = k[:, min(h, k.shape[1] - 1)], v[:, min(h, v.shape[1] - 1)]
            z = np.where(seen, scale * (q[:, h] @ kh.T + qr[:, h] @ kr.T), -np.inf)
            with np.errstate(invalid="ignore"):
                p = np.exp(z - z.max(axis=1, keepdims=True, initial=-np.inf))
            p = np.where(some[:, None], p, 0.0)
            p /= np.where(some, p.sum(axis=1), 1.0)[:, None]
            self.out[rows, h] = p @ vh
            self.spread[rows, h] = p @ np.abs(vh)
            self.square[rows, h] = (p * p) @ (vh * vh)
            if s is not None:
                codes = np.abs(vh) / np.where(s > 0, s, 1.0)[:, None]          # a page never written has no scale
                self.floor[rows, h] = (p * s).max(axis=1, initial=0.0)[:, None] * (seen @ codes)
            turned = scale * (np.abs(qr[:, h]) @ np.abs(kr).T)
            both = turned + scale * (np.abs(q[:, h]) @ np.abs(kh).T)
            most = np.maximum(np.abs(q[:, h]).max(axis=1), np.abs(qr[:, h]).max(axis=1))[:, None]
            ones = scale * most * (np.abs(kh).sum(axis=1) + np.abs(kr).sum(axis=1))
            for name, x in (("turned", turned), ("all", both), ("ones", ones)):
                getattr(self, name)[rows, h] = np.where(seen, x, 0.0).max(axis=1, initial=0.0)
