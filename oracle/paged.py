"""The paged cache in numpy: one power-of-two e4m3 scale per (page, head), and
the attention over it in fp64.

Block scale of rows whose largest magnitude is a: the smallest power of two s
with a <= 448 s, 0 when a < 2^-100; 2^120 for an infinity, whose code is the
largest.  Codes are e4m3_rn(fl32(x / s)), the
division exact.  A page that already holds rows of the sequence keeps its scale
unless the new rows need a larger one; its older codes then become
e4m3_rn(code * (old / new)).  A NaN is left out of the maximum; its code is
0x7F.
"""
import numpy as np

from . import e4m3, rope


def pow2_scale(amax):
    """fp32 amax [...] -> fp32 scale [...]."""
    amax = np.asarray(amax, dtype=np.float32)
    m, e = np.frexp(amax)                       # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = np.where(np.isinf(amax), 129, e)        # an infinity: 2^120
    m = np.where(np.isinf(amax), 0.5, m)
    k = np.where(m <= 0.875, e - 9, e - 8)
    return np.where(amax < np.float32(2.0) ** -100, np.float32(0), np.ldexp(np.float32(1), k)).astype(np.float32)


def encode(x, scale):
    """fp32 x [..., rows, D] at scale [...] -> codes."""
    s = np.asarray(scale, dtype=np.float32)[..., None, None]
    y = np.where(s > 0, x / np.where(s > 0, s, 1), 0).astype(np.float32)
    codes = np.where(s > 0, e4m3.encode_rn_satfinite(np.where(np.isnan(y), 0, y)), np.uint8(0))
    return np.where(np.isnan(x), np.uint8(0x7F), codes).astype(np.uint8)


class PagedOracle:
    def __init__(self, kv_heads, head_dim, n_pages, page_tokens, axis_dims, base=10000.0):
        self.axis_dims, self.base, self.P = axis_dims, base, page_tokens
        shape = (n_pages, kv_heads, page_tokens, head_dim)
        self.codes = {"k": np.zeros(shape, np.uint8), "v": np.zeros(shape, np.uint8)}
        self.scales = {"k": np.zeros(shape[:2], np.float32), "v": np.zeros(shape[:2], np.float32)}

    def append(self, k, v, pos, seq_start, kv_len, table):
        """k, v: fp32 [N, H, D] (values of the 16-bit inputs)."""
        k = rope.rope_f32(k, pos, self.axis_dims, self.base)
        for b, ln in enumerate(kv_len):
            r, end = seq_start[b], seq_start[b + 1]
            t = ln - (end - r)
            while r < end:
                page, off = table[b][t // self.P], t % self.P
                n = min(self.P - off, end - r)
                for name, x in (("k", k), ("v", v)):
                    self._write(name, page, off, np.transpose(x[r:r + n], (1, 0, 2)))
                t, r = t + n, r + n

    def _write(self, name, page, off, x):
        codes, scales = self.codes[name][page], self.scales[name][page]
        need = pow2_scale(np.fmax.reduce(np.abs(x).reshape(len(x), -1), axis=1, initial=0.0))   # NaN left out
        old = scales if off else np.zeros_like(scales)
        new = np.maximum(need, old)
        for h in range(len(new)):
            if off and new[h] > old[h]:
                held = e4m3.decode(codes[h, :off]) * (np.float64(old[h]) / np.float64(new[h]))
                nan = np.isnan(held)
                codes[h, :off] = e4m3.encode_rn_satfinite(np.where(nan, 0, held)) if old[h] > 0 else 0
                codes[h, :off][nan] = 0x7F
        codes[:, off:off + x.shape[1]] = encode(x, new)
        self.scales[name][page] = new

    def rows(self, name, table_row, n, head):
        """fp64 values of a sequence's first n cached rows of one head."""
        if n == 0:
            return np.zeros((0, self.codes[name].shape[3]))
        pages = np.asarray(table_row[:(n + self.P - 1) // self.P])
        x = e4m3.decode(self.codes[name][pages, head]) * self.scales[name][pages, head].astype(np.float64)[:, None, None]
        return x.reshape(-1, x.shape[-1])[:n]

    def attend(self, q, pos, seq_start, kv_len, table, causal=True, window=0, scale=None):
        """q: fp32 [N, Hq, D] -> (out, spread, logit) in fp64: the output,
        sum_t p_t |v_t| per element, and per row the largest
        scale * sum_d |q_d k_td| over the keys it sees."""
        n_rows, heads, dim = q.shape
        g = heads // self.codes["k"].shape[1]
        scale = 1.0 / np.sqrt(dim) if scale is None else scale
        q = rope.rope_f64(q, pos, self.axis_dims, self.base)
        out, spread, logit = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2])
        for b, ln in enumerate(kv_len):
            s0, n = seq_start[b], seq_start[b + 1] - seq_start[b]
            at = ln - n + np.arange(n)
            t = np.arange(ln)
            seen = np.ones((n, ln), bool)
            if causal:
                seen &= t <= at[:, None]
            if window:
                seen &= t > at[:, None] - window
            any_seen = seen.any(axis=1) if ln else np.zeros(n, bool)
            for h in range(heads):
                if not any_seen.any():
                    continue
                k, v = self.rows("k", table[b], ln, h // g), self.rows("v", table[b], ln, h // g)
                x = q[s0:s0 + n, h]
                z = np.where(seen, scale * (x @ k.T), -np.inf)
                with np.errstate(invalid="ignore"):
                    p = np.exp(z - z.max(axis=1, keepdims=True))
                p = np.where(any_seen[:, None], p, 0.0)
                p /= np.where(any_seen, p.sum(axis=1), 1.0)[:, None]
                out[s0:s0 + n, h] = p @ v
                spread[s0:s0 + n, h] = p @ np.abs(v)
                logit[s0:s0 + n, h] = np.where(seen, scale * (np.abs(x) @ np.abs(k).T), 0.0).max(axis=1)
        return out, spread, logit
