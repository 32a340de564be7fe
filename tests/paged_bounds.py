"""How far the paged attention's roundings may carry an output, as a root mean
square: a bound per element must allow for the worst case of every term at once,
and hides a query or weight that has lost its low part."""
import numpy as np

from oracle import rope


def pieces(oracle, q, pos, start, ln, table, causal=True, window=0, scale=None, change=None):
    """Per sequence and head: (rows, head, weights p, values v, scale * sum |q k|
    per row) of the formula in fp64.  change: applied to the rotated queries."""
    heads, dim = q.shape[1:]
    group = heads // oracle.codes["k"].shape[1]
    scale = dim ** -0.5 if scale is None else scale
    x = rope.rope_f64(q, pos, oracle.axis_dims, oracle.base)
    x = x if change is None else change(x)
    for b, n in enumerate(ln):
        rows = slice(start[b], start[b + 1])
        at = n - (start[b + 1] - start[b]) + np.arange(start[b + 1] - start[b])[:, None]
        t = np.arange(n)
        seen = (t <= at) if causal else np.ones((len(at), n), bool)
        if window:
            seen = seen & (t > at - window)
        for h in range(heads):
            k, v = (oracle.rows(name, table[b], n, h // group) for name in "kv")
            z = np.where(seen, scale * (x[rows, h] @ k.T), -np.inf)
            p = np.exp(z - z.max(axis=1, keepdims=True))
            yield rows, h, p / p.sum(axis=1, keepdims=True), v, scale * (np.abs(x[rows, h]) @ np.abs(k).T).max(axis=1)


def outputs(*args, **kw):
    q = args[1]
    out = np.zeros(q.shape)
    for rows, h, p, v, _ in pieces(*args, **kw):
        out[rows, h] = p @ v
    return out


def rms_limit(weight_step, out_step, *args, **kw):
    """weight_step, out_step: half a step of the weights and of the output where
    a mantissa is 1.  A rounding error is even over +- half a step, 2^e times
    that, so its mean square is a third of it squared, relative to the value over
    m^2; m (1 <= m < 2) spreads evenly in its logarithm over weights and outputs,
    and the mean of 1 / m^2 is 3 / (8 log 2).  The errors of a row's weights are
    independent.  fp32: 2^-21 of a weight per unit of its logit's absolute terms
    (products of D channels, the exponent's own rounding) and twice that for the
    exponential and the sums, all generous.  8% for the sample."""
    third = 3 / (8 * np.log(2)) / 3
    total = count = 0.0
    for _, _, p, v, logit in pieces(*args, **kw):
        want = p @ v
        spread = (p * p) @ (v * v)
        fp32 = (np.abs(p) @ np.abs(v)) ** 2 * ((2.0 ** -21 * (2 + logit)) ** 2)[:, None]
        total += (spread * weight_step ** 2 * third + want ** 2 * out_step ** 2 * third + fp32).sum()
        count += want.size
    return 1.08 * np.sqrt(total / count)


def to_fp16_of_row(x):
    """Queries as one fp16 number at a power of two of their row: no low part."""
    e = np.exp2(np.floor(np.log2(np.abs(x).max(axis=-1, keepdims=True))))
    return (x / e).astype(np.float16).astype(np.float64) * e
