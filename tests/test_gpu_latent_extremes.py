"""Latent attention at the ends of its ranges."""
import numpy as np
import pytest
import torch

import latent_bounds
from latent_bounds import U
from oracle.latent import attend_expanded
from test_gpu_latent import BF, HF, KIND, ROPE, Case, check, cu, num

pytestmark = pytest.mark.gpu


def attend(c, q, scale, qr=None):
    start, ln, pos = c.batch(c.seqs)
    qr = torch.zeros(c.n, c.heads, ROPE, dtype=c.dtype) if qr is None else qr
    out = c.kv.attend(q.cuda(), qr.cuda(), cu(pos), cu(start), cu(ln), cu(c.table), scale)
    assert c.kv.debug_state() == 0
    return out, c.oracle.attend(num(q), num(qr), pos, start, ln, c.table, scale)


def known(c, first):
    """Rows whose first channel is ``first`` [keys]; the rest drawn, nothing to rotate."""
    x = c.draw(len(first), c.C)
    x[:, 0] = torch.tensor(first).to(c.dtype)
    c.append([(len(first), 0)], x, torch.zeros(len(first), ROPE, dtype=c.dtype))


def near(out, want, dtype):
    """Single weights: 2^-9 + 2^-11 (fp16 2^-13) and fp32 sums, then the output's rounding."""
    u = U[KIND[dtype]]
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= np.abs(want) * (u + (2.0 ** -13 if dtype is HF else 2.0 ** -9 + 2.0 ** -11) * (1 + u) + 2.0 ** -16))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads", [3, 64])
@pytest.mark.parametrize("keys", [1, 40, 3000])
def test_logits_far_below_zero(keys, heads, dtype):
    """Scale 2^100 and products of one sign: the key with the largest logit has all of
    the weight, however negative its logit is."""
    c = Case([(1, keys - 1)], heads=heads, latent=128, page=16, dtype=dtype)
    first = 2.0 + np.arange(keys) % 5
    first[keys * 2 // 3] = 1.0
    if keys > 3:
        first[keys // 3] = 7.0
    known(c, first)
    for size in (1.0, 2.0 ** 14, 2.0 ** -20 if dtype is BF else 2.0 ** -10):
        for sign, at in ((-1, keys * 2 // 3), (1, keys // 3)):
            q = torch.zeros(1, heads, 128, dtype=dtype)
            q[..., 0] = sign * size
            out, r = attend(c, q, 2.0 ** 100)
            value = c.oracle.rows(c.table[0], keys)[at, :128]
            if sign < 0 or keys > 3:
                assert np.allclose(r.out, value)
            near(out, r.out, dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("seqs", [[(1, 0)], [(1, 2999), (3, 40)], [(300, 7)]])
def test_large_logits_of_the_expanded_form(seqs, dtype):
    """Products of one channel and a large scale: the keys with the largest logit that a
    row sees share its weight."""
    c = Case(seqs, heads=2, latent=128, page=16, dtype=dtype)
    start, ln, pos = c.batch(seqs)
    total = sum(c.len)
    k, v, kr = c.draw(total, 2, 128), c.draw(total, 2, 128), c.draw(total, ROPE)
    k[..., 0] = torch.from_numpy(2.0 + (np.arange(total) % 7 + np.arange(total) % 5)[:, None] / 4 + [0, 0.5]).to(dtype)
    first = np.concatenate([[0], np.cumsum(ln)]).astype(np.int32)[:len(seqs)]
    for scale in (2.0 ** 20, 2.0 ** 29, 2.0 ** 40, 2.0 ** 100):
        for sign in (1.0, -1.0):
            q = torch.zeros(c.n, 2, 192, dtype=dtype)
            q[..., 0] = sign * 1.375
            out = c.kv.attend_expanded(q.cuda(), k.cuda(), kr.cuda(), v.cuda(), cu(pos), cu(start), cu(first), cu(ln), scale=scale)
            want = attend_expanded(num(q), num(k), num(kr), num(v), pos, start, first, ln, scale=scale)
            u = U[KIND[dtype]]
            err = np.abs(out.double().cpu().numpy() - want.out)
            # weights 2^-16, sums 2^-16; then the output's rounding
            assert np.all(err <= want.spread * 2.0 ** -15 * (1 + u) + np.abs(want.out) * u + 2.0 ** -24), (scale, sign)
    assert c.kv.debug_state() == 0


@pytest.mark.parametrize("exponent", [-99, -105, -119, -128])
@pytest.mark.parametrize("heads", [3, 64])
def test_queries_near_the_smallest_numbers(exponent, heads):
    """Tiny queries, large keys and scale 2^100: logits of ordinary size."""
    c = Case([(1, 500), (2, 30)], heads=heads, latent=128, page=16)
    total = sum(c.len)
    size = np.float32(2.0 ** (-100 - exponent) / 16)
    x, r = c.draw(total, 128).float() * size, c.draw(total, ROPE).float() * size
    c.append([(n, 0) for n in c.len], x.bfloat16(), r.bfloat16())
    q = (c.draw(c.n, heads, 128).double() * 2.0 ** exponent).bfloat16()
    # rotated numbers of the last size are below what two parts hold of a row: none
    qr = (c.draw(c.n, heads, ROPE).double() * (2.0 ** exponent if exponent > -128 else 0.0)).bfloat16()
    assert float(num(q).__abs__().max()) > 0
    out, want = attend(c, q, 2.0 ** 100, qr)
    check(out, want, latent_bounds.absorbed(want, "bf16"))
    assert float(np.abs(want.out - want.out[:1]).max()) > 0


@pytest.mark.parametrize("heads", [3, 64])
def test_queries_near_the_largest_numbers(heads):
    """A query number times the scale is beyond fp32: keys without that channel have the
    logit 0, others are far away from it."""
    c = Case([(1, 299)], heads=heads, latent=128, page=16)
    first = np.where(np.arange(300) % 3 == 0, 0.0, -1.0 - np.arange(300) % 2)
    known(c, first)
    for size in (2.0 ** 30, 2.0 ** 60, 2.0 ** 120):
        q = torch.zeros(1, heads, 128, dtype=BF)
        q[..., 0] = size
        out, want = attend(c, q, 2.0 ** 80)
        # logits of one product are exact: 0, or too far away to matter.  A weight is off by
        # 2^-9 + 2^-11, sums by 2^-16, the output by its rounding.
        assert np.all(np.abs(out.double().cpu().numpy() - want.out) <=
                      want.spread * (2.0 ** -9 + 2.0 ** -11 + 2.0 ** -16) * (1 + U["bf16"]) + np.abs(want.out) * U["bf16"])
