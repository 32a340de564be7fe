"""The latent cache's numpy oracle, pinned by closed forms and by the attention of
plain keys and values; and the library's host-side checks that need no GPU."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from oracle import attention, e4m3, rope
from oracle.latent import ROPE, LatentOracle, attend_expanded, encode, row_scale

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_row_scale_is_the_smallest_power_of_two_from_its_least():
    g = np.random.default_rng(0)
    a = np.concatenate([np.exp2(g.uniform(-31, 48, 4000)), 448.0 * np.exp2(np.arange(-40, 41)),
                        np.nextafter(np.float32(448.0), np.float32(1000)) * np.exp2(np.arange(-40, 40))]).astype(np.float32)
    s = row_scale(a)
    assert np.all(np.frexp(s)[0] == 0.5)
    wide = a.astype(np.float64)
    assert np.all(wide <= 448.0 * s) and np.all((wide > 448.0 * (s.astype(np.float64) / 2)) | (s == np.float32(2.0 ** -40)))
    assert np.all(row_scale(np.float32([0.0, 1e-30, 448 * 2.0 ** -41])) == np.float32(2.0 ** -40))
    beyond = np.float32([np.inf, np.nan, np.nextafter(np.float32(448 * 2.0 ** 40), np.float32(np.inf)), 3e38])
    assert np.all(np.isnan(row_scale(beyond)))


def test_codes_are_within_half_a_step_and_marked_rows_are_zeros():
    g = np.random.default_rng(1)
    x = (g.standard_normal((40, 192)) * np.exp2(g.integers(-20, 20, (40, 1)))).astype(np.float32)
    s = row_scale(np.abs(x).max(axis=1))
    v = e4m3.decode(encode(x, s)) * s[:, None]
    assert np.all(np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, s[:, None] * 2.0 ** -10))
    x[3, 5], x[4, 0], x[5, 191] = np.nan, np.inf, 3e38
    s = row_scale(np.abs(x).max(axis=1))
    assert np.isnan(s[3:6]).all() and np.all(encode(x, s)[3:6] == 0) and np.isfinite(np.delete(s, [3, 4, 5])).all()


def _small(new=(3, 1), before=(5, 40), C=128, heads=3, page=16, seed=2):
    g = np.random.default_rng(seed)
    ln = [a + b for a, b in zip(new, before)]
    table = np.arange(8).reshape(2, 4)[:, ::-1]
    o = LatentOracle(C, 8, page)
    x, r = (g.standard_normal((sum(ln), w)).astype(np.float32) for w in (C, ROPE))
    pos = np.concatenate([np.arange(n) for n in ln])[:, None]
    o.append(x, r, pos, np.cumsum([0] + ln), ln, table)
    start = np.cumsum((0,) + new)
    q, qr = (g.standard_normal((sum(new), heads, w)) for w in (C, ROPE))
    qpos = np.concatenate([np.arange(n - a, n) for a, n in zip(new, ln)])[:, None]
    return o, q, qr, qpos, start, ln, table


def test_absorbed_attention_is_plain_attention_over_the_rows():
    o, q, qr, pos, start, ln, table = _small()
    got = o.attend(q, qr, pos, start, ln, table, 0.05).out
    turned = rope.rope_f64(qr, pos, (ROPE,), 10000.0)
    for b in range(2):
        kv = o.rows(table[b], ln[b])
        for i in range(start[b], start[b + 1]):
            n = ln[b] - (start[b + 1] - start[b]) + (i - start[b]) + 1
            x = np.concatenate([q[i], turned[i]], 1)                 # [heads, C + 64]
            k = np.repeat(kv[None, :n], 3, 0)                        # a key head per query head
            want = attention.attend_f64(x[None] * 0.05 * math.sqrt(x.shape[1]), k, k[..., :o.C])[0]
            assert np.allclose(got[i], want, rtol=1e-9, atol=1e-9)


def test_the_two_forms_agree():
    """q . (W c) = (W^T q) . c, and the outputs' expansion likewise."""
    o, _, qr, pos, start, ln, table = _small()
    g = np.random.default_rng(3)
    heads, d = 3, 128
    wk, wv = g.standard_normal((2, heads, d, o.C)) / 10
    qn = g.standard_normal((start[-1], heads, d))
    scale = (d + ROPE) ** -0.5
    absorbed = o.attend(np.einsum("nhd,hdc->nhc", qn, wk), qr, pos, start, ln, table, scale).out
    absorbed = np.einsum("nhc,hdc->nhd", absorbed, wv)
    rows = o.read(np.cumsum([0] + ln), ln, table)
    c, r = rows[:, :o.C], rows[:, o.C:]
    k, v = np.einsum("tc,hdc->thd", c, wk), np.einsum("tc,hdc->thd", c, wv)
    expanded = attend_expanded(np.concatenate([qn, qr], 2), k, r, v, pos, start, [0, ln[0]], ln).out
    assert np.allclose(absorbed, expanded, rtol=1e-10, atol=1e-10)


def test_masks_windows_and_empty_rows():
    o, q, qr, pos, start, ln, table = _small(new=(6, 4), before=(0, 30))
    short = [4, 34]                                          # the first two queries of the first see nothing
    out = o.attend(q, qr, pos, start, short, table, 0.05).out
    assert np.all(out[:2] == 0) and np.all(np.abs(out[2:]).max(axis=(1, 2)) > 0)
    assert np.allclose(out[2], o.rows(table[0], 1)[0, :o.C])            # one key: its value
    wide = o.attend(q, qr, pos, start, ln, table, 0.05, window=100).out
    assert np.array_equal(wide, o.attend(q, qr, pos, start, ln, table, 0.05).out)
    one = o.attend(q, qr, pos, start, ln, table, 0.05, window=1).out
    for i in range(4):
        assert np.allclose(one[6 + i], o.rows(table[1], 34)[30 + i, :o.C])


# ---------------------------------------------------------------- host checks, no GPU
@pytest.fixture(scope="module")
def lib():
    from fp8_ring_kv_gb300 import kvring as K
    if not os.path.exists(K.LIB_PATH):
        from fp8_ring_kv_gb300 import build
        build.build()
    return K.load()


def config(**kw):
    from fp8_ring_kv_gb300.latent import make_latent_config
    base = dict(q_heads=16, latent_dim=512, n_pages=10, page_tokens=64, axis_dims=(64,), pos_min=(0,), pos_count=(1000,))
    fields = {k: kw.pop(k) for k in list(kw) if k not in base}
    c = make_latent_config(**dict(base, **kw))
    for k, v in fields.items():
        setattr(c, k, v)
    return c


def test_workspace_bytes(lib):
    from fp8_ring_kv_gb300.latent import kvring_latent_workspace_bytes as size
    a, b = size(config()), size(config(n_pages=11))
    assert a > 10 * 64 * 576 and 0 < b - a < 2 * 64 * 580 + 4096
    for heads in (1, 256):
        assert size(config(q_heads=heads)) == a
    for dims in ((64,), (16, 24, 24), (2, 62)):
        n = len(dims)
        assert size(config(axis_dims=dims, pos_min=(0,) * n, pos_count=(10,) * n)) > 0


@pytest.mark.parametrize("kw", [dict(q_heads=0), dict(q_heads=257), dict(latent_dim=64), dict(latent_dim=500), dict(latent_dim=640),
                                dict(page_tokens=48), dict(page_tokens=256), dict(n_pages=0), dict(n_pages=1 << 25), dict(layers=0),
                                dict(layers=1 << 22), dict(axis_dims=(128,)), dict(axis_dims=(32,)), dict(in_dtype=2),
                                dict(pos_count=(0,)), dict(rope_base=1.0), dict(n_axes=0)])
def test_bad_configurations(lib, kw):
    from fp8_ring_kv_gb300.latent import kvring_latent_workspace_bytes as size
    assert size(config(**kw)) == 0


def test_null_handles_and_arguments(lib):
    from fp8_ring_kv_gb300 import kvring as K
    p, bad = ctypes.c_void_p(1 << 20), K.KVRING_ERR_INVALID_ARG
    assert lib.kvring_latent_append(None, 0, p, 512, p, 64, p, p, p, 1, 1, p, 1, 1, None) == bad
    assert lib.kvring_latent_read(None, 0, p, p, 1, 1, p, 1, 1, p, 576, None) == bad
    assert lib.kvring_latent_attend(None, 0, p, 512, 512, p, 64, 64, p, p, p, 1, 1, 1, p, 1, 1, 1, 0, 1.0, p, 512, 512, None) == bad
    assert lib.kvring_latent_attend_expanded(None, p, 192, 192, p, 128, 128, p, 64, p, 128, 128, 1, p, p, p, p, 1, 1, 1, 1, 0, 0.0,
                                             p, 128, 128, None) == bad
    assert lib.kvring_latent_layout(None, None, None, None) == bad
    err = ctypes.c_int32()
    assert lib.kvring_latent_debug_state(None, None, ctypes.byref(err)) == bad
    assert lib.kvring_latent_destroy(None) == K.KVRING_OK
    h = ctypes.c_void_p()
    assert lib.kvring_latent_create(ctypes.byref(config()), None, 1 << 30, None, ctypes.byref(h)) == bad and not h.value
    assert lib.kvring_latent_create(ctypes.byref(config()), ctypes.c_void_p((1 << 20) + 64), 1 << 30, None, ctypes.byref(h)) == \
        K.KVRING_ERR_MISALIGNED
    assert lib.kvring_latent_create(ctypes.byref(config()), p, 1 << 10, None, ctypes.byref(h)) == K.KVRING_ERR_WORKSPACE


def test_binding_constants_match_the_header():
    from fp8_ring_kv_gb300 import kvring as K
    text = re.sub(r"/\*.*?\*/", " ", open(os.path.join(ROOT, "include", "kvring_latent.h")).read(), flags=re.S)
    found = dict(re.findall(r"(KVRING_LATENT_[A-Z]+)\s*=\s*(\d+)", text))
    assert set(found) == {"KVRING_LATENT_ROPE", "KVRING_LATENT_HEAD"}
    for name, value in found.items():
        assert getattr(K, name) == int(value)


def test_unknown_types_are_refused():
    from fp8_ring_kv_gb300.kvring import KVRingError
    from fp8_ring_kv_gb300.latent import make_latent_config
    with pytest.raises(KVRingError, match="float32"):
        make_latent_config(1, 128, 1, 16, (64,), (0,), (1,), dtype=torch.float32)
    with pytest.raises(KVRingError, match="axes"):
        make_latent_config(1, 128, 1, 16, (16, 16, 16, 16), (0,) * 4, (1,) * 4)
