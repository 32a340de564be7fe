"""The paged cache's numpy oracle, pinned by closed forms and by the ring's own
oracles; and the library's host-side checks that need no GPU."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from oracle import attention, e4m3, rope
from oracle.paged import PagedOracle, encode, pow2_scale

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_block_scale_is_the_smallest_power_of_two():
    g = np.random.default_rng(0)
    a = np.concatenate([np.exp2(g.uniform(-99, 120, 4000)), 448.0 * np.exp2(np.arange(-100, 118)),
                        np.nextafter(np.float32(448.0), np.float32(1000)) * np.exp2(np.arange(-90, 100))]).astype(np.float32)
    s = pow2_scale(a)
    m, _ = np.frexp(s)
    assert np.all(m == 0.5)                                  # powers of two
    wide = a.astype(np.float64)
    assert np.all(wide <= 448.0 * s) and np.all(wide > 448.0 * (s.astype(np.float64) / 2))
    assert np.all(pow2_scale(np.float32([0.0, 2.0 ** -101, 1e-38])) == 0)
    assert pow2_scale(np.float32(2.0) ** -100) > 0


def test_codes_are_within_half_a_step():
    g = np.random.default_rng(1)
    x = (g.standard_normal((5, 7, 64)) * np.exp2(g.integers(-20, 20, (5, 1, 1)))).astype(np.float32)
    s = pow2_scale(np.abs(x).max(axis=(1, 2)))
    v = e4m3.decode(encode(x, s)) * s[:, None, None]
    step = np.maximum(np.abs(x) * 2.0 ** -4, s[:, None, None] * 2.0 ** -10)
    assert np.all(np.abs(v - x) <= step)


@pytest.mark.parametrize("pieces", [1, 2, 7, 40])
def test_how_a_page_was_filled_hardly_matters(pieces):
    """Scales are powers of two, so a code that stays normal is carried over
    exactly: the cache is the same however many calls filled it, but for half a
    step of the subnormals at the final scale."""
    g = np.random.default_rng(2)
    n, h, d, p = 40, 2, 64, 16
    x = (g.standard_normal((n, h, d)) * np.exp2(g.uniform(-6, 6, (n, 1, 1)))).astype(np.float32)
    pos = np.arange(n)[:, None]
    table = np.arange(3)[None]
    whole, parts = PagedOracle(h, d, 3, p, (d,)), PagedOracle(h, d, 3, p, (d,))
    whole.append(x, x, pos, [0, n], [n], table)
    cut = [n * i // pieces for i in range(pieces + 1)]
    for a, b in zip(cut, cut[1:]):
        parts.append(x[a:b], x[a:b], pos[a:b], [0, b - a], [b], table)
    for name in "kv":
        assert np.array_equal(whole.scales[name], parts.scales[name])
        s = whole.scales[name].astype(np.float64)[..., None, None]
        diff = np.abs(e4m3.decode(whole.codes[name]) - e4m3.decode(parts.codes[name])) * s
        assert np.all(diff <= s * 2.0 ** -9)
        normal = np.abs(e4m3.decode(whole.codes[name])) >= 2.0 ** -5
        assert np.all(diff[normal] == 0)


def _filled(seed=3, n=50, h=2, d=64, p=16):
    g = np.random.default_rng(seed)
    o = PagedOracle(h, d, 8, p, (d,))
    x = g.standard_normal((2, n, h, d)).astype(np.float32)
    table = g.permutation(8)[None, :(n + p - 1) // p]
    o.append(x[0], x[1], np.arange(n)[:, None], [0, n], [n], table)
    return o, x, table


def test_attention_is_the_dense_one_over_the_cached_rows():
    o, x, table = _filled()
    g = np.random.default_rng(4)
    q = g.standard_normal((50, 4, 64)).astype(np.float32)
    pos = np.arange(50)[:, None]
    k = np.stack([o.rows("k", table[0], 50, h // 2) for h in range(4)])
    v = np.stack([o.rows("v", table[0], 50, h // 2) for h in range(4)])
    out, spread, logit = o.attend(q, pos, [0, 50], [50], table, causal=False)
    want = attention.attend_f64(rope.rope_f64(q, pos, (64,), 10000.0), k, v)
    assert np.abs(out - want).max() < 1e-12
    assert np.all(spread >= np.abs(out) - 1e-12) and np.all(logit > 0)
    # causal and a window: each row is the dense attention over what it sees
    out, _, _ = o.attend(q, pos, [0, 50], [50], table, causal=True, window=7)
    for i in (0, 3, 6, 7, 49):
        lo = max(0, i - 6)
        want = attention.attend_f64(rope.rope_f64(q[i:i + 1], pos[i:i + 1], (64,), 10000.0), k[:, lo:i + 1], v[:, lo:i + 1])
        assert np.abs(out[i] - want[0]).max() < 1e-12
    # a row that sees nothing
    out, _, _ = o.attend(q[:3], pos[:3], [0, 3], [1], table)
    assert np.all(out[:2] == 0) and np.any(out[2] != 0)


def test_equal_keys_average_the_values():
    o = PagedOracle(1, 64, 4, 16, (64,))
    v = np.random.default_rng(5).standard_normal((20, 1, 64)).astype(np.float32)
    o.append(np.zeros((20, 1, 64), np.float32), v, np.arange(20)[:, None], [0, 20], [20], [[2, 0]])
    out, _, _ = o.attend(np.ones((1, 1, 64), np.float32), [[5]], [0, 1], [20], [[2, 0]])
    assert np.abs(out[0, 0] - o.rows("v", [2, 0], 20, 0).mean(axis=0)).max() < 1e-12


# ---------------------------------------------------------------- the library without a GPU
@pytest.fixture(scope="module")
def K():
    from fp8_ring_kv_gb300 import kvring
    if not os.path.exists(kvring.LIB_PATH):
        from fp8_ring_kv_gb300 import build
        build.build()
    kvring.load()
    return kvring


def config(**kw):
    from fp8_ring_kv_gb300.paged import make_paged_config
    args = dict(kv_heads=8, q_heads=32, head_dim=128, n_pages=100, page_tokens=64, axis_dims=(128,), pos_min=(0,),
                pos_count=(8192,))
    fields = {k: kw.pop(k) for k in list(kw) if k not in args and k not in ("rope_base", "dtype", "layers")}
    c = make_paged_config(**dict(args, **kw))
    for k, v in fields.items():
        setattr(c, k, v)
    return c


def size(c):
    from fp8_ring_kv_gb300.paged import kvring_paged_workspace_bytes
    return kvring_paged_workspace_bytes(c)


def test_workspace_bytes(K):
    n = size(config())
    codes = 2 * 100 * 8 * 64 * 128
    assert n > codes + 2 * 100 * 8 * 4 + 8192 * 64 * 8 and n % 1024 == 0
    assert size(config(layers=3)) >= n + 2 * codes
    assert size(config(dtype=torch.float16)) == n
    assert size(config(axis_dims=(32, 48, 48), pos_min=(-5, 0, 0), pos_count=(64, 8, 8))) > codes


@pytest.mark.parametrize("kw", [
    dict(kv_heads=0), dict(kv_heads=129, q_heads=129), dict(q_heads=20), dict(q_heads=1032), dict(q_heads=0), dict(head_dim=96),
    dict(head_dim=256), dict(n_pages=0), dict(n_pages=-1), dict(n_pages=1 << 22), dict(page_tokens=8), dict(page_tokens=48),
    dict(page_tokens=256), dict(layers=0), dict(layers=1 << 30, n_pages=1 << 30), dict(axis_dims=(64,)), dict(axis_dims=(126, 1)),
    dict(axis_dims=(-2147483520,)), dict(pos_count=(0,)), dict(pos_count=((1 << 24) + 1,)), dict(rope_base=1.0),
    dict(rope_base=math.inf), dict(rope_base=math.nan), dict(in_dtype=2), dict(n_axes=0), dict(n_axes=4),
])
def test_invalid_configurations(K, kw):
    if len(kw.get("axis_dims", (0,))) == 2:
        kw = dict(kw, pos_min=(0, 0), pos_count=(4, 4))
    assert size(config(**kw)) == 0


def test_configuration_in_python(K):
    with pytest.raises(K.KVRingError, match="float32"):
        config(dtype=torch.float32)
    with pytest.raises(K.KVRingError, match="axes"):
        config(pos_min=(0, 0))


def test_create_and_null_handles(K):
    lib, c, h = K.load(), config(), ctypes.c_void_p()
    need, at = size(c), ctypes.c_void_p
    # the addresses are never used: each case fails a host check first
    ref, out = ctypes.byref(c), ctypes.byref(h)
    assert lib.kvring_paged_create(None, at(1 << 20), need, None, out) == K.KVRING_ERR_INVALID_ARG
    assert lib.kvring_paged_create(ref, None, need, None, out) == K.KVRING_ERR_INVALID_ARG
    assert lib.kvring_paged_create(ref, at((1 << 20) + 16), need, None, out) == K.KVRING_ERR_MISALIGNED
    assert lib.kvring_paged_create(ref, at(1 << 20), need - 1, None, out) == K.KVRING_ERR_WORKSPACE
    assert lib.kvring_paged_create(ref, at(1 << 20), need, None, None) == K.KVRING_ERR_INVALID_ARG
    assert h.value is None
    p = 1 << 20
    assert lib.kvring_paged_append(None, 0, p, 1024, p, 1024, p, p, p, 1, 1, p, 4, 4, None) == K.KVRING_ERR_INVALID_ARG
    assert lib.kvring_paged_attend(None, 0, p, 4096, p, p, p, 1, 1, 1, p, 4, 4, 1, 0, 0.0, p, 4096, None) \
        == K.KVRING_ERR_INVALID_ARG
    assert lib.kvring_paged_destroy(None) == K.KVRING_OK
    assert lib.kvring_paged_layout(None, None, None, None, None, None) == K.KVRING_ERR_INVALID_ARG
    err = ctypes.c_int32()
    assert lib.kvring_paged_debug_state(None, None, ctypes.byref(err)) == K.KVRING_ERR_INVALID_ARG


def test_constants_match_the_header(K):
    text = open(os.path.join(ROOT, "include", "kvring_paged.h")).read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    found = {}
    for body in re.findall(r"enum\s*\{(.*?)\}", text, flags=re.S):
        for name, value in re.findall(r"(KVRING_[A-Z0-9_]+)\s*=\s*([\d <]+)", body):
            found[name] = eval(value)
    assert len(found) == 6
    for name, value in found.items():
        assert getattr(K, name) == value, name


def _shell():
    """A PagedKV without a device: its checks alone (CPU tensors have device index -1)."""
    from fp8_ring_kv_gb300.paged import PagedKV
    kv = object.__new__(PagedKV)
    kv.handle, kv.layers, kv.kv_heads, kv.q_heads, kv.head_dim = ctypes.c_void_p(1), 2, 2, 4, 64
    kv.page_tokens, kv.n_axes, kv.dtype, kv._index = 16, 1, torch.bfloat16, -1
    return kv


def test_the_wrappers_checks(K):
    kv = _shell()
    try:
        t = torch.zeros((5, 8, 64), dtype=torch.bfloat16)
        assert kv._row_stride(t[:, 2:4], 5, 2, "k") == 512
        assert kv._row_stride(t[:1, 2:4], 1, 2, "k") == 128
        assert kv._row_stride(t[:0, 2:4], 0, 2, "k") == 128
        for bad, n, heads, why in ((t.float(), 5, 8, "float32"), (t, 4, 8, "shape"), (t.transpose(0, 1), 8, 5, "strides"),
                                   (t[:, ::2], 5, 4, "strides"), (t[:, :, ::2], 5, 8, "shape"),
                                   (t[:, :2].expand(5, 2, 64)[:1].expand(5, 2, 64), 5, 2, "strides")):
            with pytest.raises(K.KVRingError, match=why):
                kv._row_stride(bad, n, heads, "k")
        ints = dict(pos=torch.zeros((5, 1), dtype=torch.int32), pos_name="pos", seq_start=torch.zeros(3, dtype=torch.int32),
                    kv_len=torch.zeros(2, dtype=torch.int32), page_table=torch.zeros((2, 4), dtype=torch.int32))
        *_, n_seqs, _, stride, width = kv._batch(0, 5, **ints)
        assert (n_seqs, stride, width) == (2, 4, 4)
        wide = torch.zeros((2, 9), dtype=torch.int32)[:, 3:7]
        assert kv._batch(1, 5, **dict(ints, page_table=wide))[-2:] == (9, 4)
        for change, why in ((dict(pos=ints["pos"].long()), "int64"), (dict(seq_start=torch.zeros(2, dtype=torch.int32)), "shape"),
                            (dict(kv_len=torch.zeros(4, dtype=torch.int32)[::2]), "contiguous"),
                            (dict(page_table=wide.t()), "strides|shape"), (dict(page_table=wide[0]), "shape"),
                            (dict(page_table=wide.long()), "int64")):
            with pytest.raises(K.KVRingError, match=why):
                kv._batch(0, 5, **dict(ints, **change))
        for layer in (-1, 2):
            with pytest.raises(K.KVRingError, match="layer"):
                kv._batch(layer, 5, **ints)
        kv._index = 0
        with pytest.raises(K.KVRingError, match="cpu"):
            kv._batch(0, 5, **ints)
        with pytest.raises(K.KVRingError, match="cpu"):
            kv._row_stride(t, 5, 8, "k")
    finally:
        kv.handle = None
