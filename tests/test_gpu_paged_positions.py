"""Positions at the ends of their 32 bits: outside the tables they are clamped and
flagged, however far."""
import numpy as np
import pytest
import torch

from oracle.paged import PagedOracle
from test_gpu_paged import BF, cu, paged

pytestmark = pytest.mark.gpu

LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("axis_dims", [(128,), (32, 48, 48), (12, 68, 48)])   # whole lanes, three axes, odd places
@pytest.mark.parametrize("pos_min", [LOW, -5, 0, 7, HIGH - 20])
@pytest.mark.parametrize("n", [3, 40])
def test_positions_outside_the_tables(n, pos_min, axis_dims):
    from fp8_ring_kv_gb300 import kvring as K
    count, axes = 50, len(axis_dims)
    last = min(pos_min + count - 1, HIGH)                     # of the table and of 32 bits
    kv = paged(1, 2, 128, 4, 32, axis_dims, (pos_min,) * axes, (count,) * axes)
    oracle = PagedOracle(1, 128, 4, 32, axis_dims)
    g = np.random.default_rng(3)
    x = lambda rows, heads: torch.from_numpy(g.standard_normal((rows, heads, 128)).astype(np.float32)).to(BF)
    table, start, ln = cu(np.arange(4, dtype=np.int32)[None]), cu(np.array([0, n], np.int32)), cu(np.array([n], np.int32))

    def call(pos):
        k, v = x(n, 1), x(n, 1)
        kv.append(k.cuda(), v.cuda(), cu(pos), start, ln, table)
        err = kv.debug_state()
        kv.workspace[:4].zero_()
        oracle.append(k.float().numpy(), v.float().numpy(), np.clip(pos.astype(np.int64), pos_min, last), [0, n], [n], np.arange(4)[None])
        assert np.array_equal(kv.k_codes[0].cpu().numpy(), oracle.codes["k"])
        kv.attend(x(n, 2).cuda(), cu(pos), start, ln, table)
        assert kv.debug_state() == err
        kv.workspace[:4].zero_()
        return err

    inside = g.integers(pos_min, last + 1, (n, axes)).astype(np.int32)
    assert call(inside) == 0
    for far in (LOW, HIGH, pos_min - 1, last + 1, pos_min + 2 ** 31, pos_min - 2 ** 31):
        if LOW <= far <= HIGH and not pos_min <= far <= last:
            pos = inside.copy()
            pos[n // 2, -1] = far
            assert call(pos) == K.KVRING_DEVERR_POS_RANGE, far
