"""Refusals of the paged cache's C entry points, beside those of the wrapper."""
import pytest

from test_gpu_paged import paged

pytestmark = pytest.mark.gpu


def test_a_scale_beyond_fp32_is_refused():
    """scale * log2(e) is what the kernels multiply by: infinite from 2^128 / log2(e) on."""
    from fp8_ring_kv_gb300 import kvring as K
    kv = paged(1, 1, 64, 2, 16, (64,), (0,), (8,))
    p = kv.workspace.data_ptr()                              # never read: the call is refused
    for scale in (3.0e38, 2.4e38):
        args = [kv.handle, 0, p, 64, p, p, p, 1, 1, 1, p, 2, 2, 1, 0, scale, p, 64, None]
        assert K.load().kvring_paged_attend(*args) == K.KVRING_ERR_INVALID_ARG
    assert kv.debug_state() == 0
