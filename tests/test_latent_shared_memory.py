"""Shared memory that changes hands in the latent kernels, read from their sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_ring_kv_gb300", "csrc")


@pytest.mark.parametrize("name", ["latent_attend.cu", "latent_expanded.cu"])
def test_room_of_the_prefix_sums_is_fenced_before_tma_writes_there(name):
    """Ordinary accesses are not ordered before TMA's by a barrier alone: after the last
    read of the prefix sums every thread fences, then the block meets."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    after = text[text.index("find_place<"):]
    before_barrier = after[:after.index("__syncthreads();")]
    assert re.search(r"\n  fence_proxy_async_smem\(\);\s*$", before_barrier)
