"""The paged cache's kernels give the same bits every time: first calls on fresh
caches whose workspace held something else, and calls that follow one another
without a pause."""
import numpy as np
import pytest
import torch

from test_gpu_paged import BF, HF, Case, cu, paged

pytestmark = pytest.mark.gpu


def first_call(c, how, times, pattern):
    """``times`` fresh caches in one workspace, each filled with a byte pattern
    before: two appends and the first attention.  The outputs of the first, all
    others compared with them bit for bit; the error word before the outputs."""
    from fp8_ring_kv_gb300.paged import kvring_paged_workspace_bytes, make_paged_config
    shape = (c.kv_heads, c.q_heads, c.dim, c.n_pages, c.page, c.axis_dims, (0,) * len(c.axis_dims), c.pos_count)
    ws = torch.empty(kvring_paged_workspace_bytes(make_paged_config(*shape, dtype=c.dtype)), dtype=torch.uint8, device="cuda")
    half = [n // 2 for n in c.len]
    calls = []
    for seqs in ([(n, 0) for n in half], [(n - a, a) for n, a in zip(c.len, half)]):
        start, ln, pos = c.batch(seqs)
        k, v = c.draw(int(start[-1]), c.kv_heads), c.draw(int(start[-1]), c.kv_heads)
        calls.append([x.cuda() for x in (k, v)] + [cu(x) for x in (pos, start, ln)])
        c.oracle.append(k.float().numpy(), v.float().numpy(), pos, start, ln, c.table)
    start, ln, pos = c.batch(c.seqs)
    q = c.draw(c.n, c.q_heads)
    args, table, qd = [cu(x) for x in (pos, start, ln)], cu(c.table), q.cuda()
    first = None
    for i in range(times):
        ws.fill_(pattern[i % len(pattern)])
        kv = paged(*shape, dtype=c.dtype, workspace=ws)
        for x in calls:
            kv.append(*x, table)
        if i % 2:
            torch.cuda.synchronize()
        out = torch.full((c.n, c.q_heads, c.dim), 7.0, dtype=c.dtype, device="cuda")
        kv.attend(qd, *args, table, out=out, **how)
        assert kv.debug_state() == 0
        if first is None:
            first = out
            c.kv = kv
            c.check_cache()
            c.check_out(out, *c.oracle.attend(q.float().numpy(), pos, start, ln, c.table, how.get("causal", True), how.get("window") or 0))
        else:
            bad = (out.view(torch.int16) != first.view(torch.int16)).nonzero()
            assert len(bad) == 0, f"call {i}: {len(bad)} elements differ, first {bad[:6].tolist()}"


@pytest.mark.parametrize("window", [200, None])
@pytest.mark.parametrize("dtype,dim", [(BF, 128), (HF, 128), (BF, 64), (HF, 64)])
def test_first_calls_on_fresh_caches(dtype, dim, window):
    """Chunks of 520 and 64 tokens, 8 query heads per key head: pieces of two key
    tiles, some of whose workers have none; the next product over the weights of
    the one before."""
    c = Case([(520, 0), (64, 1000)], kv_heads=2, group=8, page=64, dim=dim, dtype=dtype)
    first_call(c, dict(window=window), 300, (0xFF, 0xA5, 0x00, 0x7F))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_first_calls_of_few_rows(dtype):
    c = Case([(1, 900), (3, 200), (2, 0), (1, 3000), (4, 77)], kv_heads=2, group=8, page=16, dtype=dtype)
    first_call(c, {}, 200, (0xFF, 0xA5, 0x00, 0x7F))
