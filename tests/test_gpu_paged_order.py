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


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("page,dim", [(16, 64), (64, 128)])
def test_steps_without_a_pause(page, dim, new):
    """Append and attention step after step, every step's values twice those of
    the step before, so that page scales grow and codes are rounded again while
    the next kernels are already waiting: the outputs and the cache of the same
    steps with a pause after each kernel."""
    steps = 24
    c = Case([(0, 30 + steps * new), (0, 5 + steps * new), (0, 300 + steps * new)], kv_heads=4, group=4, page=page, dim=dim)
    table = cu(c.table)
    have, work = [30, 5, 300], []
    first = c.batch([(n, 0) for n in have])
    prompt = [c.draw(int(first[0][-1]), 4).cuda() for _ in range(2)] + [cu(x) for x in (first[2], first[0], first[1])]
    for step in range(steps):
        start, ln, pos = c.batch([(new, n) for n in have])
        have = [n + new for n in have]
        k, v, q = (c.draw(3 * new, h) for h in (4, 4, 16))
        grow = 2.0 ** (step - 12)
        work.append([(x * s).cuda() for x, s in ((k, grow), (v, grow), (q, 1.0))] + [cu(x) for x in (pos, start, ln)])
    got = []
    for pause in (True, False, False, False):
        c.kv.workspace[c.kv.k_codes.data_ptr() - c.kv.workspace.data_ptr():].zero_()   # an empty cache
        wait = torch.cuda.synchronize if pause else lambda: None
        wait()
        c.kv.append(*prompt, table)
        outs = []
        for k, v, q, pos, start, ln in work:
            wait()
            c.kv.append(k, v, pos, start, ln, table)
            wait()
            outs.append(c.kv.attend(q, pos, start, ln, table, max_new=new))
        torch.cuda.synchronize()
        assert c.kv.debug_state() == 0
        got.append(outs + [c.kv.k_codes.clone(), c.kv.v_codes.clone(), c.kv.k_scales.clone(), c.kv.v_scales.clone()])
    for other in got[1:]:
        for i, (a, b) in enumerate(zip(got[0], other)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i


@pytest.mark.parametrize("raw", [False, True])
def test_a_cache_made_on_another_stream(raw):
    """Its workspace is not a block that the current stream's queued work still
    writes to."""
    from fp8_ring_kv_gb300.paged import kvring_paged_workspace_bytes, make_paged_config
    c = Case([(30, 100), (1, 50)], kv_heads=2, group=4)
    shape = (2, 8, 128, c.n_pages, c.page, c.axis_dims, (0,), c.pos_count)
    start, ln, pos = c.batch([(n, 0) for n in c.len])
    k, v = c.draw(int(start[-1]), 2), c.draw(int(start[-1]), 2)
    c.oracle.append(k.float().numpy(), v.float().numpy(), pos, start, ln, c.table)
    side = torch.cuda.Stream()
    args = [k.cuda(), v.cuda()] + [cu(x) for x in (pos, start, ln, c.table)]
    block = torch.empty(kvring_paged_workspace_bytes(make_paged_config(*shape)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                            # some 0.1 s
    block.fill_(0xFF)
    del block
    c.kv = paged(*shape, stream=side.cuda_stream if raw else side)
    c.kv.append(*args, stream=side)
    torch.cuda.synchronize()
    c.check_cache()
    q = c.draw(c.n, 8)
    start, ln, pos = c.batch(c.seqs)
    out = c.kv.attend(q.cuda(), cu(pos), cu(start), cu(ln), cu(c.table))
    c.check_out(out, *c.oracle.attend(q.float().numpy(), pos, start, ln, c.table))
    assert c.kv.debug_state() == 0


def test_the_default_streams_handle():
    """A raw handle of 0 is the default stream, also for the memory of outputs."""
    from fp8_ring_kv_gb300.paged import _as_stream
    default, side = torch.cuda.default_stream(), torch.cuda.Stream()
    assert default.cuda_stream == 0
    for device in ("cuda", torch.device("cuda", torch.cuda.current_device())):
        assert _as_stream(0, device) == default and _as_stream(default, device) == default
        assert _as_stream(side.cuda_stream, device).cuda_stream == side.cuda_stream
        assert _as_stream(side, device) is side
    c = Case([(3, 40)], group=4)
    c.fill(1)
    start, ln, pos = c.batch(c.seqs)
    q = c.draw(c.n, c.q_heads)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        out = c.kv.attend(q.cuda(), cu(pos), cu(start), cu(ln), cu(c.table), stream=0)
    torch.cuda.synchronize()
    c.check_out(out, *c.oracle.attend(q.float().numpy(), pos, start, ln, c.table))
