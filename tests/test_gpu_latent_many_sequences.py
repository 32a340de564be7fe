"""Calls of very many sequences: the kernels' sums over them lie where the first codes
come to lie."""
import numpy as np
import pytest
import torch

import latent_bounds
from test_gpu_latent import BF, HF, KIND, SCALE, ROPE, Case, check, cu, num

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,heads", [(BF, 64), (BF, 3), (HF, 20)])
def test_many_sequences_again_and_again(dtype, heads):
    c = Case([(1, 1 + i % 150) for i in range(2048)], heads=heads, latent=128, page=16, dtype=dtype)
    c.fill(1)
    c.check_cache()
    start, ln, pos = c.batch(c.seqs)
    q, qr = c.draw(c.n, heads, 128), c.draw(c.n, heads, ROPE)
    args = [q.cuda(), qr.cuda()] + [cu(x) for x in (pos, start, ln, c.table)]
    outs = [c.kv.attend(*args, SCALE, max_new=1) for _ in range(30)]
    assert all(bool((o == outs[0]).all()) for o in outs[1:])
    some = np.r_[0:64, 1000:1064, 1984:2048]
    r = c.oracle.attend(num(q[some]), num(qr[some]), pos[some], np.arange(len(some) + 1), ln[some], c.table[some], SCALE)
    check(outs[0][torch.from_numpy(some).cuda()], r, latent_bounds.absorbed(r, KIND[dtype]))
    assert c.kv.debug_state() == 0
