"""Absorbed latent attention on rows where one key has most of the weight and
thousands of others share the rest: what the small weights add up to stays in the
output, whether a context is one piece or cut into many."""
import numpy as np
import pytest
import torch

from latent_bounds import U
from oracle.latent import ROPE, LatentOracle

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
SCALE = 192 ** -0.5
# share of the one key, spread of the others' logits
HEADS = [(at, share, sd) for at in range(3) for share in (0.6, 0.9) for sd in (0.1, 1.4)]


class Peaked:
    """A context whose first, middle and last keys have a channel of their own each,
    where a query finds it; the others' channels have a mean in common."""

    def __init__(self, keys, latent, dtype, kind, page=64, seed=0):
        self.keys, self.C, self.dtype = keys, latent, dtype
        self.g = g = np.random.default_rng(seed)
        x = g.standard_normal(latent) + 0.5 * g.standard_normal((keys, latent))
        x[:, :3] = 0
        ones = (0, keys // 2, keys - 1)
        for i, t in enumerate(ones):
            if kind == "empty":                              # next to no value beside its own channel
                x[t] /= 64
            x[t, i] = 3.0
        self.latent = torch.from_numpy(x.astype(np.float32)).to(dtype)
        pages = (keys + page - 1) // page
        self.table = g.permutation(pages).astype(np.int32)[None]
        self.start, self.len = np.array([0, keys], np.int32), np.array([keys], np.int32)
        self.oracle = LatentOracle(latent, pages, page)
        zero = np.zeros((keys, 1), np.int32)
        self.oracle.append(self.latent.float().numpy(), np.zeros((keys, ROPE), np.float32), zero, self.start, self.len, self.table)
        rows = self.oracle.rows(self.table[0], keys)
        self.q = torch.zeros(1, len(HEADS), latent)
        for h, (at, share, sd) in enumerate(HEADS):
            q = g.standard_normal(latent) * sd / (SCALE * 0.5 * (latent - 3) ** 0.5)
            q[:3] = 0
            z = SCALE * rows[:, :latent] @ q
            most = np.delete(z, ones[at]).max()
            rest = most + np.log(np.exp(np.delete(z, ones[at]) - most).sum())
            q[at] = (np.log(share / (1 - share)) + rest - z[ones[at]]) / (SCALE * rows[ones[at], at])
            # 8 significant bits of at least 2^-9.8 of the largest: exact as two e4m3 numbers
            q[np.abs(q) < np.abs(q).max() * 2.0 ** -9.8] = 0
            self.q[0, h] = torch.from_numpy(q.astype(np.float32)).bfloat16().float()
        self.q = self.q.to(dtype)
        self.want = self.oracle.attend(self.q.float().numpy(), np.zeros((1, len(HEADS), ROPE)), [[0]], [0, 1], self.len, self.table,
                                       SCALE)

    def bound(self):
        """A weight is a sum of parts of 3 + 3 + 3 bits (bf16), each off by half a step:
        2^-9 of it, behind a rounding to fp16, 2^-11; of 4 + 3 + 4 + 3 bits (fp16), 2^-14,
        and 2^-15 for what fp16 leaves.  The last part's smallest step: half of it is 2^-17
        where the largest weight is 3584 at least, 2^-21 where it is 112.  Logits: exact
        queries, fp32 sums (2^-18 of the terms), and their effect on the weight and on the
        sum of weights; 2^-16 for sums over the keys.  Then the output's own rounding."""
        r, half = self.want, self.dtype is HF
        weight = 2.0 ** -14 + 2.0 ** -15 if half else 2.0 ** -9 + 2.0 ** -11
        floor = 2.0 ** -21 / 112 if half else 2.0 ** -17 / 3584
        u = U["f16" if half else "bf16"]
        err = r.spread * (np.expm1(2.0 ** -17 * r.all)[..., None] + weight + 2.0 ** -16) + r.floor * floor
        return err * (1 + u) + np.abs(r.out) * u + (2.0 ** -24 if half else 1e-30)

    def attend(self, heads, seqs):
        from fp8_ring_kv_gb300 import LatentKV
        cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        kv = LatentKV(heads, self.C, self.table.shape[1], 64, (ROPE,), (0,), (1,), dtype=self.dtype)
        kv.append(self.latent.cuda(), torch.zeros(self.keys, ROPE, dtype=self.dtype, device="cuda"), cu(np.zeros((self.keys, 1), np.int32)),
                  cu(self.start), cu(self.len), cu(self.table))
        order = [h % len(HEADS) for h in range(heads)]
        q = self.q[:, order].expand(seqs, -1, -1).cuda().contiguous()
        out = kv.attend(q, torch.zeros(seqs, heads, ROPE, dtype=self.dtype, device="cuda"), torch.zeros(seqs, 1, dtype=torch.int32, device="cuda"),
                        torch.arange(seqs + 1, dtype=torch.int32, device="cuda"), cu(self.len).expand(seqs).contiguous(),
                        cu(self.table).expand(seqs, -1).contiguous(), SCALE, max_new=1)
        assert kv.debug_state() == 0
        return out, order


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", ["empty", "full"])
@pytest.mark.parametrize("keys,latent", [(2500, 512), (8192, 512), (32768, 256)])
def test_small_weights_beside_a_large_one(keys, latent, kind, dtype):
    c = Peaked(keys, latent, dtype, kind)
    bound = c.bound()
    # a few roundings of the output, however many keys there are
    assert np.all(bound.mean(axis=2) <= 3 * U["bf16" if keys > 10000 or dtype is BF else "f16"] * c.want.spread.mean(axis=2))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for heads in (64, 32):
        # as many items as there are blocks, none of them cut; and one context cut for all blocks
        for seqs in (sms // 2 if heads == 64 and dtype is HF else sms, 1):
            out, order = c.attend(heads, seqs)
            assert bool((out == out[:1]).all())
            err = np.abs(out[0].double().cpu().numpy() - c.want.out[0, order])
            worst = (err / bound[0, order]).max(axis=1)
            h = int(worst.argmax())
            assert worst[h] <= 1.0, f"{heads} heads, {seqs} sequences: {worst[h]:.2f} of the bound at {HEADS[order[h]]}"
