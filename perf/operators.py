"""The paged FP8 KV cache's operators as a set of measured cases.

Two operators: appending keys and values to a paged cache (rotation on the
way, e4m3 codes, one power-of-two scale per page and head), and the attention
that reads that cache.  ``listed()`` names the cases, ``draw()`` makes more of
the same ranges, ``prepare()`` builds the inputs of one, ``run()`` makes one
pass: the plain form in elementary torch operations, or, with ``own`` true, the
calls of ``fp8_ring_kv_gb300.paged``.  ``exact()`` is the definition in 64 bits.

Definitions.  Sequence b has ``new[b]`` new tokens (rows start[b] ..
start[b+1]-1 of the packed inputs) and ``length[b]`` tokens in the cache once
they are in; token i of it has cache index t = length[b] - new[b] + i, in page
table[b, t // P] at row t % P.

append: K is rotated by RoPE at the token's positions (interleaved pairs,
fp32), V is not.  A page's scale for a head is the smallest power of two s with
amax <= 448 s over the rows of the page (0 when amax < 2^-100); a page that
already holds rows keeps its scale unless the new rows need a larger one, and
its older codes are then rounded again at that scale.  Codes are
e4m3(x / s), round to nearest even.

attend: query row i of head h attends over t < length[b] (causal: t <= its own
index; window w: the last w of those):
out = sum_t softmax_t(q . k_t / sqrt(D)) v_t with q rotated, k and v the
cache's dequantised rows; a row that sees nothing gives zeros.
"""
import math

import torch

own = False

ROPE_BASE = 10000.0
FRAME = 96          # three-axis positions: frames of 8 x 12 tokens
GOLDEN = 0.6180339887498949


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence decodes one token: the latency of the smallest write
        dict(name="append_one", op="append", seqs=1, new_lo=1, new_hi=1, ctx_lo=1000, ctx_hi=1000, q_heads=8,
             kv_heads=8, head_dim=128, page=64, axes=1, dtype="bf16", causal=True, window=0),
        # a decoding batch writes one token per sequence into half-filled pages
        dict(name="append_batch", op="append", seqs=128, new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=2000, q_heads=8,
             kv_heads=8, head_dim=128, page=64, axes=1, dtype="bf16", causal=True, window=0),
        # prompts of several users, ragged, each continuing inside a page
        dict(name="append_prompts", op="append", seqs=7, new_lo=37, new_hi=5000, ctx_lo=1, ctx_hi=300, q_heads=8,
             kv_heads=8, head_dim=128, page=64, axes=1, dtype="bf16", causal=True, window=0),
        # two video frames' worth of tokens, three position axes, small pages
        dict(name="append_frames", op="append", seqs=2, new_lo=757, new_hi=757, ctx_lo=757, ctx_hi=1514, q_heads=24,
             kv_heads=24, head_dim=64, page=16, axes=3, dtype="f16", causal=True, window=0),
        # one short conversation decodes one token
        dict(name="decode_one", op="attend", seqs=1, new_lo=1, new_hi=1, ctx_lo=776, ctx_hi=776, q_heads=32,
             kv_heads=8, head_dim=128, page=64, axes=1, dtype="bf16", causal=True, window=0),
        # a decoding batch of ragged contexts
        dict(name="decode_batch", op="attend", seqs=64, new_lo=1, new_hi=1, ctx_lo=200, ctx_hi=8000, q_heads=32,
             kv_heads=8, head_dim=128, page=64, axes=1, dtype="bf16", causal=True, window=0),
        # two very long contexts: few rows, the cache split along its length
        dict(name="decode_long", op="attend", seqs=2, new_lo=1, new_hi=1, ctx_lo=100001, ctx_hi=131000, q_heads=64,
             kv_heads=8, head_dim=128, page=128, axes=1, dtype="bf16", causal=True, window=0),
        # one key head per query head, small pages and heads
        dict(name="decode_heads", op="attend", seqs=32, new_lo=1, new_hi=1, ctx_lo=500, ctx_hi=3000, q_heads=16,
             kv_heads=16, head_dim=64, page=16, axes=1, dtype="f16", causal=True, window=0),
        # a scheduler's step: prompt chunks and a few drafted tokens together, a sliding window
        dict(name="mixed_window", op="attend", seqs=9, new_lo=2, new_hi=301, ctx_lo=0, ctx_hi=6000, q_heads=32,
             kv_heads=4, head_dim=128, page=32, axes=1, dtype="bf16", causal=True, window=1024),
        # whole prompts, causal
        dict(name="prompts", op="attend", seqs=3, new_lo=1000, new_hi=4096, ctx_lo=0, ctx_hi=0, q_heads=32,
             kv_heads=8, head_dim=128, page=64, axes=1, dtype="bf16", causal=True, window=0),
        # a chunk of a long prompt over what is already cached
        dict(name="chunk_long", op="attend", seqs=1, new_lo=512, new_hi=512, ctx_lo=65000, ctx_hi=65000, q_heads=32,
             kv_heads=8, head_dim=128, page=64, axes=1, dtype="bf16", causal=True, window=0),
        # a video chunk: 757 tokens over 5,788 slots, every query sees all of them
        dict(name="frames", op="attend", seqs=1, new_lo=757, new_hi=757, ctx_lo=5031, ctx_hi=5031, q_heads=24,
             kv_heads=24, head_dim=128, page=64, axes=3, dtype="bf16", causal=False, window=0),
    ]


def _between(rng, lo, hi):
    """Spread over the logarithm of lo .. hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    head_dim = rng.choice((64, 128, 128))
    kv_heads = rng.choice((1, 2, 3, 4, 5, 8, 8, 12, 16))
    group = rng.choice((1, 1, 2, 3, 4, 4, 7, 8)) if kv_heads <= 8 else 1
    c = dict(op=rng.choice(("append", "append", "attend", "attend", "attend")), seqs=1, new_lo=1, new_hi=1, ctx_lo=0,
             ctx_hi=0, q_heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, page=rng.choice((16, 32, 64, 64, 128)),
             axes=rng.choice((1, 1, 3)), dtype=rng.choice(("bf16", "bf16", "f16")), causal=True, window=0)
    if c["op"] == "append":
        if rng.random() < 0.5:
            c["seqs"] = _between(rng, 1, 200)
            c["new_hi"] = rng.choice((1, 1, 3))
        else:
            c["seqs"] = _between(rng, 1, 12)
            c["new_hi"] = _between(rng, 5, 24000 // c["seqs"])
            c["new_lo"] = max(1, c["new_hi"] // rng.choice((1, 3, 20)))
        c["ctx_lo"], c["ctx_hi"] = rng.randrange(0, 100), _between(rng, 100, 3000)
    elif rng.random() < 0.5:                   # single tokens
        c["seqs"] = _between(rng, 1, 96)
        most = min(120000, 240000 // c["seqs"])
        c["ctx_hi"] = _between(rng, 50, most)
        c["ctx_lo"] = rng.randrange(0, c["ctx_hi"] + 1)
        c["window"] = rng.choice((0, 0, 0, 517))
    else:                                      # chunks and prompts
        c["seqs"] = _between(rng, 1, 6)
        c["new_hi"] = _between(rng, 5, 3000 // c["seqs"])
        c["new_lo"] = max(1, c["new_hi"] // rng.choice((1, 2, 9)))
        c["ctx_hi"] = _between(rng, 1, 12000 // c["seqs"])
        c["ctx_lo"] = rng.randrange(0, c["ctx_hi"] + 1)
        c["causal"] = rng.random() < 0.8
        c["window"] = rng.choice((0, 0, 300)) if c["causal"] else 0
    return c


def _ragged(case):
    """(new, ctx) per sequence: spread over the case's ranges, the same on every call."""
    n = case["seqs"]
    part = [((b + 1) * GOLDEN) % 1.0 if n > 1 else 1.0 for b in range(n)]
    other = [((b + 1) * GOLDEN * GOLDEN + 0.37) % 1.0 if n > 1 else 1.0 for b in range(n)]
    new = [case["new_lo"] + int(round(p * (case["new_hi"] - case["new_lo"]))) for p in part]
    ctx = [case["ctx_lo"] + int(round(p * (case["ctx_hi"] - case["ctx_lo"]))) for p in other]
    return new, ctx


def _axis_dims(case):
    d = case["head_dim"]
    return (d,) if case["axes"] == 1 else (d // 4, d * 3 // 8, d * 3 // 8)


def _pos_count(case):
    new, ctx = _ragged(case)
    most = max(a + b for a, b in zip(new, ctx)) + 1
    return (most,) if case["axes"] == 1 else (most // FRAME + 1, 8, 12)


def work(case):
    new, ctx = _ragged(case)
    h, q, d, p, w = case["kv_heads"], case["q_heads"], case["head_dim"], case["page"], case["window"]
    n = sum(new)
    if case["op"] == "append":
        # the tokens in 16 bits and their positions in, their codes and the touched pages' scales out
        pages = sum((c + a + p - 1) // p - c // p for a, c in zip(new, ctx))
        return {"bytes": n * h * d * 2 * 2 + n * 4 * case["axes"] + n * h * d * 2 + pages * h * 8, "flops": 3 * n * h * d}
    keys = pairs = 0
    for a, c in zip(new, ctx):
        if not case["causal"]:
            keys += a + c
            pairs += a * (a + c)
        elif not w:
            keys += a + c
            pairs += a * c + a * (a + 1) // 2
        else:
            first = max(0, c + 1 - w)
            keys += a + c - first
            pairs += sum(min(w, c + i + 1) for i in range(a))
    return {"bytes": keys * h * (2 * d + 8 / p) + n * q * d * 4 + n * 4 * case["axes"], "flops": 4 * d * q * pairs}


# ------------------------------------------------------------------ inputs
def _block_codes(x, page):
    """x [pages, H, P, D] float32 -> codes (uint8) and power-of-two scales [pages, H]: a filled cache."""
    a = x.abs().amax((2, 3))
    m, e = torch.frexp(a)
    s = torch.ldexp(torch.ones_like(a), e - torch.where(m <= 0.875, 9, 8))
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dev = torch.device("cuda")
    dt = torch.float16 if case["dtype"] == "f16" else torch.bfloat16
    h, d, p, b = case["kv_heads"], case["head_dim"], case["page"], case["seqs"]
    new, ctx = _ragged(case)
    n = sum(new)
    held = [(a + c + p - 1) // p for a, c in zip(new, ctx)]
    width, pages = max(held), sum(held) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    starts = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32)
    first = torch.tensor([0] + held, dtype=torch.int32).cumsum(0)
    slot = torch.arange(width)[None, :].expand(b, width)
    mine = slot < torch.tensor(held)[:, None]
    at = torch.where(mine, first[:b, None] + slot, 0).to(dev)
    # entries past a sequence's last page are never read
    table = torch.where(mine.to(dev), order[at], -1).to(torch.int32)
    length = torch.tensor([a + c for a, c in zip(new, ctx)], dtype=torch.int32, device=dev)
    index = torch.cat([torch.arange(c, c + a) for a, c in zip(new, ctx)])
    if case["axes"] == 1:
        pos = index[:, None]
    else:
        pos = torch.stack([index // FRAME, index // 12 % 8, index % 12], 1)
    s = dict(case=case, length=length, start=starts.to(dev), table=table, pos=pos.to(torch.int32).to(dev), n=n,
             max_new=max(new))
    # the cache: keys and values of unit variance, a few channels larger, head by head
    loud = 1.0 + 3.0 * (torch.rand((1, h, 1, d), generator=g, device=dev) < 0.02)
    k = torch.randn((pages, h, p, d), generator=g, device=dev) * loud
    s["k_codes"], s["k_scales"] = _block_codes(k, p)
    del k
    v = torch.randn((pages, h, p, d), generator=g, device=dev)
    s["v_codes"], s["v_scales"] = _block_codes(v, p)
    del v
    # q, k and v as a projection leaves them: one row per token, side by side
    qh = case["q_heads"]
    rows = torch.randn((n, qh + 2 * h, d), generator=g, device=dev)
    rows[:, qh:qh + h] *= loud[0].transpose(0, 1)
    s["qkv"] = rows.to(dt)
    s["q"], s["k"], s["v"] = s["qkv"][:, :qh], s["qkv"][:, qh:qh + h], s["qkv"][:, qh + h:]
    if own:
        from fp8_ring_kv_gb300.paged import PagedKV
        kv = PagedKV(h, qh, d, pages, p, _axis_dims(case), (0,) * case["axes"], _pos_count(case), ROPE_BASE, dtype=dt)
        for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
            getattr(kv, name)[0].copy_(s[name])
            s[name] = getattr(kv, name)[0]
        s["kv"] = kv
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    s, case = state, state["case"]
    if case["op"] == "append":
        if own:
            s["kv"].append(s["k"], s["v"], s["pos"], s["start"], s["length"], s["table"])
        else:
            _append(s, case)
        e4m3 = torch.float8_e4m3fn
        return dict(k_codes=s["k_codes"].view(e4m3), v_codes=s["v_codes"].view(e4m3), k_scales=s["k_scales"],
                    v_scales=s["v_scales"])
    if own:
        return s["kv"].attend(s["q"], s["pos"], s["start"], s["length"], s["table"], causal=case["causal"],
                              window=case["window"] or None, max_new=s["max_new"])
    return _attend(s, case)


def _rotate(x, pos, axis_dims):
    """RoPE of x [n, heads, D] in 32 bits; the angles in 64."""
    omega = [ROPE_BASE ** (-torch.arange(0, d, 2, dtype=torch.float64, device=x.device) / d) for d in axis_dims]
    angle = torch.cat([pos[:, a:a + 1].double() * w for a, w in enumerate(omega)], 1)
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x0, x1 = x.float().unflatten(2, (-1, 2)).unbind(3)
    return torch.stack((x0 * c - x1 * s, x0 * s + x1 * c), 3).flatten(2)


def _append(s, case):
    p = case["page"]
    row = torch.arange(s["n"], device=s["pos"].device)
    seq = torch.searchsorted(s["start"][1:].contiguous(), row, right=True)
    new = s["start"][1:] - s["start"][:-1]
    t = s["length"][seq] - new[seq] + row - s["start"][seq]
    page, off = s["table"][seq, t // p].long(), t % p
    # rows of the pages that were there before: below the first new row of the page
    before = torch.full((s["k_scales"].shape[0],), p, device=row.device).scatter_reduce(0, page, off, "amin")
    touched = torch.zeros_like(before, dtype=torch.bool).index_fill(0, page, True)
    for x, codes, scales in ((_rotate(s["k"], s["pos"], _axis_dims(case)), s["k_codes"], s["k_scales"]),
                             (s["v"].float(), s["v_codes"], s["v_scales"])):
        a = torch.zeros_like(scales).index_reduce(0, page, x.abs().amax(2), "amax")
        m, e = torch.frexp(a)
        need = torch.ldexp(torch.ones_like(a), e - torch.where(m <= 0.875, 9, 8)) * (a >= 2.0 ** -100)
        old = torch.where((before > 0)[:, None], scales, 0.0)
        s_new = torch.maximum(old, need)
        inv = torch.where(s_new > 0, 1.0 / s_new, 0.0)
        again = (codes.view(torch.float8_e4m3fn).float() * (old * inv)[:, :, None, None]).to(torch.float8_e4m3fn)
        keep = torch.arange(p, device=row.device) < torch.where(touched, before, 0)[:, None]
        grown = (s_new > old)[:, :, None] & keep[:, None]
        codes.copy_(torch.where(grown[..., None], again.view(torch.uint8), codes))
        iv = inv[page][:, :, None]
        q = torch.where(iv > 0, x * iv, 0.0).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[page, :, off] = q
        scales.copy_(torch.where(touched[:, None], s_new, scales))


def _attend(s, case):
    h, qh, d, p = case["kv_heads"], case["q_heads"], case["head_dim"], case["page"]
    b, nm, g = case["seqs"], s["max_new"], qh // h
    new = (s["start"][1:] - s["start"][:-1]).long()
    dev = new.device
    i = torch.arange(nm, device=dev)
    there = i < new[:, None]
    row = torch.where(there, s["start"][:-1, None] + i, 0)
    q = _rotate(s["q"], s["pos"], _axis_dims(case))[row] * d ** -0.5      # [b, nm, qh, d]
    q = q.unflatten(2, (h, g)).permute(0, 2, 1, 3, 4).reshape(b, h, nm * g, d)
    pages = s["table"].clamp_min(0).long()
    k, v = ((s[x + "_codes"][pages].view(torch.float8_e4m3fn).float() * s[x + "_scales"][pages][..., None, None])
            .transpose(1, 2).reshape(b, h, -1, d) for x in "kv")
    t = torch.arange(k.shape[2], device=dev)
    seen = t < s["length"][:, None, None]
    at = (s["length"] - new)[:, None] + i
    if case["causal"]:
        seen = seen & (t <= at[..., None])
    if case["window"]:
        seen = seen & (t > at[..., None] - case["window"])
    score = (q @ k.transpose(2, 3)).unflatten(2, (nm, g))
    score = torch.where(seen.expand(b, nm, -1)[:, None, :, None], score, -math.inf)
    m = score.amax(-1, keepdim=True).clamp_min(-1e30)
    e = torch.exp(score - m)
    o = e.flatten(2, 3) @ v / e.sum(-1).flatten(2, 3).clamp_min(1e-30)[..., None]
    o = o.unflatten(2, (nm, g)).permute(0, 2, 1, 3, 4).reshape(b, nm, qh, d)
    return o[there].to(s["q"].dtype)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    start, length = s["start"].tolist(), s["length"].tolist()
    table, p, d = s["table"].tolist(), case["page"], case["head_dim"]
    turn = []
    for a, width in enumerate(_axis_dims(case)):
        for j in range(width // 2):
            turn.append(s["pos"][:, a].double() * math.exp(-2.0 * j / width * math.log(ROPE_BASE)))
    turn = torch.polar(torch.ones_like(turn[0])[:, None].expand(-1, d // 2).contiguous(), torch.stack(turn, 1))[:, None]

    def rotated(x):
        z = torch.view_as_complex(x.double().reshape(x.shape[0], x.shape[1], d // 2, 2)) * turn
        return torch.view_as_real(z).reshape(x.shape)

    def value(codes):
        c = codes.long()
        e, m = c >> 3 & 15, (c & 7).double()
        return torch.where(c > 127, -1.0, 1.0) * torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7).double(), m * 2.0 ** -9)

    if case["op"] == "append":
        out = {}
        for name, x in (("k", rotated(s["k"])), ("v", s["v"].double())):
            vals, scales = value(s[name + "_codes"]), s[name + "_scales"].double()
            for b in range(case["seqs"]):
                t, r = length[b] - (start[b + 1] - start[b]), start[b]
                while r < start[b + 1]:
                    pg, off = table[b][t // p], t % p
                    n = min(p - off, start[b + 1] - r)
                    new = x[r:r + n].transpose(0, 1)                       # [H, n, D]
                    need = new.abs().amax((1, 2))
                    k = torch.ceil(torch.log2(need / 448))
                    k = torch.where(448 * 2.0 ** (k - 1) >= need, k - 1, k)
                    need = torch.where(need < 2.0 ** -100, 0.0, 2.0 ** k)
                    was = scales[pg] * (off > 0)
                    now = torch.maximum(was, need)
                    full = torch.where(now > 0, now, 1.0)[:, None, None]
                    page = torch.cat([vals[pg, :, :off] * was[:, None, None], new * (now > 0)[:, None, None]], 1) / full
                    step = 2.0 ** (torch.frexp(page)[1].clamp_min(-5) - 4).double()
                    vals[pg, :, :off + n] = torch.round(page / step) * step
                    scales[pg] = now
                    t, r = t + n, r + n
            out[name + "_codes"], out[name + "_scales"] = vals, scales
        return dict(k_codes=out["k_codes"], v_codes=out["v_codes"], k_scales=out["k_scales"], v_scales=out["v_scales"])

    h, g = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    q, out = rotated(s["q"]), torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["seqs"]):
        n, ln = start[b + 1] - start[b], length[b]
        if n == 0 or ln == 0:
            continue
        own_index = torch.arange(ln - n, ln, device="cuda")
        pages = s["table"][b, :(ln + p - 1) // p].long()
        for j in range(h):
            k = (value(s["k_codes"][pages, j]) * s["k_scales"][pages, j].double()[:, None, None]).reshape(-1, d)[:ln]
            v = (value(s["v_codes"][pages, j]) * s["v_scales"][pages, j].double()[:, None, None]).reshape(-1, d)[:ln]
            at = torch.arange(ln, device="cuda")
            hide = torch.zeros((n, ln), dtype=torch.bool, device="cuda")
            if case["causal"]:
                hide |= at > own_index[:, None]
            if case["window"]:
                hide |= own_index[:, None] - at >= case["window"]
            for i in range(j * g, (j + 1) * g):
                z = q[start[b]:start[b + 1], i] @ k.T / math.sqrt(d)
                w = torch.softmax(z.masked_fill_(hide, -math.inf), 1)
                out[start[b]:start[b + 1], i] = w @ v
    return out
