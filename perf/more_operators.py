"""The paged latent cache's operators as a set of measured cases.

Latent attention keeps one row per token: a latent vector of C numbers that is
key and value of every head at once, and a rotated key part of R = 64 numbers
that all heads share.  Four operators work on it: appending rows to a paged
e4m3 cache (rotation on the way, one power-of-two scale per token), reading
rows back, attention over the cache in the absorbed form (queries already in
the latent space), and attention in the expanded form (keys and values of every
head made from the latents by the caller).  ``listed()`` names the cases,
``draw()`` makes more of the same ranges, ``prepare()`` builds the inputs of
one, ``run()`` makes one pass: the plain form in elementary torch operations,
or, with ``own`` true, the calls of ``fp8_ring_kv_gb300.latent``.  ``exact()``
is the definition in 64 bits.

Definitions.  Sequence b has ``new[b]`` new tokens (rows start[b] ..
start[b+1]-1 of the packed inputs) and ``length[b]`` tokens in the cache; row i
of it has cache index t = length[b] - new[b] + i, in page table[b, t // P] at
row t % P.

append: x = [latent, RoPE(k_rope)] (interleaved pairs, fp32); s is the smallest
power of two with max |x| <= 448 s, at least 2^-40; codes e4m3(x / s), round to
nearest even.

read: row i of sequence b is code * s of its cache index, in the cache's type.

attend: query row i of head h attends over t < length[b] (causal: t <= its own
index; window w: the last w of those):
out = sum_t softmax_t(scale (q_latent . c_t + RoPE(q_rope) . r_t)) c_t with
(c_t, r_t) the cached row's value; a row that sees nothing gives zeros.

expanded: the same with k_t = [k[t, h], k_rope[t]] (k_rope rotated already), v_t
= v[t, h], q = [128 numbers, RoPE(64 numbers)], scale = 1 / sqrt(192).
"""
import math

import torch

own = False

ROPE_BASE = 10000.0
ROPE = 64
HEAD = 128          # a head's own key and value numbers in the expanded form
SCALE = (HEAD + ROPE) ** -0.5
FRAME = 96          # three-axis positions: frames of 8 x 12 tokens
GOLDEN = 0.6180339887498949


# ------------------------------------------------------------------ cases
def _case(name, op, seqs, new, ctx, heads, latent=512, page=64, axes=1, dtype="bf16", causal=True, window=0):
    return dict(name=name, op=op, seqs=seqs, new_lo=new[0], new_hi=new[1], ctx_lo=ctx[0], ctx_hi=ctx[1], heads=heads,
                latent=latent, page=page, axes=axes, dtype=dtype, causal=causal, window=window)


def listed():
    return [
        # a decoding batch writes one token per sequence
        _case("append_batch", "append", 128, (1, 1), (100, 2000), 32),
        # prompts of several users, ragged, each continuing inside a page
        _case("append_prompts", "append", 7, (37, 5000), (1, 300), 32),
        # one short prompt's rows, for the keys and values of the expanded form
        _case("read_short", "read", 1, (777, 777), (0, 0), 32, page=16, latent=256, dtype="f16"),
        # long cached prefixes, read back before a chunk of new tokens is computed in the expanded form
        _case("read_prefixes", "read", 6, (1000, 30000), (0, 0), 32),
        # one conversation decodes one token: the latency of the smallest call
        _case("decode_one", "attend", 1, (1, 1), (900, 900), 32),
        # a decoding batch of ragged contexts, 64 heads
        _case("decode_batch", "attend", 64, (1, 1), (200, 8000), 64),
        # two very long contexts, 128 heads: few rows, the cache split along its length
        _case("decode_long", "attend", 2, (1, 1), (100001, 131000), 128, page=128),
        # a smaller latent in fp16, few heads, small pages, three position axes
        _case("decode_small", "attend", 24, (1, 1), (300, 5000), 20, latent=256, page=16, axes=3, dtype="f16"),
        # a scheduler's step: a chunk and a few drafted tokens together, a sliding window
        _case("mixed_window", "attend", 9, (2, 131), (0, 6000), 32, page=32, window=1024),
        # a short prompt in the expanded form
        _case("prompt_short", "expanded", 1, (90, 90), (0, 0), 20, dtype="f16"),
        # whole prompts, causal, in the expanded form
        _case("prompts", "expanded", 3, (1000, 4096), (0, 0), 32),
        # a chunk of a long prompt over what was read back from the cache
        _case("chunk_long", "expanded", 1, (512, 512), (16001, 16001), 20),
    ]


def _between(rng, lo, hi):
    """Spread over the logarithm of lo .. hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        if w["flops"] <= 8e10 and w["bytes"] <= 2e8:
            return c


def _draw(rng):
    op = rng.choice(("append", "read", "attend", "attend", "attend", "expanded", "expanded"))
    heads = rng.choice((1, 2, 5, 8, 12, 16, 20, 32, 40, 64, 96, 128)) if op != "expanded" else rng.choice((1, 2, 5, 8, 10, 20, 32))
    c = _case(None, op, 1, (1, 1), (0, 0), heads, rng.choice((512, 512, 512, 384, 256, 128)), rng.choice((16, 32, 64, 64, 128)),
              rng.choice((1, 1, 3)), rng.choice(("bf16", "bf16", "f16")))
    del c["name"]
    if op in ("append", "read"):
        if rng.random() < 0.4:
            c["seqs"] = _between(rng, 1, 200)
            c["new_hi"] = rng.choice((1, 1, 3))
        else:
            c["seqs"] = _between(rng, 1, 12)
            c["new_hi"] = _between(rng, 5, 60000 // c["seqs"])
            c["new_lo"] = max(1, c["new_hi"] // rng.choice((1, 3, 20)))
        c["ctx_lo"], c["ctx_hi"] = rng.randrange(0, 100), _between(rng, 100, 3000)
    elif op == "attend" and rng.random() < 0.6:      # single tokens
        c["seqs"] = _between(rng, 1, 96)
        c["ctx_hi"] = _between(rng, 50, min(120000, 240000 // c["seqs"]))
        c["ctx_lo"] = rng.randrange(0, c["ctx_hi"] + 1)
        c["window"] = rng.choice((0, 0, 0, 517))
    else:                                            # chunks and prompts
        c["seqs"] = _between(rng, 1, 6)
        c["new_hi"] = _between(rng, 2 if op == "attend" else 5, (400 if op == "attend" else 5000) // c["seqs"])
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
    return (ROPE,) if case["axes"] == 1 else (ROPE // 4, ROPE * 3 // 8, ROPE * 3 // 8)


def _pos_count(case):
    new, ctx = _ragged(case)
    most = max(a + b for a, b in zip(new, ctx)) + 1
    return (most,) if case["axes"] == 1 else (most // FRAME + 1, 8, 12)


def work(case):
    new, ctx = _ragged(case)
    h, c, w, n = case["heads"], case["latent"], case["window"], sum(new)
    row = c + ROPE
    if case["op"] == "append":
        return {"bytes": n * row * 2 + n * 4 * case["axes"] + n * (row + 4), "flops": 3 * n * row}
    if case["op"] == "read":
        return {"bytes": n * (row + 4) + n * row * 2, "flops": n * row}
    keys = pairs = 0
    for a, b in zip(new, ctx):
        if not case["causal"]:
            keys += a + b
            pairs += a * (a + b)
        elif not w:
            keys += a + b
            pairs += a * b + a * (a + 1) // 2
        else:
            first = max(0, b + 1 - w)
            keys += a + b - first
            pairs += sum(min(w, b + i + 1) for i in range(a))
    if case["op"] == "attend":
        return {"bytes": keys * (row + 4) + n * h * (row + c) * 2 + n * 4 * case["axes"], "flops": 2 * h * (row + c) * pairs}
    return {"bytes": keys * (2 * HEAD * h + ROPE) * 2 + n * h * (2 * HEAD + ROPE) * 2 + n * 4 * case["axes"],
            "flops": 2 * h * (2 * HEAD + ROPE) * pairs}


# ------------------------------------------------------------------ inputs
def _rows(n, c, g, dev):
    """Latents as a normalisation leaves them (unit mean square, a weight per channel), and key parts."""
    x = torch.randn((n, c), generator=g, device=dev)
    x *= torch.rsqrt(x.square().mean(1, keepdim=True))
    x *= 0.5 + torch.rand((1, c), generator=g, device=dev) + 3.0 * (torch.rand((1, c), generator=g, device=dev) < 0.01)
    return x, 1.5 * torch.randn((n, ROPE), generator=g, device=dev)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dev = torch.device("cuda")
    dt = torch.float16 if case["dtype"] == "f16" else torch.bfloat16
    h, c, p, b = case["heads"], case["latent"], case["page"], case["seqs"]
    new, ctx = _ragged(case)
    n = sum(new)
    lens = [a + e for a, e in zip(new, ctx)]
    starts = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32)
    index = torch.cat([torch.arange(e, e + a) for a, e in zip(new, ctx)])
    if case["axes"] == 1:
        pos = index[:, None]
    else:
        pos = torch.stack([index // FRAME, index // 12 % 8, index % 12], 1)
    s = dict(case=case, length=torch.tensor(lens, dtype=torch.int32, device=dev), start=starts.to(dev),
             pos=pos.to(torch.int32).to(dev), n=n, max_new=max(new), dtype=dt, pages=1)
    if case["op"] == "expanded":
        t = sum(lens)
        s["kv_start"] = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32)[:b].to(dev)
        # q as a projection leaves it, k and v side by side as the expansion does, the shared part beside the latents
        s["q"] = torch.randn((n, h, HEAD + ROPE), generator=g, device=dev).to(dt)
        kv = torch.randn((t, h, 2 * HEAD), generator=g, device=dev).to(dt)
        s["k"], s["v"] = kv[..., :HEAD], kv[..., HEAD:]
        rows = torch.cat(_rows(t, c, g, dev), 1).to(dt)
        s["k_rope"] = rows[:, c:]
    else:
        held = [(a + p - 1) // p for a in lens]
        width, pages = max(held), sum(held) + 3
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        first = torch.tensor([0] + held, dtype=torch.int32).cumsum(0)
        slot = torch.arange(width)[None, :].expand(b, width)
        mine = slot < torch.tensor(held)[:, None]
        at = torch.where(mine, first[:b, None] + slot, 0).to(dev)
        # entries past a sequence's last page are never read
        s["table"] = torch.where(mine.to(dev), order[at], -1).to(torch.int32)
        s["pages"] = pages
        # the cache, filled
        x = torch.cat(_rows(pages * p, c, g, dev), 1)
        m, e = torch.frexp(x.abs().amax(1))
        scale = torch.ldexp(torch.ones_like(m), e - torch.where(m <= 0.875, 9, 8))
        s["codes"] = (x / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(pages, p, c + ROPE)
        s["scales"] = scale.view(pages, p)
        del x
        if case["op"] == "append":
            s["latent"], k_rope = (y.to(dt) for y in _rows(n, c, g, dev))
            # the key part as a slice of its projection's rows
            s["k_rope"] = torch.cat([s["latent"], k_rope], 1)[:, c:]
        elif case["op"] == "attend":
            # latent queries as a batched product over heads leaves them, the rotated part a slice of its heads
            s["q_latent"] = (0.7 * torch.randn((h, n, c), generator=g, device=dev)).to(dt).transpose(0, 1)
            s["q_rope"] = torch.randn((n, h, HEAD + ROPE), generator=g, device=dev).to(dt)[..., HEAD:]
    if own:
        from fp8_ring_kv_gb300.latent import LatentKV
        kv = LatentKV(h, c, s["pages"], p, _axis_dims(case), (0,) * case["axes"], _pos_count(case), ROPE_BASE, dtype=dt)
        if case["op"] != "expanded":
            for name in ("codes", "scales"):
                getattr(kv, name)[0].copy_(s[name])
                s[name] = getattr(kv, name)[0]
        s["kv"] = kv
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    s, case = state, state["case"]
    kv = s.get("kv")
    if case["op"] == "append":
        if own:
            kv.append(s["latent"], s["k_rope"], s["pos"], s["start"], s["length"], s["table"])
        else:
            _append(s, case)
        return dict(codes=s["codes"].view(torch.float8_e4m3fn), scales=s["scales"])
    if case["op"] == "read":
        return kv.read(s["start"], s["length"], s["table"], s["n"]) if own else _read(s, case)
    if case["op"] == "attend":
        if own:
            return kv.attend(s["q_latent"], s["q_rope"], s["pos"], s["start"], s["length"], s["table"], SCALE,
                             causal=case["causal"], window=case["window"] or None, max_new=s["max_new"])
        return _attend(s, case)
    if own:
        return kv.attend_expanded(s["q"], s["k"], s["k_rope"], s["v"], s["pos"], s["start"], s["kv_start"], s["length"],
                                  causal=case["causal"], window=case["window"] or None, max_new=s["max_new"])
    return _expanded(s, case)


def _rotate(x, pos, axis_dims):
    """RoPE of x [n, heads, ROPE] in 32 bits; the angles in 64."""
    omega = [ROPE_BASE ** (-torch.arange(0, d, 2, dtype=torch.float64, device=x.device) / d) for d in axis_dims]
    angle = torch.cat([pos[:, a:a + 1].double() * w for a, w in enumerate(omega)], 1)
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x0, x1 = x.float().unflatten(2, (-1, 2)).unbind(3)
    return torch.stack((x0 * c - x1 * s, x0 * s + x1 * c), 3).flatten(2)


def _places(s, case):
    """Page and row of every new token."""
    row = torch.arange(s["n"], device=s["pos"].device)
    seq = torch.searchsorted(s["start"][1:].contiguous(), row, right=True)
    t = s["length"][seq] - s["start"][seq + 1] + row
    return s["table"][seq, t // case["page"]].long(), t % case["page"]


def _append(s, case):
    page, off = _places(s, case)
    x = torch.cat([s["latent"].float(), _rotate(s["k_rope"][:, None], s["pos"], _axis_dims(case))[:, 0]], 1)
    m, e = torch.frexp(x.abs().amax(1))
    scale = torch.ldexp(torch.ones_like(m), e - torch.where(m <= 0.875, 9, 8)).clamp_min(2.0 ** -40)
    s["codes"][page, off] = (x / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    s["scales"][page, off] = scale


def _read(s, case):
    page, off = _places(s, case)
    x = s["codes"][page, off].view(torch.float8_e4m3fn).float() * s["scales"][page, off][:, None]
    return x.to(s["dtype"])


def _seen(s, case, keys):
    """[b, max_new, keys]: what each query sees; and where a query is one."""
    new = (s["start"][1:] - s["start"][:-1]).long()
    i = torch.arange(s["max_new"], device=new.device)
    t = torch.arange(keys, device=new.device)
    seen = t < s["length"][:, None, None]
    at = (s["length"] - new)[:, None] + i
    if case["causal"]:
        seen = seen & (t <= at[..., None])
    if case["window"]:
        seen = seen & (t > at[..., None] - case["window"])
    there = i < new[:, None]
    return seen.expand(len(new), len(i), keys), there, torch.where(there, s["start"][:-1, None] + i, 0)


def _softmax(score, seen):
    score = torch.where(seen, score, -math.inf)
    e = torch.exp(score - score.amax(-1, keepdim=True).clamp_min(-1e30))
    return e, e.sum(-1, keepdim=True).clamp_min(1e-30)


def _attend(s, case):
    c, h = case["latent"], case["heads"]
    pages = s["table"].clamp_min(0).long()
    k = (s["codes"][pages].view(torch.float8_e4m3fn).float() * s["scales"][pages][..., None]).flatten(1, 2)   # [b, t, c + ROPE]
    seen, there, row = _seen(s, case, k.shape[1])
    q = torch.cat([s["q_latent"].float(), _rotate(s["q_rope"], s["pos"], _axis_dims(case))], 2) * SCALE
    score = q[row].flatten(1, 2) @ k.transpose(1, 2)                              # [b, max_new * h, t]
    e, total = _softmax(score, seen.repeat_interleave(h, 1))
    o = e @ k[..., :c] / total
    return o.unflatten(1, (-1, h))[there].to(s["dtype"])


def _expanded(s, case):
    h, b = case["heads"], case["seqs"]
    longest = max(a + e for a, e in zip(*_ragged(case)))
    t = torch.arange(longest, device=s["kv_start"].device)
    at = s["kv_start"][:, None] + torch.where(t < s["length"][:, None], t, 0)     # [b, t]
    seen, there, row = _seen(s, case, longest)
    q = torch.cat([s["q"][..., :HEAD].float(), _rotate(s["q"][..., HEAD:], s["pos"], _axis_dims(case))], 2) * SCALE
    q = q[row].transpose(1, 2)                                                    # [b, h, max_new, 192]
    k = torch.cat([s["k"].float(), s["k_rope"].float()[:, None].expand(-1, h, -1)], 2)[at].transpose(1, 2)
    e, total = _softmax(q @ k.transpose(2, 3), seen[:, None])
    o = e @ s["v"].float()[at].transpose(1, 2) / total                            # [b, h, max_new, 128]
    return o.transpose(1, 2)[there].to(s["dtype"])


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    start, length = s["start"].tolist(), s["length"].tolist()
    c, h, p = case["latent"], case["heads"], case["page"]
    turn = []
    for a, width in enumerate(_axis_dims(case)):
        for j in range(width // 2):
            turn.append(s["pos"][:, a].double() * math.exp(-2.0 * j / width * math.log(ROPE_BASE)))
    turn = torch.polar(torch.ones_like(turn[0])[:, None].expand(-1, ROPE // 2).contiguous(), torch.stack(turn, 1))

    def rotated(x):
        z = torch.view_as_complex(x.double().reshape(*x.shape[:-1], ROPE // 2, 2))
        return torch.view_as_real(z * (turn if x.dim() == 2 else turn[:, None])).reshape(x.shape)

    def value(codes):
        u = codes.long()
        e, m = u >> 3 & 15, (u & 7).double()
        return torch.where(u > 127, -1.0, 1.0) * torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7).double(), m * 2.0 ** -9)

    if case["op"] in ("append", "read"):
        pages, offs = [], []
        table = s["table"].cpu()
        for b in range(case["seqs"]):
            t = torch.arange(length[b] - (start[b + 1] - start[b]), length[b])
            pages.append(table[b][t // p].long())
            offs.append(t % p)
        at = (torch.cat(pages).cuda(), torch.cat(offs).cuda())
        vals, scales = value(s["codes"]), s["scales"].double()
        if case["op"] == "read":
            return vals[at] * scales[at][:, None]
        x = torch.cat([s["latent"].double(), rotated(s["k_rope"])], 1)
        most = x.abs().amax(1)
        k = torch.ceil(torch.log2(most / 448))
        k = torch.where(448 * 2.0 ** (k - 1) >= most, k - 1, k).clamp_min(-40.0)
        x = x / (2.0 ** k)[:, None]
        step = 2.0 ** (torch.frexp(x)[1].clamp_min(-5) - 4).double()
        vals[at] = torch.round(x / step) * step
        scales[at] = 2.0 ** k
        return dict(codes=vals, scales=scales)

    def weights(z, b):
        own_index = torch.arange(length[b] - z.shape[0], length[b], device="cuda")
        at = torch.arange(length[b], device="cuda")
        hide = torch.zeros(z.shape, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hide |= at > own_index[:, None]
        if case["window"]:
            hide |= own_index[:, None] - at >= case["window"]
        return torch.softmax(z.masked_fill_(hide, -math.inf), 1)

    expanded = case["op"] == "expanded"
    if expanded:
        q_own, q_turned = s["q"][..., :HEAD], rotated(s["q"][..., HEAD:])
    else:
        q_own, q_turned = s["q_latent"], rotated(s["q_rope"])
    out = torch.zeros((s["n"], h, HEAD if expanded else c), dtype=torch.float64, device="cuda")
    for b in range(case["seqs"]):
        rows, ln = slice(start[b], start[b + 1]), length[b]
        if expanded:
            first = int(s["kv_start"][b])
            shared = s["k_rope"][first:first + ln].double()
        else:
            pages = s["table"][b, :(ln + p - 1) // p].long()
            cached = (value(s["codes"][pages]) * s["scales"][pages].double()[..., None]).reshape(-1, c + ROPE)[:ln]
            keys = values = cached[:, :c]
            shared = cached[:, c:]
        for i in range(h):
            if expanded:
                keys, values = s["k"][first:first + ln, i].double(), s["v"][first:first + ln, i].double()
            z = (q_own[rows, i].double() @ keys.T + q_turned[rows, i] @ shared.T) * SCALE
            out[rows, i] = weights(z, b) @ values
    return out
