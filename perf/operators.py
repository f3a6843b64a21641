"""Measured cases of the 4-bit KV cache operators: writing a cache, reading it back and
decoding against it.

The cache is one uint8 tensor [2, num_pages, G, page_size / 16, 10 d]: plane 0 holds K
(normed and rotated), plane 1 raw V, and every 16 tokens of one KV head are one block
of 10 d bytes,
  codes   [d / 64][16 tokens][32 bytes]  the 64 features of a slab as eight 32-bit words;
          word w holds features 4w .. 4w+3 in its low half and 32+4w .. 32+4w+3 in its
          high half, lowest feature in the lowest four bits,
  scales  [d / 32][16 tokens] bf16,
  centres [d / 32][16 tokens] bf16,
and a feature stands for centre + scale * (code - 8).  A group of 32 features with the
extremes lo and hi is written as
  scale = bf16((hi - lo) / 15),  centre = bf16(lo + 8 (hi - lo) / 15),
  code - 8 = round_half_even((x - centre) * fp32(1 / scale)) within [-8, 7].
"""
import math
import random

import torch

own = False
DEV = "cuda"
GROUP, BLOCK, SLAB = 32, 16, 64


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one user's first tokens: a short sequence, where latency is everything
        dict(name="decode_one_short", op="decode", B=1, H=8, G=2, d=256, rd=64, base=1e7, page=64, lo=500, hi=517,
             gate="elementwise", append=False, mix=1),
        # the framework's decode benchmark shape: 64 sequences of 16k to 32k cached tokens
        dict(name="decode_64_long", op="decode", B=64, H=8, G=2, d=256, rd=64, base=1e7, page=64, lo=16384, hi=32768,
             gate="elementwise", append=False, mix=2),
        # a serving batch of mixed lengths over small pages, the new token written in the same step
        dict(name="decode_append_ragged", op="decode", B=48, H=16, G=8, d=128, rd=128, base=1e6, page=16, lo=1,
             hi=4096, gate="headwise", append=True, mix=3),
        # a few very long contexts, the work split along them
        dict(name="decode_4_very_long", op="decode", B=4, H=32, G=4, d=128, rd=64, base=1e6, page=256, lo=60001,
             hi=131072, gate="head_shared", append=False, mix=4),
        # many short sequences, unused rows among them, no gate
        dict(name="decode_200_tiny", op="decode", B=200, H=12, G=4, d=64, rd=32, base=1e4, page=32, lo=0, hi=301,
             gate="none", append=False, mix=5),
        # one new token for each of 64 sequences
        dict(name="write_64_tokens", op="write", B=64, G=2, d=256, rd=64, base=1e7, page=64, lo=1, hi=1, before=8000,
             dtype="bf16", packed=False, mix=6),
        # a chunk of prompts of odd lengths, all features rotated
        dict(name="write_ragged_chunk", op="write", B=11, G=8, d=128, rd=128, base=1e6, page=128, lo=1, hi=1500,
             before=3001, dtype="bf16", packed=True, mix=7),
        # a long prefill
        dict(name="write_long_prefill", op="write", B=8, G=2, d=256, rd=64, base=1e7, page=64, lo=16384, hi=16384,
             before=0, dtype="bf16", packed=False, mix=8),
        # fp32 projections, an odd number of heads
        dict(name="write_fp32", op="write", B=5, G=3, d=64, rd=32, base=1e4, page=16, lo=100, hi=2001, before=77,
             dtype="fp32", packed=True, mix=9),
        # one short prefix read back
        dict(name="read_short", op="read", B=1, G=2, d=256, page=64, lo=333, hi=333, before=100, dtype="bf16", mix=10),
        # prefixes of a whole batch read back, starting inside pages
        dict(name="read_long_ragged", op="read", B=24, G=4, d=128, page=64, lo=1001, hi=16384, before=2001,
             dtype="bf16", mix=11),
        # a prefix read back in fp32
        dict(name="read_fp32", op="read", B=6, G=8, d=64, page=32, lo=0, hi=4099, before=500, dtype="fp32", mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """The ranges: head_dim 64 to 256, any rotary share of it, 1 to 8 KV heads with 1 to 8
    query heads each, pages of 16 to 256 tokens, 1 to 256 sequences of 0 to 131072 tokens."""
    op = rng.choice(("decode", "write", "read"))
    d = rng.choice((64, 128, 256))
    c = dict(op=op, B=_log(rng, 1, 256), G=rng.randint(1, 8), d=d, page=rng.choice((16, 32, 64, 128, 256)),
             mix=rng.randrange(1 << 20))
    if op == "decode":
        c.update(H=c["G"] * rng.randint(1, 8), gate=rng.choice(("elementwise", "headwise", "head_shared", "none")),
                 append=rng.random() < 0.4)
        total = _log(rng, 1 << 9, 1 << 28) / (c["G"] * d)  # cached tokens of the batch
        c["hi"] = max(2, min(131072, int(2 * total / c["B"])))
        c["lo"] = rng.choice((int(c["append"]), 1, c["hi"] // 2, c["hi"] - 1))
    else:
        total = _log(rng, 1 << 9, 1 << 26) / (c["G"] * d)
        c["hi"] = 1 if rng.random() < 0.2 else max(1, min(32768, int(2 * total / c["B"])))
        c["lo"] = rng.choice((0, 1, (c["hi"] + 1) // 2)) if c["B"] > 1 and c["hi"] > 1 else c["hi"]
        c.update(before=rng.choice((0, 1, 999, 8000)), dtype="fp32" if rng.random() < 0.25 else "bf16")
        if op == "write":
            c["packed"] = rng.random() < 0.5
    if op != "read":
        c.update(rd=16 * rng.randint(0, d // 16), base=rng.choice((1e4, 1e6, 1e7)))
    return c


def _lengths(case):
    """The batch's lengths, from the case alone: uniform over [lo, hi], at least one token in all."""
    r = random.Random(case["mix"])
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    n[r.randrange(len(n))] = max(1, case["hi"])
    return n


def _before(case):
    """Tokens cached ahead of the ones a write or read deals with."""
    r = random.Random(case["mix"] + 1)
    return [r.randint(0, case["before"]) for _ in range(case["B"])]


def work(case):
    G, d = case["G"], case["d"]
    n = sum(_lengths(case))
    row = 2 * G * d  # numbers of K and V a token has
    if case["op"] == "decode":
        H, B = case["H"], case["B"]
        gates = {"elementwise": H * d, "headwise": H, "head_shared": d, "none": 0}[case["gate"]]
        new = 2 * B * row * (2 + 0.625) if case["append"] else 0  # projections in, rows written and returned
        return {"bytes": n * row * 0.625 + 2 * B * (2 * H * d + gates) + new, "flops": 4 * H * d * n}
    elt = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "write":  # projections read, cache rows written, the values they stand for returned
        return {"bytes": n * row * (elt + 0.625 + 2), "flops": 12 * n * row}
    return {"bytes": n * row * (0.625 + elt), "flops": 2 * n * row}


# ------------------------------------------------------------------ the format, plainly

def _code_bytes(n):
    """Codes 0..15 [..., d] as the format's bytes [..., d/64, 32]."""
    x = n.to(torch.uint8).unflatten(-1, (-1, 2, 8, 2, 2))  # slab, half, word, byte of the half, nibble
    x = x[..., 0] | (x[..., 1] << 4)
    return x.transpose(-3, -2).flatten(-3)  # slab, (word, half, byte)


def _codes(b):
    """The inverse: bytes [..., d/64, 32] to codes [..., d] as int16."""
    x = b.unflatten(-1, (8, 2, 2)).transpose(-3, -2)  # slab, half, word, byte
    return torch.stack((x & 15, x >> 4), -1).flatten(-5).to(torch.int16)


def _encode(x):
    """Codes, scales and centres of fp32 x [..., d]."""
    g = x.unflatten(-1, (-1, GROUP))
    hi, lo = g.amax(-1), g.amin(-1)
    step = (0.5 * hi - 0.5 * lo) * torch.tensor(2 / 15, dtype=torch.float32, device=x.device)
    scale, centre = step.bfloat16(), (lo + 8 * step).bfloat16()
    s, c = scale.float()[..., None], centre.float()[..., None]
    inv = torch.where(s > 0, 1 / s, torch.zeros_like(s))
    n = torch.round((g - c).double() * inv.double()).clamp(-8, 7) + 8  # 64 bits: values next to a border
    return n.flatten(-2), scale, centre


def _parts(cache):
    """Views of a cache: codes [2,pages,G,blocks,slabs,16,32], scales and centres
    [2,pages,G,blocks,groups,16]."""
    d = cache.shape[-1] // 10
    codes = cache[..., :8 * d].unflatten(-1, (d // SLAB, BLOCK, 32))
    sc = cache[..., 8 * d:9 * d].view(torch.bfloat16).unflatten(-1, (d // GROUP, BLOCK))
    ce = cache[..., 9 * d:].view(torch.bfloat16).unflatten(-1, (d // GROUP, BLOCK))
    return codes, sc, ce


def _put(cache, plane, page, slot, x):
    """Writes fp32 rows x [T,G,d] to slot `slot` of page `page` (both [T])."""
    n, s, c = _encode(x)
    codes, sc, ce = _parts(cache)
    blk, row = slot // BLOCK, slot % BLOCK
    codes[plane][page, :, blk, :, row] = _code_bytes(n)
    sc[plane][page, :, blk, :, row] = s
    ce[plane][page, :, blk, :, row] = c


def _get(cache, plane, page, slot):
    """The fp32 values of those rows, [T,G,d]."""
    codes, sc, ce = _parts(cache)
    blk, row = slot // BLOCK, slot % BLOCK
    n = _codes(codes[plane][page, :, blk, :, row]).float().unflatten(-1, (-1, GROUP))
    s = sc[plane][page, :, blk, :, row].float()[..., None]
    c = ce[plane][page, :, blk, :, row].float()[..., None]
    return (c + s * (n - 8)).flatten(-2)


def _whole(cache, plane, table):
    """The fp32 values of whole pages, [B, G, max_pages * page_size, d]."""
    codes, sc, ce = (t[plane][table.long()] for t in _parts(cache))  # [B, pages, G, blocks, ...]
    n = _codes(codes.transpose(-3, -2)).float().unflatten(-1, (-1, GROUP))  # [..., 16, groups, 32]
    x = (ce.transpose(-1, -2).float()[..., None] + sc.transpose(-1, -2).float()[..., None] * (n - 8)).flatten(-2)
    return x.transpose(1, 2).flatten(2, 4)


def _norm_rope(x, w, pos, rd, base, eps=1e-6, dtype=torch.float32):
    """QK-RMSNorm of x [T,heads,d], then rotate-half RoPE over the first rd features; angles in 64 bits."""
    x = x.to(dtype)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.to(dtype)
    if rd == 0:
        return x
    f = base ** (-2.0 * torch.arange(rd // 2, device=x.device, dtype=torch.float64) / rd)
    a = (pos.double()[:, None] * f)[:, None]
    cos, sin = a.cos().to(dtype), a.sin().to(dtype)
    x1, x2 = x[..., :rd // 2], x[..., rd // 2:rd]
    return torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin, x[..., rd:]), -1)


# ------------------------------------------------------------------ what a program has in hand

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _pages(case, reach, g):
    """An empty cache for sequences of the lengths `reach`, and its table over shuffled pages."""
    page = case["page"]
    per = max(1, -(-max(reach) // page))
    num = sum(-(-n // page) for n in reach) + 3
    perm = torch.randperm(num, generator=g, device=DEV).int()
    table = torch.full((case["B"], per), -1, dtype=torch.int32, device=DEV)  # unused entries name no page
    at = 0
    for b, n in enumerate(reach):
        k = -(-n // page)
        table[b, :k] = perm[at:at + k]
        at += k
    cache = torch.full((2, num, case["G"], page // BLOCK, 10 * case["d"]), 255, dtype=torch.uint8, device=DEV)
    return cache, table


def _fill(cache, g, spare=0):
    """Every page holds tokens: keys of unit norm per feature, values with their own spread."""
    _, num, G, blocks, row = cache.shape
    d = row // 10
    step = max(1, (1 << 26) // (G * blocks * BLOCK * d))
    slot = torch.arange(blocks * BLOCK, device=DEV)
    for p in range(0, num, step):
        page = torch.arange(p, min(num, p + step), device=DEV).repeat_interleave(len(slot))
        at = slot.repeat(len(page) // len(slot))
        _put(cache, 0, page, at, _randn(g, len(page), G, d))
        _put(cache, 1, page, at, 0.7 * _randn(g, len(page), G, d) + 0.1)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    B, G, d = case["B"], case["G"], case["d"]
    n = _lengths(case)
    s = {"case": case}
    if case["op"] == "decode":
        H = case["H"]
        s["cache"], s["table"] = _pages(case, n, g)
        _fill(s["cache"], g)
        s["seqlens"] = _ints(n)
        qw = (1 + 0.1 * _randn(g, d)).bfloat16()
        both = _randn(g, B, H, 2 * d).bfloat16()  # the query projection packs the queries with their gate
        s.update(q=both[..., :d], qw=qw)
        s["gate"] = {"elementwise": both[..., d:], "headwise": _randn(g, B, H).bfloat16(),
                     "head_shared": _randn(g, B, d).bfloat16(), "none": None}[case["gate"]]
        if case["append"]:
            s["k"], s["v"] = (_randn(g, B, G, d).bfloat16() for _ in range(2))
            s["kw"] = (1 + 0.1 * _randn(g, d)).bfloat16()
            s["starts"] = s["seqlens"] - 1
        return s
    before = _before(case)
    s["cache"], s["table"] = _pages(case, [a + b for a, b in zip(before, n)], g)
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    T = cu[-1]
    one = all(x == 1 for x in n)
    s.update(total=T, starts=_ints(before), cu=None if one else _ints(cu))
    dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    if case["op"] == "write":
        s["seqlens"] = _ints([a + b for a, b in zip(before, n)])
        if case["packed"]:  # K and V as slices of one projection's output
            both = _randn(g, T, 2, G, d).to(dt)
            s["k"], s["v"] = both[:, 0], both[:, 1]
        else:
            s["k"], s["v"] = _randn(g, T, G, d).to(dt), _randn(g, T, G, d).to(dt)
        s["kw"] = (1 + 0.1 * _randn(g, d)).to(dt)
    else:
        _fill(s["cache"], g)
        s["dtype"] = dt
    return s


# ------------------------------------------------------------------ one pass

def _token_places(s, page):
    """Sequence, position, page and slot of every token a write or read deals with."""
    starts, cu, T = s["starts"].long(), s["cu"], s["total"]
    t = torch.arange(T, device=DEV)
    b = t if cu is None else torch.searchsorted(cu[1:].contiguous(), t.int(), right=True)
    pos = starts[b] + (0 if cu is None else t - cu.long()[b])
    return b, pos, s["table"][b, pos // page].long(), pos % page


def _attend(s, case, dtype=torch.float32):
    B, H, G, d = case["B"], case["H"], case["G"], case["d"]
    L = s["seqlens"].long()
    table = s["table"].clamp(min=0)
    q = _norm_rope(s["q"], s["qw"], (L - 1).clamp(min=0), case["rd"], case["base"], dtype=dtype)
    live = torch.arange(table.shape[1] * case["page"], device=DEV)[None, :] < L[:, None]  # [B, Lmax]
    k = _whole(s["cache"], 0, table)
    x = torch.einsum("bgrd,bgld->bgrl", q.view(B, G, H // G, d), k) / math.sqrt(d)
    del k
    x = x.masked_fill(~live[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    v = _whole(s["cache"], 1, table).masked_fill(~live[:, None, :, None], 0)
    o = torch.einsum("bgrl,bgld->bgrd", p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.reshape(B, H, d)
    if s["gate"] is not None:
        z = s["gate"].to(dtype)
        z = z[..., None] if case["gate"] == "headwise" else z[:, None] if case["gate"] == "head_shared" else z
        o = o / (1 + torch.exp(-z))
    return o.reshape(B, H * d).bfloat16()


def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    page = case["page"]
    if case["op"] == "decode":
        if not case["append"]:
            return {"out": _attend(s, case)}
        pos = s["starts"].long()
        pg, slot = s["table"].gather(1, (pos // page)[:, None])[:, 0].long(), pos % page
        k = _norm_rope(s["k"], s["kw"], pos, case["rd"], case["base"], dtype=torch.float64).float()
        _put(s["cache"], 0, pg, slot, k)
        _put(s["cache"], 1, pg, slot, s["v"].float())
        return {"out": _attend(s, case), "k": _get(s["cache"], 0, pg, slot).bfloat16(),
                "v": _get(s["cache"], 1, pg, slot).bfloat16()}
    b, pos, pg, slot = _token_places(s, page)
    if case["op"] == "write":
        k = _norm_rope(s["k"], s["kw"], pos, case["rd"], case["base"], dtype=torch.float64).float()
        _put(s["cache"], 0, pg, slot, k)
        _put(s["cache"], 1, pg, slot, s["v"].float())
        dt = torch.bfloat16
    else:
        dt = s["dtype"]
    return {"k": _get(s["cache"], 0, pg, slot).to(dt), "v": _get(s["cache"], 1, pg, slot).to(dt)}


def _own(s, case):
    import gated_softmax_attention_gqa_gb300 as ga

    rope = dict(rotary_dim=case.get("rd"), rope_base=case.get("base"))
    if case["op"] == "decode":
        if "workspace" not in s:  # kept from step to step, as a serving loop does
            size = ga.gattn_decode_qcache_workspace_size(case["B"], case["H"], case["G"], case["d"],
                                                         s["table"].shape[1] * case["page"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
        new = dict(k_new=s["k"], v_new=s["v"], knorm_w=s["kw"]) if case["append"] else {}
        out = ga.gattn_decode_qcache(s["q"], s["cache"], s["table"], s["seqlens"], s["gate"], s["qw"],
                                     gate_mode=case["gate"], workspace=s["workspace"], **rope, **new)
        if not case["append"]:
            return {"out": out}
        k, v = ga.gattn_qcache_read(s["cache"], s["table"], s["starts"])
        return {"out": out, "k": k, "v": v}
    if case["op"] == "write":
        ga.gattn_qcache_write(s["k"], s["v"], s["cache"], s["table"], s["seqlens"], s["kw"], s["cu"], **rope)
    return dict(zip("kv", ga.gattn_qcache_read(s["cache"], s["table"], s["starts"], s["cu"], total=s["total"],
                                               dtype=torch.bfloat16 if case["op"] == "write" else s["dtype"])))


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_rows(cache, plane, page, slot):
    """fp64 values [n,G,d] of the rows `slot` of pages `page`, feature by feature from the layout."""
    _, num, G, blocks, row = cache.shape
    d = row // 10
    f = torch.arange(d, device=cache.device)
    byte = (f // 64) * 512 + 4 * (f % 32 // 4) + 2 * (f % 64 // 32) + f % 4 // 2  # of token 0 of a block
    par = 8 * d + (f // 32) * 32
    t = (slot % 16)[:, None]
    rows = cache[plane].permute(0, 2, 1, 3)[page, slot // 16]  # [n, G, 10 d]
    take = lambda at: rows.gather(2, at[:, None].expand(-1, G, -1)).long()  # noqa: E731
    code = (take(byte + 32 * t) >> (4 * (f % 2))) & 15
    half = lambda at: ((take(at + 2 * t + 1) << 24 | take(at + 2 * t) << 16).to(torch.int32)  # noqa: E731
                       .view(torch.float32).double())
    return half(par + d) + half(par) * (code.double() - 8)


def _exact_stored(x):
    """fp64 x [...,d] as the cache holds it."""
    out = torch.empty_like(x)
    for g in range(0, x.shape[-1], 32):
        y = x[..., g:g + 32]
        lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
        s = ((hi - lo) / 15).bfloat16().double()
        c = (lo + 8 * (hi - lo) / 15).bfloat16().double()
        r = torch.where(s > 0, (1 / s).float().double(), 0 * s)
        out[..., g:g + 32] = c + s * ((y - c) * r).round().clamp(-8, 7)
    return out


def _exact_rope(x, w, pos, rd, base):
    """fp64 RMSNorm and RoPE of x [n,heads,d] as complex rotations."""
    x = x.double()
    y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * w.double()
    h = rd // 2
    if h:
        i = torch.arange(h, device=x.device, dtype=torch.float64)
        turn = torch.polar(torch.ones(len(pos), h, device=x.device, dtype=torch.float64),
                           pos.double()[:, None] * torch.exp(-math.log(base) * 2 * i / rd))[:, None]
        z = torch.complex(y[..., :h].contiguous(), y[..., h:rd].contiguous()) * turn
        y = torch.cat((z.real, z.imag, y[..., rd:]), -1)
    return y


def exact(case, seed):
    s = prepare(case, seed)
    page, table = case["page"], s["table"].long()
    if case["op"] == "decode":
        H, G, d = case["H"], case["G"], case["d"]
        out, ks, vs = [], [], []
        for b, n in enumerate(_lengths(case)):
            o = torch.zeros(H, d, dtype=torch.float64, device=DEV)
            if n:
                pos = torch.arange(n, device=DEV)
                k, v = (_exact_rows(s["cache"], i, table[b, pos // page], pos % page) for i in (0, 1))
                last = pos[-1:]
                if case["append"]:
                    k[-1:] = _exact_stored(_exact_rope(s["k"][b:b + 1], s["kw"], last, case["rd"], case["base"]))
                    v[-1:] = _exact_stored(s["v"][b:b + 1].double())
                    ks.append(k[-1])
                    vs.append(v[-1])
                q = _exact_rope(s["q"][b:b + 1], s["qw"], last, case["rd"], case["base"])[0]
                for h in range(H):
                    a = torch.softmax(k[:, h * G // H] @ q[h] / math.sqrt(d), 0)
                    o[h] = a @ v[:, h * G // H]
            if s["gate"] is not None:
                z = s["gate"][b].double()
                o = o * torch.sigmoid(z[:, None] if case["gate"] == "headwise" else z)
            out.append(o.reshape(-1))
        got = {"out": torch.stack(out)}
        return got | {"k": torch.stack(ks), "v": torch.stack(vs)} if case["append"] else got
    seq = torch.tensor(_lengths(case), device=DEV)
    b = torch.repeat_interleave(torch.arange(case["B"], device=DEV), seq)
    pos = torch.arange(s["total"], device=DEV) - (seq.cumsum(0) - seq)[b] + s["starts"].long()[b]
    if case["op"] == "write":
        return {"k": _exact_stored(_exact_rope(s["k"], s["kw"], pos, case["rd"], case["base"])),
                "v": _exact_stored(s["v"].double())}
    pg = table[b, pos // page]
    return {n: _exact_rows(s["cache"], i, pg, pos % page) for i, n in enumerate("kv")}
