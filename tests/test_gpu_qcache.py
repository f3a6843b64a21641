"""GPU parity of the 4-bit KV cache: writing, reading back and decoding, against plain
references in 64 bits (tests/qcache_ref.py).

Tolerances.  A stored number is exact given its code, scale and centre, so a read is
compared for equality.  A written code is compared with the real-valued position of the
exact K' or V on the grid of the scale and centre that were written: at most half a step
away, plus what fp32 arithmetic adds -- K' carries a handful of 2^-24 roundings, taken as
2^-20 of the row's largest value, and the position itself one of 2^-24 of at most 16 steps
for each of a subtraction, a reciprocal and a product (2^-18 steps bounds them).  Decoding
rounds q' once to 11 or more bits and each softmax weight at most twice to bf16 (half a step
is 2^-8 of the value) before the products, and the output once: errors uniform over those
half steps have a relative rms of at most sqrt(3 * 2^-16 / 3) = 2^-8 where one key carries all
the weight, less where many do, and q' adds some 2^-11; REL = 5e-3 holds them, next to the
framework's bf16 bounds.  Scales and centres are bf16 too."""
import numpy as np
import pytest
import torch

from gated_softmax_attention_gqa_gb300 import (GattnError, gattn_decode_qcache, gattn_decode_qcache_workspace_size,
                                              gattn_get_device_status, gattn_qcache_read, gattn_qcache_shape,
                                              gattn_qcache_write)
from tests import qcache_ref as ref
from tests.parity import assert_close_to_oracle, gate_scale

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BAD_SEQLEN, BAD_PAGE = 0x1, 0x4
REL = 5e-3


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def make_pool(reach, G, page, d, seed, spare=2, fill=255):
    """A pool of garbage bytes (NaN scales) and a table over shuffled pages; unused entries are -1."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in reach]
    num = sum(need) + spare
    perm, at = rng.permutation(num), 0
    table = np.full((len(reach), max(1, max(need))), -1, np.int32)
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    cache = torch.full(gattn_qcache_shape(num, G, page, d), fill, dtype=torch.uint8, device=DEV)
    return cache, torch.from_numpy(table).to(DEV)


def check_rows(cache, table, b, g, plane, x, first):
    """Codes, scales and centres of the rows of exact values x [n,d] (fp64), tokens first.. of b."""
    page = 16 * cache.shape[3]
    for i, y in enumerate(x):
        pos = first + i
        n, s, c = ref.rows(cache, plane, int(table[b, pos // page]), g, pos % page)
        grp = y.reshape(-1, 32)
        step = (grp.max(-1) - grp.min(-1)) / 15
        want_c = grp.min(-1) + 8 * step
        slack = 2.0 ** -20 * np.abs(y).max()
        assert (np.abs(s - step) <= 2.0 ** -8 * step + slack).all(), (b, pos, "scale")
        assert (np.abs(c - want_c) <= 2.0 ** -8 * np.abs(want_c) + slack).all(), (b, pos, "centre")
        S, C = np.repeat(s, 32), np.repeat(c, 32)
        live = S > 0
        t = np.clip((y - C)[live] / S[live], -8, 7)
        assert (np.abs(n[live] - t) <= 0.5 + 2.0 ** -18 + slack / S[live]).all(), (b, pos, "code")
        assert (n[~live] == 0).all()


WRITES = [
    # d, G, page, rd, base, dtype, new tokens, cached before, strided
    (64, 1, 16, 0, 1e4, torch.bfloat16, [1], [0], False),
    (64, 3, 32, 64, 1e4, torch.float32, [5, 0, 33], [7, 3, 0], True),
    (128, 2, 64, 128, 1e6, torch.bfloat16, [17, 70, 1, 16], [0, 15, 63, 48], True),
    (128, 5, 16, 48, 1e6, torch.float32, [40], [9], False),
    (256, 2, 128, 64, 1e7, torch.bfloat16, [129, 3], [0, 126], True),
    (256, 1, 48, 256, 1e7, torch.bfloat16, [50, 31], [1, 47], False),
]


@pytest.mark.parametrize("case", WRITES, ids=str)
def test_write_and_read_back(case):
    d, G, page, rd, base, dt, new, before, strided = case
    T, seed = sum(new), d + G
    g = torch.Generator().manual_seed(seed)
    reach = [a + n for a, n in zip(before, new)]
    cache, table = make_pool(reach, G, page, d, seed)
    kv = torch.randn(T, 2, G, d, generator=g).to(dt)
    kw = (1 + 0.1 * torch.randn(d, generator=g)).to(dt)
    dev = kv.to(DEV)
    k, v = (dev[:, 0], dev[:, 1]) if strided else (dev[:, 0].contiguous(), dev[:, 1].contiguous())
    cu = i32(np.concatenate([[0], np.cumsum(new)]).tolist())
    before_bytes = cache.cpu().numpy().copy()
    gattn_qcache_write(k, v, cache, table, i32(reach), kw.to(DEV), cu, rotary_dim=rd, rope_base=base)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    raw, tab = cache.cpu().numpy(), table.cpu().numpy()
    touched = np.zeros_like(raw, dtype=bool)
    byte, _, par = ref.layout(d)
    at = 0
    for b, n in enumerate(new):
        pos = np.arange(before[b], before[b] + n)
        K = ref.norm_rope(kv[at:at + n, 0].double().numpy(), kw.double().numpy(), pos, rd, base)
        V = kv[at:at + n, 1].double().numpy()
        for gg in range(G):
            check_rows(raw, tab, b, gg, 0, K[:, gg], before[b])
            check_rows(raw, tab, b, gg, 1, V[:, gg], before[b])
        for p in pos:
            t = p % 16
            cols = np.unique(np.concatenate([byte + 32 * t, *(par + o + 2 * t + h for o in (0, d) for h in (0, 1))]))
            touched[:, tab[b, p // page], :, (p % page) // 16][..., cols] = True
            blk = touched[:, tab[b, p // page], :, (p % page) // 16]
            blk[..., cols] = True
            touched[:, tab[b, p // page], :, (p % page) // 16] = blk
        # V is quantised from its given bits: every code, scale and centre is reproducible
        n_ref, s_ref, c_ref = ref.encode(kv[at:at + n, 1].float().numpy())
        for i, p in enumerate(pos):
            for gg in range(G):
                got = ref.rows(raw, 1, tab[b, p // page], gg, p % page)
                assert all((x == y).all() for x, y in zip(got, (n_ref[i, gg], s_ref[i, gg], c_ref[i, gg])))
        at += n
    assert (raw[~touched] == before_bytes[~touched]).all(), "bytes of other rows changed"
    # and back, in both types, rows past the last left alone
    for out_dt in (torch.bfloat16, torch.float32):
        ko = torch.full((T + 3, G, d), 7.0, dtype=out_dt, device=DEV)
        vo = ko.clone()
        gattn_qcache_read(cache, table, i32(before), cu, k_out=ko, v_out=vo)
        torch.cuda.synchronize()
        at = 0
        for b, n in enumerate(new):
            K, V = ref.values(raw, tab, b, before[b], before[b] + n)
            for got, want in ((ko, K), (vo, V)):
                want = torch.from_numpy(want).to(out_dt)
                assert torch.equal(got[at:at + n].cpu(), want)
            at += n
        assert (ko[T:] == 7).all() and (vo[T:] == 7).all()
    assert gattn_get_device_status() == 0


def test_one_token_each_skips_unused_rows():
    d, G, page = 128, 2, 32
    lens = [0, 1, 16, 33, 0, 64]
    cache, table = make_pool(lens, G, page, d, 5)
    before = cache.clone()
    g = torch.Generator().manual_seed(3)
    k, v = torch.randn(2, len(lens), G, d, generator=g).to(torch.bfloat16)
    kw = torch.ones(d, dtype=torch.bfloat16)
    gattn_qcache_write(k.to(DEV), v.to(DEV), cache, table, i32(lens), kw.to(DEV), rotary_dim=64, rope_base=1e4)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    raw, tab = cache.cpu().numpy(), table.cpu().numpy()
    for b, L in enumerate(lens):
        if L:
            K = ref.norm_rope(k[b:b + 1].double().numpy(), kw.double().numpy(), [L - 1], 64, 1e4)
            for gg in range(G):
                check_rows(raw, tab, b, gg, 0, K[:, gg], L - 1)
                check_rows(raw, tab, b, gg, 1, v[b:b + 1, gg].double().numpy(), L - 1)
    live = sum(L > 0 for L in lens)
    assert int((cache != before).sum()) <= 2 * G * live * (d // 2 + d // 8)
    # starts picks one cached token of each sequence; an unused row's range is refused
    ko = torch.zeros(len(lens), G, d, dtype=torch.float32, device=DEV)
    vo = torch.zeros_like(ko)
    gattn_qcache_read(cache, table, i32([L - 1 for L in lens]), k_out=ko, v_out=vo)
    torch.cuda.synchronize()
    assert gattn_get_device_status() & BAD_SEQLEN
    for b, L in enumerate(lens):
        want = ref.values(raw, tab, b, L - 1, L)[1][0] if L else np.zeros((G, d))
        assert (vo[b].double().cpu().numpy() == want.astype(np.float32)).all()


def test_awkward_values():
    """Constant, zero, tiny, huge, far-from-zero, infinite and NaN groups of V."""
    d, G = 64, 1
    base = torch.randn(32, generator=torch.Generator().manual_seed(1))
    groups = [torch.zeros(32), torch.full((32,), 3.0), base * 1e-30, base * 1e-38, base.sign() * 3e38, 100 + base,
              torch.where(torch.arange(32) == 5, float("inf"), base), torch.where(torch.arange(32) == 9, float("nan"), base),
              torch.where(torch.arange(32) == 0, 50.0, 0.01 * base), -base.abs(), torch.full((32,), 1e-41),
              torch.arange(32.0)]
    v = torch.stack(groups).reshape(-1, G, d).to(torch.bfloat16)
    T = v.shape[0]
    cache, table = make_pool([T], G, 16, d, 1)
    k = torch.randn(T, G, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    k[1, 0, 3], k[2, 0, 60] = float("nan"), float("inf")
    gattn_qcache_write(k.to(DEV), v.to(DEV), cache, table, i32([T]), torch.ones(d, dtype=torch.bfloat16, device=DEV),
                       i32([0, T]), rotary_dim=0, rope_base=1e4)
    ko, vo = gattn_qcache_read(cache, table, None, i32([0, T]), total=T, dtype=torch.float32)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    got = vo.cpu().reshape(-1, 32)
    x = v.float().reshape(-1, 32)
    for i in range(len(groups)):
        if not torch.isfinite(x[i]).all():
            assert got[i].isnan().all(), i
            continue
        n, s, c = ref.encode(x[i].numpy())
        want = torch.from_numpy((c + s * n).astype(np.float32))
        assert torch.equal(got[i], want), i
        step = float(x[i].max().double() - x[i].min().double()) / 15
        # half a step, the clamped ends (the scale's rounding over 8 steps), the centre's rounding
        bound = 0.5 * step + 8 * 2.0 ** -8 * step + 2.0 ** -8 * float(x[i].abs().max()) + 1e-37
        assert float((got[i] - x[i]).abs().max()) <= bound, i
    assert ko[0].isfinite().all() and ko[1].isnan().all()  # a NaN reaches its row's norm
    assert ko[2, 0, 32:].isnan().all()                     # an infinity its group


DECODES = [
    # H, G, d, rd, base, page, lengths
    (8, 2, 256, 64, 1e7, 64, [1, 64, 65, 300, 0, 127]),
    (16, 8, 128, 128, 1e6, 16, [15, 16, 17, 129, 1]),
    (32, 4, 128, 64, 1e6, 256, [700, 2, 1025]),
    (4, 4, 64, 32, 1e4, 48, [63, 129, 0, 31, 47, 48, 49]),
    (7, 1, 64, 0, 1e4, 32, [33, 500]),
    (10, 2, 128, 16, 1e4, 64, [2000]),
    (6, 3, 256, 256, 1e4, 32, [95, 96, 97]),
    (8, 2, 256, 64, 1e7, 64, [8192]),
]


def decode_inputs(H, G, d, rd, base, page, lens, seed, layout="elementwise"):
    g = torch.Generator().manual_seed(seed)
    cache, table = make_pool(lens, G, page, d, seed)
    T = sum(lens)
    k = torch.randn(T, G, d, generator=g).to(torch.bfloat16)
    v = (0.2 + torch.randn(T, G, d, generator=g)).to(torch.bfloat16)
    kw = (1 + 0.1 * torch.randn(d, generator=g)).to(torch.bfloat16)
    cu = i32(np.concatenate([[0], np.cumsum(lens)]).tolist())
    gattn_qcache_write(k.to(DEV), v.to(DEV), cache, table, i32(lens), kw.to(DEV), cu, rotary_dim=rd, rope_base=base)
    B = len(lens)
    qg = torch.randn(B, H, 2 * d, generator=g).to(torch.bfloat16)
    gate = {"elementwise": qg[..., d:], "headwise": qg[:, :, d], "head_shared": qg[:, 0, d:], "none": None}[layout]
    qw = (1 + 0.1 * torch.randn(d, generator=g)).to(torch.bfloat16)
    return dict(cache=cache, table=table, seqlens=i32(lens), qg=qg, gate=gate, qw=qw, kw=kw)


def expected(x, lens, rd, base, layout="elementwise", **kw):
    raw, tab = x["cache"].cpu().numpy(), x["table"].cpu().numpy()
    d = raw.shape[-1] // 10
    outs = []
    for b, L in enumerate(lens):
        K, V = ref.values(raw, tab, b, 0, L)
        z = None
        if layout != "none":
            z = x["gate"][b].double().numpy()
            z = z[:, None] if layout == "headwise" else z
        outs.append(ref.decode(x["qg"][b, :, :d].double().numpy(), K, V, z, x["qw"].double().numpy(), L, rd, base, **kw))
    return np.stack([o.reshape(-1) for o in outs])


def run_decode(x, d, rd, base, layout="elementwise", **kw):
    qg = x["qg"].to(DEV)
    gate = x["gate"]
    if layout == "elementwise":
        gate = qg[..., d:]
    elif gate is not None:
        gate = gate.contiguous().to(DEV)
    return gattn_decode_qcache(qg[..., :d], x["cache"], x["table"], x["seqlens"], gate, x["qw"].to(DEV), rotary_dim=rd,
                               rope_base=base, gate_mode=layout, **kw)


def assert_close(out, want, what, scale=None):
    assert_close_to_oracle(out, want, torch.bfloat16, what, scale=scale)
    got = out.double().cpu().numpy()
    rel = np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-30)
    assert rel <= REL, f"{what}: rel {rel:.2e}"


@pytest.mark.parametrize("case", DECODES, ids=str)
def test_decode(case):
    H, G, d, rd, base, page, lens = case
    x = decode_inputs(*case, seed=H + d)
    out = run_decode(x, d, rd, base)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    assert_close(out, expected(x, lens, rd, base), str(case))


@pytest.mark.parametrize("layout", ["elementwise", "headwise", "head_shared", "none"])
def test_decode_gates(layout):
    H, G, d, rd, base, page, lens = 8, 2, 128, 64, 1e6, 32, [77, 0, 200]
    x = decode_inputs(H, G, d, rd, base, page, lens, seed=9, layout=layout)
    sig = lambda z: 1 / (1 + np.exp(-z))  # noqa: E731
    acts = {"sigmoid": sig, "ns_sigmoid": lambda z: 0.5 + 0.5 * sig(z), "silu": lambda z: z * sig(z)}
    for act, additive in [("sigmoid", False)] + ([] if layout == "none" else [
            ("ns_sigmoid", False), ("silu", False), ("silu", True), ("sigmoid", True)]):
        out = run_decode(x, d, rd, base, layout, gate_act=act, gate_additive=additive)
        torch.cuda.synchronize()
        want = expected(x, lens, rd, base, layout, act=acts[act], additive=additive)
        scale = None
        if layout != "none":
            scale = gate_scale(x["gate"].double().numpy(), layout, act, want.shape)
        assert_close(out, want, f"{layout} {act} {additive}", scale)
    assert gattn_get_device_status() == 0


@pytest.mark.parametrize("case", [(8, 2, 256, 64, 1e7, 64, [1, 64, 65, 300]), (16, 8, 128, 128, 1e6, 16, [15, 0, 17, 129]),
                                  (4, 4, 64, 32, 1e4, 48, [49, 96, 2])], ids=str)
def test_decode_appends_the_new_token(case):
    H, G, d, rd, base, page, lens = case
    x = decode_inputs(*case, seed=d + 1)
    g = torch.Generator().manual_seed(4)
    k, v = torch.randn(2, len(lens), G, d, generator=g).to(torch.bfloat16)
    alone = x["cache"].clone()
    gattn_qcache_write(k.to(DEV), v.to(DEV), alone, x["table"], x["seqlens"], x["kw"].to(DEV), rotary_dim=rd,
                       rope_base=base)
    out = run_decode(x, d, rd, base, k_new=k.to(DEV), v_new=v.to(DEV), knorm_w=x["kw"].to(DEV))
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    assert torch.equal(alone, x["cache"]), "the append writes what gattn_qcache_write writes"
    assert_close(out, expected(x, lens, rd, base), str(case))


def test_positions_far_into_a_long_sequence():
    """Tokens near position 131071, fp32: the rotation angle is exact to fp32 rounding of its
    sine.  Only the last page exists; the entries before it name no page and are not read."""
    d, G, page, rd, base = 128, 2, 64, 128, 1e6
    L = 131072
    cache, _ = make_pool([page], G, page, d, 3, spare=0)
    table = torch.full((1, L // page), -1, dtype=torch.int32, device=DEV)
    table[0, -1] = 0
    g = torch.Generator().manual_seed(8)
    k, v = torch.randn(2, 5, G, d, generator=g)
    kw = torch.ones(d)
    gattn_qcache_write(k.to(DEV), v.to(DEV), cache, table, i32([L]), kw.to(DEV), i32([0, 5]), rotary_dim=rd, rope_base=base)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    K = ref.norm_rope(k.double().numpy(), kw.double().numpy(), np.arange(L - 5, L), rd, base)
    for gg in range(G):
        check_rows(cache.cpu().numpy(), table.cpu().numpy(), 0, gg, 0, K[:, gg], L - 5)


def test_offsets_past_32_bits():
    """A pool of more than 4 GB a plane: the last pages are written, read back and attended."""
    d, G, page, rd, base = 256, 2, 256, 64, 1e7
    num = (1 << 32) // (page // 16 * 10 * d * G) + 9
    cache = torch.empty(gattn_qcache_shape(num, G, page, d), dtype=torch.uint8, device=DEV)
    assert cache.numel() > 1 << 33
    lens = [300, 40]
    table = i32([[num - 1, 5], [num - 2, -1]])
    g = torch.Generator().manual_seed(6)
    k, v = torch.randn(2, sum(lens), G, d, generator=g).to(torch.bfloat16)
    kw = torch.ones(d, dtype=torch.bfloat16)
    cu = i32([0, 300, 340])
    gattn_qcache_write(k.to(DEV), v.to(DEV), cache, table, i32(lens), kw.to(DEV), cu, rotary_dim=rd, rope_base=base)
    ko, vo = gattn_qcache_read(cache, table, None, cu, total=340, dtype=torch.float32)
    qg = torch.randn(2, 8, 2 * d, generator=g).to(torch.bfloat16)
    small = dict(cache=cache[:, [5, num - 2, num - 1]].contiguous(), table=i32([[2, 0], [1, -1]]))
    x = dict(qg=qg, gate=qg[..., d:], qw=kw, seqlens=i32(lens), **small)
    out = run_decode(dict(x, cache=cache, table=table), d, rd, base)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    raw, tab = small["cache"].cpu().numpy(), small["table"].cpu().numpy()
    for b, (lo, hi) in enumerate([(0, 300), (300, 340)]):
        K, V = ref.values(raw, tab, b, 0, hi - lo)
        assert (ko[lo:hi].cpu().numpy() == K.astype(np.float32)).all()
        assert (vo[lo:hi].cpu().numpy() == V.astype(np.float32)).all()
    assert (np.abs(vo.cpu().numpy() - v.float().numpy()) < 0.5).all()
    assert_close(out, expected(x, lens, rd, base), "far pages")


def test_bad_lengths_and_pages_are_reported_and_skipped():
    H, G, d, rd, base, page = 8, 2, 128, 64, 1e6, 32
    lens = [40, 50, 60, 64]
    x = decode_inputs(H, G, d, rd, base, page, lens, seed=2)
    want = expected(x, lens, rd, base)
    x["seqlens"] = i32([40, -1, 65, 64])  # two pages of 32: at most 64
    out = torch.full((4, H * d), 3.0, dtype=torch.bfloat16, device=DEV)
    before = x["cache"].clone()
    k = torch.randn(4, G, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    gattn_get_device_status()
    run_decode(x, d, rd, base, out=out)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == BAD_SEQLEN
    assert (out[1:3] == 3).all()
    assert_close(out[[0, 3]], want[[0, 3]], "good rows next to bad ones")
    gattn_qcache_write(k, k, x["cache"], x["table"], x["seqlens"], x["kw"].to(DEV), rotary_dim=rd, rope_base=base)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == BAD_SEQLEN
    changed = (x["cache"] != before).flatten(2).any(2).any(0).nonzero()[:, 0].tolist()
    assert set(changed) <= {int(x["table"][0, 1]), int(x["table"][3, 1])}
    # pages outside the pool: nothing is touched, the others' rows are right
    x["seqlens"] = i32(lens)
    num = x["cache"].shape[1]
    bad = x["table"].clone()
    bad[1, 1], bad[2, 0] = num, -5
    snap = x["cache"].clone()
    ko = torch.full((4, G, d), 5.0, dtype=torch.bfloat16, device=DEV)
    vo = ko.clone()
    gattn_qcache_read(x["cache"], bad, i32([10, 40, 3, 63]), k_out=ko, v_out=vo)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == BAD_PAGE
    assert (ko[1:3] == 5).all() and (vo[1:3] == 5).all() and not (ko[0] == 5).all() and not (vo[3] == 5).all()
    gattn_qcache_write(k[1:3].contiguous(), k[1:3].contiguous(), x["cache"], bad[1:3].contiguous(), i32([50, 20]),
                       x["kw"].to(DEV), rotary_dim=rd, rope_base=base)
    run_decode(dict(x, table=bad), d, rd, base, out=out)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == BAD_PAGE
    assert torch.equal(snap, x["cache"])
    assert_close(out[3:], expected(x, lens, rd, base)[3:], "a good row next to bad pages")
    # a sequence shorter than its new tokens, next to one that is right
    gattn_qcache_write(k, k, x["cache"], x["table"], i32([1, 50, 60, 64]), x["kw"].to(DEV), i32([0, 2, 2, 3, 4]),
                       rotary_dim=rd, rope_base=base)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == BAD_SEQLEN
    changed = (x["cache"] != snap).flatten(2).any(2).any(0).nonzero()[:, 0].tolist()
    assert set(changed) == {int(x["table"][2, 1])}  # sequence 3's row already held the same token


def test_workspace_is_checked():
    x = decode_inputs(8, 2, 128, 64, 1e6, 32, [40], seed=3)
    need = gattn_decode_qcache_workspace_size(1, 8, 2, 128, 64)
    with pytest.raises(GattnError):
        run_decode(x, 128, 64, 1e6, workspace=torch.empty(need - 256, dtype=torch.uint8, device=DEV))
    run_decode(x, 128, 64, 1e6, workspace=torch.empty(need, dtype=torch.uint8, device=DEV))


def test_another_stream_and_two_calls_at_once():
    """Calls on their own streams, each with its own workspace, beside work on the default one."""
    cases = [(8, 2, 256, 64, 1e7, 64, [3000, 40]), (16, 8, 128, 128, 1e6, 16, [900, 901, 17])]
    xs = [decode_inputs(*c, seed=i) for i, c in enumerate(cases)]
    on_gpu = [(x["qg"].to(DEV), x["qw"].to(DEV)) for x in xs]

    def call(x, c, qg, qw, stream=None):
        d = c[2]
        return gattn_decode_qcache(qg[..., :d], x["cache"], x["table"], x["seqlens"], qg[..., d:], qw, rotary_dim=c[3],
                                   rope_base=c[4], stream=stream)

    plain = [call(x, c, *t) for x, c, t in zip(xs, cases, on_gpu)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        outs = [call(x, c, *t, stream=s) for x, c, t, s in zip(xs, cases, on_gpu, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, plain))
    assert gattn_get_device_status() == 0


def test_captured_steps_follow_lengths_and_tables():
    """A captured step (append, decode, read back) is replayed with other lengths, tokens and pages."""
    H, G, d, rd, base, page = 8, 2, 128, 64, 1e6, 16
    lens = [30, 5, 64]
    x = decode_inputs(H, G, d, rd, base, page, [80, 80, 80], seed=12)
    x["seqlens"].copy_(i32(lens))
    qg = x["qg"].to(DEV)
    k, v = torch.randn(2, 3, G, d, device=DEV).to(torch.bfloat16)
    kw, qw = x["kw"].to(DEV), x["qw"].to(DEV)
    starts = x["seqlens"] - 1
    ws = torch.empty(gattn_decode_qcache_workspace_size(3, H, G, d, x["table"].shape[1] * page), dtype=torch.uint8,
                     device=DEV)

    def step():
        out = gattn_decode_qcache(qg[..., :d], x["cache"], x["table"], x["seqlens"], qg[..., d:], qw, rotary_dim=rd,
                                  rope_base=base, k_new=k, v_new=v, knorm_w=kw, workspace=ws)
        return (out, *gattn_qcache_read(x["cache"], x["table"], starts))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        lens = [n + 1 for n in lens] if i < 3 else [1, 80, 0]
        x["seqlens"].copy_(i32(lens))
        starts.copy_(i32([max(n - 1, 0) for n in lens]))
        x["table"].copy_(x["table"][[1, 2, 0]])
        x["qg"] = torch.randn(3, H, 2 * d, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16)
        x["gate"] = x["qg"][..., d:]
        qg.copy_(x["qg"])
        k.normal_(), v.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert gattn_get_device_status() == 0
        assert_close(got[0], expected(x, lens, rd, base), f"replay {i}")
        raw, tab = x["cache"].cpu().numpy(), x["table"].cpu().numpy()
        for b, n in enumerate(lens):
            if n:
                V = ref.values(raw, tab, b, n - 1, n)[1]
                assert torch.equal(got[2][b].cpu(), torch.from_numpy(V[0]).to(torch.bfloat16))
                assert (np.abs(V[0] - v[b].double().cpu().numpy()) < 0.6).all()


def test_results_repeat_bit_for_bit():
    x = decode_inputs(8, 2, 256, 64, 1e7, 64, [5000, 300, 70], seed=7)
    a = run_decode(x, 256, 64, 1e7)
    for _ in range(3):
        assert torch.equal(a, run_decode(x, 256, 64, 1e7))


def test_a_prompt_then_steps():
    """The operators as a server uses them: prompts written in two chunks, steps that append and
    attend, the cache read back, each step against the 64-bit reference over the raw tokens' stored
    values; and the whole close to attention over unquantised K' and V."""
    H, G, d, rd, base, page = 8, 2, 128, 64, 1e6, 32
    prompt, steps = [70, 33, 1], 4
    B, T = len(prompt), sum(prompt)
    g = torch.Generator().manual_seed(21)
    cache, table = make_pool([n + steps for n in prompt], G, page, d, 21)
    kw, qw = ((1 + 0.1 * torch.randn(d, generator=g)).to(torch.bfloat16) for _ in range(2))
    K = [torch.randn(n + steps, G, d, generator=g).to(torch.bfloat16) for n in prompt]
    V = [torch.randn(n + steps, G, d, generator=g).to(torch.bfloat16) for n in prompt]
    rope = dict(rotary_dim=rd, rope_base=base)
    first = [n // 2 for n in prompt]
    for lo, hi in (([0] * B, first), (first, prompt)):
        n = [b - a for a, b in zip(lo, hi)]
        kk, vv = (torch.cat([t[b][lo[b]:hi[b]] for b in range(B)]).to(DEV) for t in (K, V))
        gattn_qcache_write(kk, vv, cache, table, i32(hi), kw.to(DEV), i32(np.concatenate([[0], np.cumsum(n)]).tolist()), **rope)
    for s in range(steps):
        lens = [n + s + 1 for n in prompt]
        qg = torch.randn(B, H, 2 * d, generator=g).to(torch.bfloat16)
        x = dict(cache=cache, table=table, seqlens=i32(lens), qg=qg, gate=qg[..., d:], qw=qw)
        kn, vn = (torch.stack([t[b][prompt[b] + s] for b in range(B)]).to(DEV) for t in (K, V))
        out = run_decode(x, d, rd, base, k_new=kn, v_new=vn, knorm_w=kw.to(DEV))
        torch.cuda.synchronize()
        assert_close(out, expected(x, lens, rd, base), f"step {s}")
        for b, L in enumerate(lens):
            k64 = ref.norm_rope(K[b][:L].double().numpy(), kw.double().numpy(), np.arange(L), rd, base)
            o = ref.decode(qg[b, :, :d].double().numpy(), k64, V[b][:L].double().numpy(), qg[b, :, d:].double().numpy(),
                           qw.double().numpy(), L, rd, base).reshape(-1)
            # steps of about 0.28 of the values' spread: an rms error of 0.28 / sqrt(12) = 8 per cent of V,
            # and as much of each logit's unit spread again through the weights
            assert np.linalg.norm(out[b].double().cpu().numpy() - o) <= 0.25 * np.linalg.norm(o)
    ends = [n + steps for n in prompt]
    cu = i32(np.concatenate([[0], np.cumsum(ends)]).tolist())
    ko, vo = gattn_qcache_read(cache, table, None, cu, total=sum(ends))
    torch.cuda.synchronize()
    allk, allv = torch.cat(K), torch.cat(V)
    want = np.concatenate([ref.norm_rope(t.double().numpy(), kw.double().numpy(), np.arange(len(t)), rd, base) for t in K])
    for got, y in ((ko, want), (vo, allv.double().numpy())):
        assert np.linalg.norm(got.double().cpu().numpy() - y) <= 0.12 * np.linalg.norm(y)
    assert ko.shape == allk.shape and gattn_get_device_status() == 0


def written_values(v, page=16, before=0):
    """V rows [T,G,d] written to a fresh cache after `before` tokens and read back in fp32 (fp64 on the CPU)."""
    T, G, d = v.shape
    cache, table = make_pool([before + T], G, page, d, 1)
    cu = i32([0, T])
    w = torch.ones(d, dtype=v.dtype, device=DEV)
    gattn_qcache_write(v.to(DEV), v.to(DEV), cache, table, i32([before + T]), w, cu, rotary_dim=0, rope_base=1e4)
    out = gattn_qcache_read(cache, table, i32([before]), cu, total=T, dtype=torch.float32)[1]
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    return out.double().cpu().numpy()


def test_every_scale_rounds_ties_by_its_exact_reciprocal():
    """Groups whose scale is each normal bf16 s of 2^-100 .. 2^100, and whose numbers lie half way
    between two codes: which way one goes shows the last bit of 1 / s.  Extremes -7.5 s and 7.5 s
    give the step s (1 + 2^-24 at most) and the centre s / 2, both exact."""
    s = (1 + torch.arange(128, dtype=torch.float64) / 128)[None] * 2.0 ** torch.arange(-100, 101, dtype=torch.float64)[:, None]
    k = torch.arange(32) % 14 - 7.0
    x = (0.5 + k + 0.5)[None] * s.reshape(-1, 1)
    x[:, 0], x[:, 1] = -7.5 * s.reshape(-1), 7.5 * s.reshape(-1)
    x = x.float()
    n, sc, c = ref.encode(x.numpy())
    assert (sc.reshape(-1) == s.reshape(-1).numpy()).all()
    pad = -x.shape[0] % 8
    got = written_values(torch.cat([x, x[:pad]]).reshape(-1, 1, 256)).reshape(-1, 32)[:x.shape[0]]
    assert (got == (c + sc * n).astype(np.float32)).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_codes_clamped_where_the_centre_is_coarse(d, dt):
    """A spread that is small against the values: the centre's rounding pushes codes past both ends."""
    g = torch.Generator().manual_seed(d)
    far = torch.tensor([1000.0, -333.0, 77.0, 5.0])[torch.arange(24) % 4][:, None, None]
    v = (far + 0.02 * torch.rand(24, 2, d, generator=g) * far.abs()).to(dt)
    n, s, c = ref.encode(v.float().numpy())
    want = (np.repeat(c, 32, -1) + np.repeat(s, 32, -1) * n).astype(np.float32)
    assert (np.abs(n) >= 7).any()
    assert (written_values(v, before=5) == want).all()


@pytest.mark.parametrize("r", range(1, 9))
@pytest.mark.parametrize("d,rd", [(64, 48), (128, 16), (256, 112)])
def test_decode_every_ratio_of_heads(r, d, rd):
    case = (2 * r, 2, d, rd, 1e5, 48, [191, 1, 193, 385, 47])
    x = decode_inputs(*case, seed=r)
    out = run_decode(x, d, rd, 1e5)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    assert_close(out, expected(x, case[-1], rd, 1e5), str(case))


@pytest.mark.parametrize("d,page", [(128, 16), (128, 48), (128, 4096), (64, 80), (256, 1024)])
def test_decode_lengths_around_tiles_and_pages(d, page):
    """Every length around the ends of a warp's blocks and of a tile, in pages that end inside both."""
    lens = [*range(15, 19), *range(31, 34), *range(47, 50), *range(95, 98), *range(127, 130), *range(191, 194),
            *range(255, 258), 383, 384, 385, 577]
    x = decode_inputs(4, 2, d, 32, 1e4, page, lens, seed=page)
    out = run_decode(x, d, 32, 1e4)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    assert_close(out, expected(x, lens, 32, 1e4), f"{d} {page}")


@pytest.mark.parametrize("scale", [1e-20, 1e30])
def test_decode_of_small_and_large_values(scale):
    """V of far magnitudes: fp32 sums and bf16 operands carry them alike."""
    H, G, d, page, lens = 4, 2, 128, 32, [40, 300]
    x = decode_inputs(H, G, d, 64, 1e4, page, lens, seed=31)
    g = torch.Generator().manual_seed(32)
    k = torch.randn(sum(lens), G, d, generator=g).to(torch.bfloat16)
    v = (scale * torch.randn(sum(lens), G, d, generator=g)).to(torch.bfloat16)
    cu = i32([0, lens[0], sum(lens)])
    gattn_qcache_write(k.to(DEV), v.to(DEV), x["cache"], x["table"], x["seqlens"], x["kw"].to(DEV), cu, rotary_dim=64,
                       rope_base=1e4)
    out = run_decode(x, d, 64, 1e4)
    torch.cuda.synchronize()
    want = expected(x, lens, 64, 1e4)
    assert_close((out.float() / scale).to(torch.bfloat16), want / scale, f"{scale}")


def test_the_largest_batch_mostly_unused():
    """2048 rows of which a few hold tokens: the others get the gate of an empty sum."""
    H, G, d, page = 2, 1, 64, 16
    lens = [0] * 2048
    for b, n in ((0, 3), (7, 40), (1000, 17), (1023, 200), (1024, 1), (2047, 65)):
        lens[b] = n
    x = decode_inputs(H, G, d, 32, 1e4, page, lens, seed=41)
    out = run_decode(x, d, 32, 1e4)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    assert_close(out, expected(x, lens, 32, 1e4), "2048 rows")
    assert (out[[b for b in range(2048) if not lens[b]]] == 0).all()


def test_every_row_unused():
    x = decode_inputs(8, 2, 128, 64, 1e6, 32, [4, 4], seed=2)
    x["seqlens"].zero_()
    before = x["cache"].clone()
    k = torch.ones(2, 2, 128, dtype=torch.bfloat16, device=DEV)
    out = run_decode(x, 128, 64, 1e6, k_new=k, v_new=k, knorm_w=x["kw"].to(DEV))
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    assert (out == 0).all() and torch.equal(before, x["cache"])


@pytest.mark.parametrize("case", [(64, 1, 16, torch.bfloat16, 1, 3), (128, 8, 32, torch.bfloat16, 3, 700),
                                  (256, 5, 64, torch.float32, 2, 900), (64, 3, 48, torch.float32, 40, 31),
                                  (256, 2, 64, torch.bfloat16, 2, 9001), (128, 1, 16, torch.bfloat16, 1, 40000)], ids=str)
def test_write_of_many_sizes(case):
    """Short calls, whose heads are spread, and long ones, of several passes a warp, in a padded
    batch: V exactly, K against its exact values, padding and other rows untouched."""
    d, G, page, dt, B, n = case
    g = torch.Generator().manual_seed(n)
    new = [n] + [int(torch.randint(0, 40, (1,), generator=g)) for _ in range(B - 1)]
    before = [int(torch.randint(0, 100, (1,), generator=g)) for _ in range(B)]
    T, reach = sum(new), [a + b for a, b in zip(new, before)]
    cache, table = make_pool(reach, G, page, d, n)
    kv = torch.randn(T + 5, G, 2, d, generator=g).to(dt).to(DEV)  # five rows of padding, heads strided
    kw = (1 + 0.1 * torch.randn(d, generator=g)).to(dt)
    cu = i32(np.concatenate([[0], np.cumsum(new)]).tolist())
    gattn_qcache_write(kv[:, :, 0], kv[:, :, 1], cache, table, i32(reach), kw.to(DEV), cu, rotary_dim=d // 2, rope_base=1e6)
    ko, vo = gattn_qcache_read(cache, table, i32(before), cu, total=T, dtype=torch.float32)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    m, s, c = ref.encode(kv[:T, :, 1].float().cpu().numpy())
    want = (np.repeat(c, 32, -1) + np.repeat(s, 32, -1) * m).astype(np.float32)
    assert (vo.cpu().numpy() == want).all()
    pos = np.concatenate([np.arange(a, b) for a, b in zip(before, reach)])
    K = ref.norm_rope(kv[:T, :, 0].double().cpu().numpy(), kw.double().numpy(), pos, d // 2, 1e6)
    grp = K.reshape(T, G, -1, 32)
    step = np.repeat((grp.max(-1) - grp.min(-1)) / 15, 32, -1)
    # half a step, the scale's rounding over 8 steps and the centre's at the group's largest, fp32 on top
    bound = (0.5 + 8 * 2.0 ** -8) * step + (2.0 ** -8 + 2.0 ** -18) * np.repeat(np.abs(grp).max(-1), 32, -1)
    assert (np.abs(ko.double().cpu().numpy() - K) <= bound).all()
    used = {int(table[b, i]) for b in range(B) for i in range(-(-reach[b] // page))}
    spare = [i for i in range(cache.shape[1]) if i not in used]
    assert (cache[:, spare] == 255).all()


def test_work_queued_without_waiting():
    """Kernels that make the inputs, the operators, and kernels that use the outputs, queued one
    behind the other: nothing starts before what it reads is there."""
    H, G, d, rd, base, page, B, steps = 8, 2, 128, 64, 1e6, 16, 3, 20
    g = torch.Generator().manual_seed(51)
    start = [100, 1, 47]
    k, v = (torch.randn(steps, B, G, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    qg = torch.randn(steps, B, H, 2 * d, generator=g).to(torch.bfloat16).to(DEV)
    kw, qw = (torch.ones(d, dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def run(wait):
        x = decode_inputs(H, G, d, rd, base, page, [n + steps for n in start], seed=52)
        lens, pages, got = i32(start), x["table"] - 1, []
        for s in range(steps):
            lens = lens + 1
            table = pages + 1
            if s % 3 == 2:  # written and then attended, in two calls
                gattn_qcache_write(k[s] * 0.5, v[s] * 2, x["cache"], table, lens, kw, rotary_dim=rd, rope_base=base)
                new = {}
            else:
                new = dict(k_new=k[s] * 0.5, v_new=v[s] * 2, knorm_w=kw)
            if wait:
                torch.cuda.synchronize()
            o = gattn_decode_qcache(qg[s, ..., :d] * 1, x["cache"], table, lens, qg[s, ..., d:] * 1, qw, rotary_dim=rd,
                                    rope_base=base, **new)
            if wait:
                torch.cuda.synchronize()
            ko, vo = gattn_qcache_read(x["cache"], table, lens - 1)
            if wait:
                torch.cuda.synchronize()
            got += [o + 0, ko + 0, vo + 0]
        torch.cuda.synchronize()
        assert gattn_get_device_status() == 0
        return got + [x["cache"]]

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)


def test_two_graphs_and_an_eager_call_between():
    """Two captured steps, each with its own workspace, replayed in turn with an eager one between."""
    cases = [(8, 2, 256, 64, 1e7, 64, [3000, 40]), (16, 8, 128, 128, 1e6, 16, [900, 901, 17])]
    xs = [decode_inputs(*c, seed=i + 60) for i, c in enumerate(cases)]
    on_gpu = [(x["qg"].to(DEV), x["qw"].to(DEV)) for x in xs]

    def call(i, **kw):
        c, x, (qg, qw) = cases[i], xs[i], on_gpu[i]
        return gattn_decode_qcache(qg[..., :c[2]], x["cache"], x["table"], x["seqlens"], qg[..., c[2]:], qw,
                                   rotary_dim=c[3], rope_base=c[4], **kw)

    plain = [call(0), call(1)]
    graphs, outs = [], []
    for i, c in enumerate(cases):
        need = gattn_decode_qcache_workspace_size(len(c[-1]), c[0], c[1], c[2], xs[i]["table"].shape[1] * c[5])
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs.append(call(i, workspace=ws))
    for _ in range(3):
        outs[0].zero_(), outs[1].zero_()
        graphs[0].replay()
        between = call(1)
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], plain[0]) and torch.equal(outs[1], plain[1]) and torch.equal(between, plain[1])


def test_another_stream_allocates_and_two_threads():
    """Writes and reads on a stream of the caller's, their outputs made there; then two threads at once."""
    import threading

    d, G, page, T = 128, 2, 32, 500
    cache, table = make_pool([T], G, page, d, 70)
    kv = torch.randn(2, T, G, d, generator=torch.Generator().manual_seed(71)).to(torch.bfloat16).to(DEV)
    w, lens, cu = torch.ones(d, dtype=torch.bfloat16, device=DEV), i32([T]), i32([0, T])
    torch.cuda.synchronize()

    def once(stream, out):
        for _ in range(20):
            mine = torch.empty_like(cache)
            gattn_qcache_write(kv[0], kv[1], mine, table, lens, w, cu, rotary_dim=64, rope_base=1e6, stream=stream)
            out.append(gattn_qcache_read(mine, table, None, cu, total=T, stream=stream))
            stream.synchronize()

    results = [[], []]
    streams = [torch.cuda.Stream() for _ in results]
    once(streams[0], results[0])
    threads = [threading.Thread(target=once, args=a) for a in zip(streams, results)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0 and [len(r) for r in results] == [40, 20]
    for k, v in results[0] + results[1]:
        assert torch.equal(k, results[0][0][0]) and torch.equal(v, results[0][0][1])


def test_captured_behind_copies_fills_and_joins():
    """Operators whose captured predecessor is no kernel (a copy, a fill) or two (a join)."""
    H, G, d, rd, base, page, lens = 8, 2, 128, 64, 1e6, 32, [70, 33]
    x = decode_inputs(H, G, d, rd, base, page, lens, seed=81)
    g = torch.Generator().manual_seed(82)
    k, v = (torch.randn(2, G, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    qg, qw, kw = x["qg"].to(DEV), x["qw"].to(DEV), x["kw"].to(DEV)
    want_cache = x["cache"].clone()
    gattn_qcache_write(k, v, want_cache, x["table"], x["seqlens"], kw, rotary_dim=rd, rope_base=base)
    want = gattn_decode_qcache(qg[..., :d], want_cache, x["table"], x["seqlens"], qg[..., d:], qw, rotary_dim=rd, rope_base=base)
    want_rows = gattn_qcache_read(want_cache, x["table"], x["seqlens"] - 1)
    torch.cuda.synchronize()
    kc, vc, lens_c, cache = torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(x["seqlens"]), torch.zeros_like(x["cache"])
    starts, junk = x["seqlens"] - 1, torch.empty(1 << 20, device=DEV)
    ws = torch.empty(gattn_decode_qcache_workspace_size(2, H, G, d, x["table"].shape[1] * page), dtype=torch.uint8, device=DEV)
    other = torch.cuda.Stream()

    def ahead(how):
        if how == "copy":
            lens_c.copy_(x["seqlens"])
        elif how == "fill":
            junk.zero_()
        else:
            other.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(other):
                junk.mul_(0)
            torch.cuda.current_stream().wait_stream(other)

    def run(how, append):
        cache.copy_(x["cache"])
        kc.copy_(k), vc.copy_(v)
        new = dict(k_new=kc, v_new=vc, knorm_w=kw) if append else {}
        if not append:
            lens_c.copy_(x["seqlens"])
            ahead(how)
            gattn_qcache_write(kc, vc, cache, x["table"], lens_c, kw, rotary_dim=rd, rope_base=base)
        lens_c.copy_(x["seqlens"])
        ahead(how)
        out = gattn_decode_qcache(qg[..., :d], cache, x["table"], lens_c, qg[..., d:], qw, rotary_dim=rd, rope_base=base,
                                  workspace=ws, **new)
        ahead(how)
        return (out, *gattn_qcache_read(cache, x["table"], starts))

    for how in ("copy", "fill", "join"):
        for append in (False, True):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = run(how, append)
            for _ in range(2):
                lens_c.zero_(), cache.zero_(), kc.zero_()
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(got[0], want), (how, append)
                assert all(torch.equal(a, b) for a, b in zip(got[1:], want_rows)), (how, append)
                assert torch.equal(cache, want_cache)
    assert gattn_get_device_status() == 0


def test_read_returns_ordinary_tensors():
    """The two results of a read: contiguous, apart from each other, kept, cloned and changed on their own."""
    d, G, T = 64, 3, 37
    cache, table = make_pool([T], G, 16, d, 90)
    kv = torch.randn(2, T, G, d, generator=torch.Generator().manual_seed(91)).to(torch.bfloat16).to(DEV)
    cu = i32([0, T])
    gattn_qcache_write(kv[0], kv[1], cache, table, i32([T]), torch.ones(d, dtype=torch.bfloat16, device=DEV), cu,
                       rotary_dim=32, rope_base=1e4)
    for dt in (torch.bfloat16, torch.float32):
        k, v = gattn_qcache_read(cache, table, None, cu, total=T, dtype=dt)
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        gattn_qcache_read(cache, table, None, cu, k_out=ko, v_out=vo)
        assert k.shape == v.shape == (T, G, d) and k.dtype == v.dtype == dt and k.is_contiguous() and v.is_contiguous()
        assert torch.equal(k, ko) and torch.equal(v, vo)
        k.zero_()
        assert torch.equal(v, vo) and torch.equal(v.transpose(0, 1).clone(), vo.transpose(0, 1))
        del k
        v += 1
        assert torch.equal(v, vo + 1)
        with torch.inference_mode():
            assert torch.equal(gattn_qcache_read(cache, table, None, cu, total=T, dtype=dt)[1], vo)
    none = gattn_qcache_read(cache, table, None, i32([0, 0]), total=0)
    assert none[0].shape == none[1].shape == (0, G, d)
