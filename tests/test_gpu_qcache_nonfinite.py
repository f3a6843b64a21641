"""Decoding over a 4-bit KV cache that holds NaN: attention is a sum over all live keys, so a NaN
in a live token's K makes every feature of its KV head's outputs NaN and one in its V the features
of its group, wherever the token lies in the work split and however small its weight; all other
outputs are what they are without it."""
import pytest
import torch

from gated_softmax_attention_gqa_gb300 import gattn_get_device_status, gattn_qcache_write
from tests.test_gpu_qcache import DEV, assert_close, decode_inputs, expected, i32, make_pool, run_decode

pytestmark = pytest.mark.gpu


def spoil(x, plane, b, g, pos, group):
    """A NaN scale and centre for one group of features of a cached token, as a write of a NaN leaves them."""
    cache, d = x["cache"], x["cache"].shape[-1] // 10
    page = 16 * cache.shape[3]
    row = cache[plane, int(x["table"][b, pos // page]), g, pos % page // 16]
    nan = torch.tensor([0xC0, 0x7F], dtype=torch.uint8, device=DEV)
    for at in (8 * d, 9 * d):
        at += 32 * group + 2 * (pos % 16)
        row[at:at + 2] = nan


# Lengths whose last token is alone in its warp's blocks (a warp takes 32 keys of a tile, 48 at
# head_dim 128), shares them, or lies in one of many CTAs' parts; tokens at the start, end and between.
KEYS = [(64, 33, 32), (128, 49, 48), (256, 33, 32), (256, 32, 31), (64, 1, 0), (256, 65, 64), (128, 192, 60),
        (64, 6000, 5999), (128, 6000, 17), (256, 6000, 5999), (256, 6000, 2500), (128, 5761, 5760)]


@pytest.mark.parametrize("case", KEYS, ids=str)
def test_nan_in_a_key(case):
    d, L, pos = case
    H, G, rd, base, lens = 6, 2, 32, 1e4, [L, 40]
    x = decode_inputs(H, G, d, rd, base, 32, lens, seed=L + d)
    clean = run_decode(x, d, rd, base)
    assert_close(clean, expected(x, lens, rd, base), str(case))
    spoil(x, 0, 0, 1, pos, d // 32 - 1)
    out = run_decode(x, d, rd, base)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    out, clean = out.view(2, G, H // G, d), clean.view(2, G, H // G, d)
    assert out[0, 1].isnan().all()
    assert torch.equal(out[0, 0], clean[0, 0]) and torch.equal(out[1], clean[1])


@pytest.mark.parametrize("case", KEYS, ids=str)
def test_nan_in_a_value(case):
    d, L, pos = case
    H, G, rd, base, lens = 6, 2, 32, 1e4, [L, 40]
    x = decode_inputs(H, G, d, rd, base, 32, lens, seed=L + d)
    clean = run_decode(x, d, rd, base)
    spoil(x, 1, 0, 0, pos, 1)
    out = run_decode(x, d, rd, base)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    assert out.view(2, H, d)[0, :3, 32:64].isnan().all()
    keep = torch.ones(2, H, d, dtype=torch.bool, device=DEV)
    keep[0, :3, 32:64] = False
    assert torch.equal(out.view(2, H, d)[keep], clean.view(2, H, d)[keep])


@pytest.mark.parametrize("d,L", [(64, 64), (128, 96), (256, 64), (256, 3000), (128, 9000)])
def test_nan_value_of_a_weight_that_underflows(d, L):
    """One key along the query and all others against it, norm weights that put the logits some
    hundreds apart: the others' weights are below every fp32 number, and zero times NaN is NaN."""
    H, G, page = 1, 1, 48
    cache, table = make_pool([L], G, page, d, 5)
    g = torch.Generator().manual_seed(L)
    q = torch.randn(d, generator=g).to(torch.bfloat16)
    k = (-q).repeat(L, 1, 1)
    k[0, 0] = q
    v = torch.randn(L, G, d, generator=g).to(torch.bfloat16)
    x = dict(cache=cache, table=table, seqlens=i32([L]), qg=q.repeat(1, 1, 2), gate=None,
             qw=torch.full((d,), 30.0, dtype=torch.bfloat16))
    gattn_qcache_write(k.to(DEV), v.to(DEV), cache, table, x["seqlens"], torch.ones(d, dtype=torch.bfloat16, device=DEV),
                       i32([0, L]), rotary_dim=0, rope_base=1e4)
    clean = run_decode(x, d, 0, 1e4, "none")
    assert_close(clean, expected(x, [L], 0, 1e4, "none"), "finite")
    spoil(x, 1, 0, 0, L - 1, 1)
    out = run_decode(x, d, 0, 1e4, "none")
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    assert out[0, 32:64].isnan().all()
    assert torch.equal(out[0, :32], clean[0, :32]) and torch.equal(out[0, 64:], clean[0, 64:])


def test_nan_query_and_masked_nan():
    """A NaN query makes its head NaN alone; NaN rows behind the last token change nothing."""
    H, G, d, rd, base, lens = 4, 2, 128, 64, 1e6, [50, 300]
    x = decode_inputs(H, G, d, rd, base, 32, lens, seed=3)
    clean = run_decode(x, d, rd, base)
    for b, pos in ((0, 50), (0, 63), (1, 300), (1, 319)):
        for plane in (0, 1):
            for group in range(d // 32):
                spoil(x, plane, b, 1, pos, group)
    assert torch.equal(run_decode(x, d, rd, base), clean)
    x["qg"][1, 2, 5] = float("nan")
    out = run_decode(x, d, rd, base)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    assert out.view(2, H, d)[1, 2].isnan().all()
    keep = [h for h in range(H) if h != 2]
    assert torch.equal(out.view(2, H, d)[0], clean.view(2, H, d)[0])
    assert torch.equal(out.view(2, H, d)[1, keep], clean.view(2, H, d)[1, keep])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_nan_stays_in_its_piece(d):
    """Many short sequences, several (sequence, KV head) pieces to a CTA: a NaN key or value of one
    leaves those ahead of it and behind it alone."""
    H, G, rd, base, B = 4, 2, 32, 1e4, 900
    lens = [1 + 37 * b % 70 for b in range(B)]
    x = decode_inputs(H, G, d, rd, base, 16, lens, seed=d)
    clean = run_decode(x, d, rd, base).view(B, H, d)
    x["table"] = x["table"].cpu()
    want = torch.zeros(B, H, d, dtype=torch.bool)
    for b in range(0, B, 7):
        spoil(x, 0, b, b & 1, lens[b] - 1, 0)
        want[b, 2 * (b & 1):2 * (b & 1) + 2] = True
    for b in range(3, B, 7):
        spoil(x, 1, b, b & 1, lens[b] // 2, 1)
        want[b, 2 * (b & 1):2 * (b & 1) + 2, 32:64] = True
    x["table"] = x["table"].to(DEV)
    out = run_decode(x, d, rd, base).view(B, H, d)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    want = want.to(DEV)
    assert torch.equal(out.isnan(), want)
    assert torch.equal(out[~want], clean[~want])
