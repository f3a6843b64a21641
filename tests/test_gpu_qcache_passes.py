"""Long calls of the 4-bit KV cache: every number of passes that a warp of the write or of the
read may take, at every head_dim, over all rows of the call.

A write's warps take 1, 2, 4 or 8 passes by the call's length, its KV heads and what a warp can
look up; the lengths below are just past each step (3 (passes / 2)^2 waves of 8 warps an SM,
512 / d tokens to a pass), and not a multiple of what a warp takes.  V is quantised from its given bits, so all that
is read back is compared for equality.  K is compared with its exact value: half a step, the
scale's rounding (2^-8 at most) over eight steps, the centre's at the group's largest number,
and 2^-18 of that for fp32 arithmetic."""
import numpy as np
import pytest
import torch

from gated_softmax_attention_gqa_gb300 import gattn_get_device_status, gattn_qcache_read, gattn_qcache_write
from tests import qcache_ref as ref
from tests.test_gpu_qcache import DEV, i32, make_pool

pytestmark = pytest.mark.gpu


def rows_of(d, passes, beyond):
    """Tokens at which the write's warps come to `passes` passes, and some more."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return 512 // d * 3 * (passes // 2) ** 2 * 8 * sms + beyond


def batch(T, before_most, seed):
    """Six sequences of T tokens in all, one empty and one of a single token, and what each holds ahead of them."""
    rng = np.random.default_rng(seed)
    cuts = np.sort(rng.integers(1, T - 1, 3))
    n = [int(cuts[0]), 0, int(cuts[1] - cuts[0]), 1, int(cuts[2] - cuts[1]), int(T - 1 - cuts[2])]
    return n, [int(x) for x in rng.integers(0, before_most, len(n))]


def stored(x):
    """Values [T,G,d] (fp64) that the format holds for fp32 x, with its own roundings."""
    g = x.float().unflatten(-1, (-1, 32))
    hi, lo = g.amax(-1), g.amin(-1)
    step = (0.5 * hi - 0.5 * lo) * torch.tensor(2 / 15, dtype=torch.float32, device=x.device)
    s, c = step.bfloat16().float()[..., None], (lo + 8 * step).bfloat16().float()[..., None]
    n = torch.round((g - c).double() * (1 / s).double()).clamp(-8, 7)
    return (c.double() + s.double() * n).flatten(-2)


def exact_keys(k, w, pos, rd, base, eps=1e-6):
    """fp64 RMSNorm and rotate-half RoPE of k [T,G,d]."""
    x = k.double()
    x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    h = rd // 2
    f = torch.tensor(base, dtype=torch.float64, device=k.device) ** (-2.0 * torch.arange(h, device=k.device).double() / rd)
    a = (pos.double()[:, None] * f)[:, None]
    lo, hi = x[..., :h].clone(), x[..., h:rd].clone()
    x[..., :h], x[..., h:rd] = lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()
    return x


WRITES = [
    # d, G, passes by the length alone, rd, dtype
    (64, 1, 2, 64, torch.bfloat16), (64, 1, 4, 32, torch.float32), (64, 1, 4, 64, torch.bfloat16),
    (64, 1, 8, 64, torch.bfloat16), (64, 1, 8, 48, torch.float32),
    (64, 2, 4, 64, torch.bfloat16), (64, 3, 8, 32, torch.bfloat16),
    (128, 1, 2, 128, torch.float32), (128, 1, 4, 64, torch.bfloat16), (128, 1, 8, 128, torch.bfloat16),
    (128, 1, 8, 48, torch.float32), (128, 2, 4, 128, torch.bfloat16),
    (256, 1, 2, 256, torch.bfloat16), (256, 1, 4, 64, torch.float32), (256, 1, 8, 64, torch.bfloat16),
    (256, 1, 8, 192, torch.bfloat16), (256, 2, 4, 64, torch.float32),
]


@pytest.mark.parametrize("case", WRITES, ids=str)
def test_write_of_every_number_of_passes(case):
    d, G, passes, rd, dt = case
    page, pad, base = 48, 5, 1e6
    T = rows_of(d, passes, 37)
    new, before = batch(T, 100, d + passes)
    reach = [a + n for a, n in zip(before, new)]
    cache, table = make_pool(reach, G, page, d, passes)
    g = torch.Generator(DEV).manual_seed(d + G + passes)
    kv = torch.randn(T + pad, 2, G, d, generator=g, device=DEV).to(dt)
    w = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(dt)
    cu = i32(np.concatenate([[0], np.cumsum(new)]).tolist())
    gattn_qcache_write(kv[:, 0], kv[:, 1], cache, table, i32(reach), w, cu, rotary_dim=rd, rope_base=base)
    k, v = gattn_qcache_read(cache, table, i32(before), cu, total=T, dtype=torch.float32)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    assert torch.equal(v, stored(kv[:T, 1]).float())
    pos = torch.cat([torch.arange(a, b, device=DEV) for a, b in zip(before, reach)])
    want = exact_keys(kv[:T, 0], w, pos, rd, base)
    grp = want.unflatten(-1, (-1, 32))
    bound = (0.5 + 8 * 2.0 ** -8) * (grp.amax(-1) - grp.amin(-1)) / 15 + (2.0 ** -8 + 2.0 ** -18) * grp.abs().amax(-1)
    assert ((k.double() - want).unflatten(-1, (-1, 32)).abs() <= bound[..., None]).all()
    # rows ahead of the new ones (NaN scales) and spare pages are as they were
    ahead = i32(np.concatenate([[0], np.cumsum(before)]).tolist())
    k, v = gattn_qcache_read(cache, table, None, ahead, total=sum(before))
    assert k.isnan().all() and v.isnan().all()
    used = torch.zeros(cache.shape[1], dtype=torch.bool, device=DEV)
    used[table[table >= 0].long()] = True
    assert (cache[:, ~used] == 255).all()


def rounded_bf16(x):
    """fp64 rounded once to bf16's eight bits, half to even (normal numbers and zero)."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256), e - 8)


@pytest.mark.parametrize("G", [1, 2])
def test_long_read_of_two_passes(G):
    """Reads to bf16 whose warps take two passes (head_dim 256, from 8 waves of 8 warps an SM on)."""
    d, page = 256, 80
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = 2 * 64 * sms + 3
    n, starts = batch(T, 200, G)
    reach = [a + b for a, b in zip(starts, n)]
    cache, table = make_pool(reach, G, page, d, G)
    g = torch.Generator(DEV).manual_seed(G)
    # any codes; scales and centres of ordinary size and either sign
    cache[..., :8 * d] = torch.randint(0, 256, cache[..., :8 * d].shape, generator=g, device=DEV, dtype=torch.uint8)
    par = torch.randn(cache[..., 8 * d::2].shape, generator=g, device=DEV)
    cache[..., 8 * d:] = par.to(torch.bfloat16).view(torch.uint8)
    cu = i32(np.concatenate([[0], np.cumsum(n)]).tolist())
    k, v = (torch.full((T + 4, G, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    gattn_qcache_read(cache, table, i32(starts), cu, k_out=k, v_out=v)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    raw, tab = cache.cpu().numpy(), table.cpu().numpy()
    rows = [ref.values(raw, tab, b, starts[b], reach[b]) for b in range(len(n))]
    for got, plane in ((k, 0), (v, 1)):
        want = rounded_bf16(np.concatenate([r[plane] for r in rows]))
        assert (got[:T].double().cpu().numpy() == want).all()
        assert (got[T:] == 7).all()
