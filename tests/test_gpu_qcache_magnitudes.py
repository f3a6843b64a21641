"""Writing keys of far magnitudes into the 4-bit KV cache."""
import pytest
import torch

from gated_softmax_attention_gqa_gb300 import gattn_get_device_status, gattn_qcache_write
from tests import qcache_ref as ref
from tests.test_gpu_qcache import DEV, check_rows, i32, make_pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rd", [(64, 0), (128, 64), (256, 256)])
def test_keys_of_far_magnitudes(d, rd, dt):
    """Rows of 5e-39 to 1e15, neighbours in a warp.  eps = 1e-6 lifts a tiny row by 1000: its groups have
    steps from 1e-36 on, normal numbers whose reciprocals, times those 1000, pass fp32's range.  Numbers below
    2^-126 are off by up to 2^-150 for each of three roundings (two products and their sum), times 1000: 3e-42, within
    the 2^-20 of a row's largest number (64 normals of 5e-36: above 7e-36, so 7e-42) that the check allows."""
    G, page, base = 2, 32, 1e4
    scale = torch.tensor([1e-37, 1.0, 5e-39, 1e-36, 1e15, 1e-38, 2e-38, 1e-20, 5e-37])
    T = 4 * len(scale)
    g = torch.Generator().manual_seed(d)
    k = (torch.randn(T, G, d, generator=g) * scale.repeat(4)[:, None, None]).to(dt)
    v = torch.randn(T, G, d, generator=g).to(dt)
    kw = (1 + 0.1 * torch.randn(d, generator=g)).to(dt)
    cache, table = make_pool([T], G, page, d, d)
    gattn_qcache_write(k.to(DEV), v.to(DEV), cache, table, i32([T]), kw.to(DEV), i32([0, T]), rotary_dim=rd, rope_base=base)
    torch.cuda.synchronize()
    assert gattn_get_device_status() == 0
    K = ref.norm_rope(k.double().numpy(), kw.double().numpy(), range(T), rd, base)
    raw, tab = cache.cpu().numpy(), table.cpu().numpy()
    for gg in range(G):
        check_rows(raw, tab, 0, gg, 0, K[:, gg], 0)
        check_rows(raw, tab, 0, gg, 1, v[:, gg].double().numpy(), 0)
