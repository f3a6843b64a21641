"""The 4-bit KV cache's size queries: a geometry that the calls refuse has no size."""
import ctypes

import pytest

import __graft_entry__
import gated_softmax_attention_gqa_gb300 as ga
from gated_softmax_attention_gqa_gb300 import _lib


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build_library()
    return _lib.load()


@pytest.mark.parametrize("d", [0, -64, 1, 32, 63, 65, 96, 192, 320, 512, 1024])
def test_no_cache_of_other_head_dims(lib, d):
    assert lib.gattn_qcache_bytes(7, 3, 48, d) == 0
    with pytest.raises(ValueError):
        ga.gattn_qcache_shape(7, 3, 48, d)


@pytest.mark.parametrize("bad", [(-1, 3, 48), (7, 0, 48), (7, -2, 48), (7, 3, 0), (7, 3, -16), (7, 3, 8), (7, 3, 47)])
def test_no_cache_of_other_pages(lib, bad):
    assert all(lib.gattn_qcache_bytes(*bad, d) == 0 for d in (64, 128, 256))


def test_bytes_are_the_shape_s_and_pass_32_bits(lib):
    for d in (64, 128, 256):
        for args in ((1, 1, 16, d), (7, 3, 48, d), (1 << 20, 8, 64, d)):
            n = 1
            for x in ga.gattn_qcache_shape(args[0], args[1], args[2], d):
                n *= x
            assert lib.gattn_qcache_bytes(*args) == n


# what gattn_decode_qcache refuses of B, H, G, d and Lmax, next to what it takes
REFUSED = [(0, 8, 2, 128, 64), (1, 0, 2, 128, 64), (1, 8, 0, 128, 64), (1, 8, 3, 128, 64), (1, 8, 2, 128, 0),
           (1, 8, 2, 96, 64), (1, 8, 2, 192, 64), (1, 8, 2, 32, 64), (1, 8, 2, 512, 64), (1, 9, 1, 128, 64),
           (1, 18, 2, 64, 64), (2049, 8, 2, 128, 64), (2048, 64, 64, 128, 1 << 20), (1, 8, 2, 128, (1 << 31) - 16)]
TAKEN = [(1, 8, 1, 64, 16), (2048, 8, 2, 128, 64), (2048, 64, 8, 256, 1 << 13), (1, 1, 1, 128, 1 << 30)]


@pytest.mark.parametrize("case", REFUSED, ids=str)
def test_no_workspace_for_what_is_refused(lib, case):
    """Without a GPU every answer is 0; the same on one is in the test below."""
    assert ga.gattn_decode_qcache_workspace_size(*case) == 0


@pytest.mark.gpu
def test_workspace_sizes_on_the_gpu(lib):
    fake = ctypes.c_void_p(0x7F0000000000)

    def status(B, H, G, d, Lmax):  # a workspace of no bytes: refused last, before anything runs
        return lib.gattn_decode_qcache(fake, None, None, fake, fake, 64, 16, Lmax // 16, fake, None, fake, None, B, H, G, d, 0,
                                       1e4, 1e-6, 0, 0, 0, 0, 0, fake, 0, fake, None)

    workspace = 4  # GATTN_ERR_WORKSPACE
    for case in REFUSED:
        assert ga.gattn_decode_qcache_workspace_size(*case) == 0 and status(*case) != workspace, case
    for case in TAKEN:
        assert ga.gattn_decode_qcache_workspace_size(*case) > 0 and status(*case) == workspace, case
