"""Refusals of the 4-bit KV cache's entry points: the C argument checks (fake pointers that
are never dereferenced) and the Python wrappers' layout checks, both without a GPU."""
import ctypes

import pytest
import torch

import __graft_entry__
import gated_softmax_attention_gqa_gb300 as ga
from gated_softmax_attention_gqa_gb300 import _lib

OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = range(5)
FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build_library()
    return _lib.load()


def P(off=0):
    return ctypes.c_void_p(FAKE + off)


def write(lib, **kw):
    a = dict(k=P(), v=P(), qc=P(), bt=P(), np_=64, ps=64, mp=16, sl=P(), cu=P(), kw=P(), T=100, B=4, G=2, d=128, rd=64,
             base=1e6, eps=1e-6, s=(0, 0, 0, 0), dt=0)
    a.update(kw)
    return lib.gattn_qcache_write(a["k"], a["v"], a["qc"], a["bt"], a["np_"], a["ps"], a["mp"], a["sl"], a["cu"], a["kw"],
                                  a["T"], a["B"], a["G"], a["d"], a["rd"], a["base"], a["eps"], *a["s"], a["dt"], None)


COMMON = [
    (dict(qc=None), INVALID), (dict(bt=None), INVALID), (dict(np_=0), INVALID), (dict(mp=0), INVALID),
    (dict(ps=0), INVALID), (dict(ps=24), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(d=32), UNSUPPORTED),
    (dict(G=0), INVALID), (dict(B=0), INVALID), (dict(qc=P(8)), INVALID), (dict(bt=P(2)), INVALID),
    (dict(mp=1 << 26, ps=64), INVALID),  # positions past 31 bits
]


@pytest.mark.parametrize("kw,expect", COMMON + [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(sl=None), INVALID), (dict(kw=None), INVALID),
    (dict(T=-1), INVALID), (dict(cu=None), INVALID),            # one token each: T must be B
    (dict(dt=2), INVALID), (dict(rd=7), INVALID), (dict(rd=130), INVALID), (dict(rd=24), UNSUPPORTED),
    (dict(base=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(k=P(8)), INVALID), (dict(s=(1028, 0, 0, 0)), INVALID), (dict(s=(0, 0, 0, 130)), INVALID),
    (dict(s=(-256, 0, 0, 0)), INVALID), (dict(T=1 << 30, G=2), INVALID),
    (dict(T=0), OK),                                             # nothing to write
], ids=str)
def test_write_rejects_bad_arguments(lib, kw, expect):
    assert write(lib, **kw) == expect


def read(lib, **kw):
    a = dict(qc=P(), bt=P(), np_=64, ps=64, mp=16, st=P(), cu=P(), T=100, B=4, G=2, d=128, dt=0, k=P(), v=P())
    a.update(kw)
    return lib.gattn_qcache_read(a["qc"], a["bt"], a["np_"], a["ps"], a["mp"], a["st"], a["cu"], a["T"], a["B"], a["G"],
                                 a["d"], a["dt"], a["k"], a["v"], None)


@pytest.mark.parametrize("kw,expect", COMMON + [
    (dict(k=None), INVALID), (dict(v=P(4)), INVALID), (dict(T=-1), INVALID), (dict(cu=None), INVALID),
    (dict(dt=5), INVALID), (dict(T=0), OK), (dict(T=1 << 30, G=4), INVALID), (dict(st=P(1)), INVALID),
], ids=str)
def test_read_rejects_bad_arguments(lib, kw, expect):
    assert read(lib, **kw) == expect


def decode(lib, **kw):
    a = dict(q=P(), kn=None, vn=None, qc=P(), bt=P(), np_=64, ps=64, mp=16, sl=P(), gate=P(), qw=P(), kw=None, B=4, H=8,
             G=2, d=256, rd=64, base=1e7, eps=1e-6, gm=1, s=(0, 0, 0, 0), ws=P(), wsb=1 << 40, out=P(1 << 20))
    a.update(kw)
    return lib.gattn_decode_qcache(a["q"], a["kn"], a["vn"], a["qc"], a["bt"], a["np_"], a["ps"], a["mp"], a["sl"],
                                   a["gate"], a["qw"], a["kw"], a["B"], a["H"], a["G"], a["d"], a["rd"], a["base"],
                                   a["eps"], a["gm"], *a["s"], a["ws"], a["wsb"], a["out"], None)


@pytest.mark.parametrize("kw,expect", COMMON + [
    (dict(q=None), INVALID), (dict(sl=None), INVALID), (dict(qw=None), INVALID), (dict(out=None), INVALID),
    (dict(gate=None), INVALID), (dict(gm=0x40), INVALID), (dict(gm=0x100), INVALID), (dict(H=9), INVALID),
    (dict(H=18), UNSUPPORTED), (dict(B=2049), UNSUPPORTED), (dict(rd=40), UNSUPPORTED), (dict(q=P(4)), INVALID),
    (dict(s=(2052, 0, 0, 0)), INVALID), (dict(s=(0, 0, -1, 0)), INVALID), (dict(out=P(8)), INVALID),
    (dict(kn=P()), INVALID), (dict(vn=P()), INVALID), (dict(kn=P(), vn=P()), INVALID),
    (dict(kn=P(), vn=P(4), kw=P()), INVALID),
], ids=str)
def test_decode_rejects_bad_arguments(lib, kw, expect):
    assert decode(lib, **kw) == expect


def test_sizes(lib):
    assert lib.gattn_qcache_bytes(7, 3, 48, 128) == 2 * 7 * 3 * 3 * 1280
    assert lib.gattn_qcache_bytes(7, 3, 40, 128) == 0 and lib.gattn_qcache_bytes(0, 3, 48, 128) == 0
    assert ga.gattn_qcache_shape(7, 3, 48, 128) == (2, 7, 3, 3, 1280)
    for bad in ((7, 3, 40, 128), (7, 3, 0, 128), (7, 3, 48, 96)):
        with pytest.raises(ValueError):
            ga.gattn_qcache_shape(*bad)
    assert lib.gattn_decode_qcache_workspace_size(0, 8, 2, 128, 64) == 0
    assert lib.gattn_decode_qcache_workspace_size(1, 8, 3, 128, 64) == 0


def args(T=6, B=3, G=2, d=64, dt=torch.bfloat16):
    return dict(k=torch.zeros(T, G, d, dtype=dt), v=torch.zeros(T, G, d, dtype=dt),
                qcache=torch.zeros(ga.gattn_qcache_shape(4, G, 32, d), dtype=torch.uint8),
                block_table=torch.zeros(B, 2, dtype=torch.int32), seqlens=torch.ones(B, dtype=torch.int32),
                knorm_w=torch.ones(d, dtype=dt), cu_seqlens=torch.tensor([0, 2, 4, 6], dtype=torch.int32))


@pytest.mark.parametrize("change", [
    dict(v=torch.zeros(6, 2, 64)), dict(knorm_w=torch.ones(64)), dict(k=torch.zeros(6, 2, 128, dtype=torch.bfloat16)),
    dict(k=torch.zeros(6, 64, 2, dtype=torch.bfloat16).transpose(1, 2)), dict(cu_seqlens=None),
    dict(cu_seqlens=torch.zeros(4, dtype=torch.int64)), dict(cu_seqlens=torch.zeros(3, dtype=torch.int32)),
    dict(seqlens=torch.ones(3, dtype=torch.int64)), dict(block_table=torch.zeros(2, 2, dtype=torch.int32)),
    dict(block_table=torch.zeros(3, 2, dtype=torch.int64)), dict(qcache=torch.zeros(2, 4, 2, 2, 640, dtype=torch.int8)),
    dict(qcache=torch.zeros(2, 4, 2, 2, 641, dtype=torch.uint8)), dict(qcache=torch.zeros(4, 2, 2, 640, dtype=torch.uint8)),
    dict(k=torch.zeros(1, 2, 64, dtype=torch.bfloat16).expand(6, 2, 64)),
    dict(k=torch.zeros(6, 2, 64, dtype=torch.float16), v=torch.zeros(6, 2, 64, dtype=torch.float16)),
], ids=lambda c: ",".join(f"{k}:{tuple(v.shape) if v is not None else None}" for k, v in c.items()))
def test_write_wrapper_refuses(change):
    a = args()
    a.update(change)
    with pytest.raises(ValueError):
        ga.gattn_qcache_write(**a, rotary_dim=32, rope_base=1e4)


@pytest.mark.parametrize("kw", [
    dict(cu_seqlens=torch.tensor([0, 2, 4, 6], dtype=torch.int32)),          # how many rows?
    dict(total=5), dict(dtype=torch.float16), dict(k_out=torch.zeros(3, 2, 64, dtype=torch.bfloat16)),
    dict(k_out=torch.zeros(3, 2, 64), v_out=torch.zeros(3, 2, 64, dtype=torch.bfloat16)),
    dict(k_out=torch.zeros(4, 2, 64), v_out=torch.zeros(4, 2, 64)),
    dict(starts=torch.zeros(4, dtype=torch.int32)),
], ids=lambda c: ",".join(c))
def test_read_wrapper_refuses(kw):
    a = args()
    with pytest.raises(ValueError):
        ga.gattn_qcache_read(a["qcache"], a["block_table"], **kw)


@pytest.mark.parametrize("change", [
    dict(q_new=torch.zeros(3, 4, 64)), dict(q_new=torch.zeros(3, 4, 128, dtype=torch.bfloat16)),
    dict(gate=None), dict(gate=torch.zeros(3, 4, dtype=torch.bfloat16)), dict(qnorm_w=torch.ones(64)),
    dict(k_new=torch.zeros(3, 2, 64, dtype=torch.bfloat16)), dict(out=torch.zeros(3, 4, 64, dtype=torch.bfloat16)),
    dict(gate=torch.zeros(3, 1, 64, dtype=torch.bfloat16).expand(3, 4, 64)),
    dict(q_new=torch.zeros(3, 1, 64, dtype=torch.bfloat16).expand(3, 4, 64)),
], ids=lambda c: ",".join(f"{k}:{tuple(v.shape) if v is not None else None}" for k, v in c.items()))
def test_decode_wrapper_refuses(change):
    c = args()
    a = dict(q_new=torch.zeros(3, 4, 64, dtype=torch.bfloat16), qcache=c["qcache"], block_table=c["block_table"],
             seqlens=c["seqlens"], gate=torch.zeros(3, 4, 64, dtype=torch.bfloat16),
             qnorm_w=torch.ones(64, dtype=torch.bfloat16), workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    a.update(change)
    with pytest.raises(ValueError):
        ga.gattn_decode_qcache(**a, rotary_dim=32, rope_base=1e4)


class AnyStream:
    cuda_stream = 0


def calls():
    """Each wrapper with arguments that only lack a GPU."""
    c = args()
    one = {**args(T=3), "cu_seqlens": None}
    yield lambda **kw: ga.gattn_qcache_write(**{**c, "rotary_dim": 32, "rope_base": 1e4, **kw})
    yield lambda **kw: ga.gattn_qcache_write(**{**one, "rotary_dim": 32, "rope_base": 1e4, **kw})
    yield lambda **kw: ga.gattn_qcache_read(**{**dict(qcache=c["qcache"], block_table=c["block_table"]), **kw})
    yield lambda **kw: ga.gattn_decode_qcache(**{**dict(
        q_new=torch.zeros(3, 4, 64, dtype=torch.bfloat16), qcache=c["qcache"], block_table=c["block_table"],
        seqlens=c["seqlens"], gate=torch.zeros(3, 4, 64, dtype=torch.bfloat16),
        qnorm_w=torch.ones(64, dtype=torch.bfloat16), rotary_dim=32, rope_base=1e4), **kw})


def test_wrappers_refuse_host_tensors_and_things_that_are_none():
    for call in calls():
        with pytest.raises(ValueError, match="CUDA device"):
            call()
        with pytest.raises(ValueError, match="CUDA device"):
            call(stream=AnyStream())
        for bad in (None, 3, [1, 2]):
            with pytest.raises(ValueError, match="must be a tensor"):
                call(block_table=bad)


def test_wrappers_refuse_options_of_other_types_and_sizes():
    write_packed, write_one, read, decode = calls()
    for call in (write_packed, write_one, decode):
        with pytest.raises(ValueError):
            call(rotary_dim=1 << 40)
        with pytest.raises((TypeError, OverflowError)):
            call(rotary_dim=1 << 90)
        with pytest.raises(TypeError):
            call(rotary_dim="32")
        with pytest.raises(TypeError):
            call(rope_base="1e4")
    with pytest.raises(ValueError):
        read(cu_seqlens=torch.zeros(4, dtype=torch.int32), stream=AnyStream())  # how many rows?
    with pytest.raises(ValueError):
        read(cu_seqlens=torch.zeros(4, dtype=torch.int32), total=1 << 40)
    with pytest.raises(ValueError):
        read(cu_seqlens=torch.zeros(4, dtype=torch.int32), total=-1)
    with pytest.raises(ValueError):
        decode(workspace=torch.zeros(64, 2, dtype=torch.uint8)[:, 0])
