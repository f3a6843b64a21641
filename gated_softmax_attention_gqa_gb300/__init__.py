"""GB300-native gated softmax attention with GQA (libgattn).

The Python names mirror the C ABI in include/gattn.h.  Each call hands raw
device pointers, sizes and the current CUDA stream to libgattn.so; every step of
the computation runs in the library's CUDA kernels.  PyTorch only supplies
device memory and streams.  If the library is not built, calls raise: there is
no CPU fallback.

    out = gattn_prefill(q, k, v, gate, qnorm_w, knorm_w, rotary_dim=64, rope_base=1e7)
    out = gattn_decode(q_new, kv_cache, seqlens, gate, qnorm_w, rotary_dim=64, rope_base=1e7)
"""
import ctypes

import torch

from . import _lib
from ._lib import GattnError, check

# gate_mode = layout | activation | additive (the bit fields of gattn_gate_mode in gattn.h)
GATE_MODES = {"none": 0, "elementwise": 1, "headwise": 2, "head_shared": 3}
GATE_ACTS = {"sigmoid": 0x00, "ns_sigmoid": 0x10, "silu": 0x20}
GATE_ADDITIVE = 0x100
DTYPES = {torch.bfloat16: 0, torch.float32: 1}

__all__ = ["gattn_prefill", "gattn_prefill_varlen", "gattn_decode", "gattn_decode_append", "gattn_decode_paged", "gattn_decode_noalloc", "gattn_prefill_workspace_size", "gattn_prefill_varlen_workspace_size", "gattn_decode_workspace_size",
           "gattn_get_device_status", "gattn_set_profile_events", "gattn_selftest_wait_timeout", "gattn_o_proj", "gattn_strerror", "GattnError", "GATE_MODES",
           "GATE_ACTS", "GATE_ADDITIVE", "gattn_qcache_shape", "gattn_qcache_write", "gattn_qcache_read",
           "gattn_decode_qcache", "gattn_decode_qcache_workspace_size"]


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream, device):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _mode(gate_mode, gate_act="sigmoid", gate_additive=False):
    """The C gate_mode for a layout name, an activation name and the additive flag
    (an int is passed through unchanged)."""
    if not isinstance(gate_mode, str):
        return int(gate_mode)
    m = GATE_MODES[gate_mode]
    if m == 0:
        if gate_act != "sigmoid" or gate_additive:
            raise ValueError("gate_act / gate_additive need a gate")
        return 0
    return m | GATE_ACTS[gate_act] | (GATE_ADDITIVE if gate_additive else 0)


def gattn_strerror(status: int) -> str:
    return _lib.strerror(status)


def gattn_prefill_workspace_size(B, S, H, G, d, dtype=torch.bfloat16) -> int:
    return _lib.load().gattn_prefill_workspace_size(B, S, H, G, d, DTYPES[dtype])


def gattn_prefill_varlen_workspace_size(T, nseq, H, G, d, dtype=torch.bfloat16) -> int:
    return _lib.load().gattn_prefill_varlen_workspace_size(T, nseq, H, G, d, DTYPES[dtype])


def gattn_decode_workspace_size(B, H, G, d, Lmax) -> int:
    return _lib.load().gattn_decode_workspace_size(B, H, G, d, Lmax)


def gattn_set_profile_events(start=None, stop=None):
    """Record `start`/`stop` (torch.cuda.Event) around the main attention kernel of
    every later call; None, None switches it off."""
    for e in (start, stop):
        if e is not None and e.cuda_event == 0:
            e.record()  # torch creates the underlying cudaEvent lazily, on first record
    _lib.load().gattn_set_profile_events(ctypes.c_void_p(start.cuda_event) if start is not None else None,
                                         ctypes.c_void_p(stop.cuda_event) if stop is not None else None)


def gattn_get_device_status(stream=None) -> int:
    """Read and clear the device status bits (GATTN_DEVICE_* in gattn.h)."""
    bits = ctypes.c_uint(0)
    st = _lib.load().gattn_get_device_status(ctypes.byref(bits), _stream_handle(stream, None))
    if st not in (0, 5, 6):
        check(st, "gattn_get_device_status")
    return bits.value


def gattn_selftest_wait_timeout(limit_ns, waited_ns=None, stream=None):
    """Launch the bounded-wait self-test: a wait on an mbarrier nothing arrives on,
    given up after limit_ns (1e6 .. 1e8).  waited_ns: optional int64 CUDA tensor of
    one element that receives the wait's duration.  The timeout is read back with
    gattn_get_device_status()."""
    st = _lib.load().gattn_selftest_wait_timeout(int(limit_ns), _ptr(waited_ns), _stream_handle(stream, None))
    check(st, "gattn_selftest_wait_timeout")


def gattn_o_proj(x, w_o, out=None, stream=None):
    """Output projection of the attention output: out = x w_o^T.

    x [..., K] bf16 CUDA (the [B,S,H*d] or [T,H*d] output of gattn_prefill /
    gattn_prefill_varlen), contiguous; w_o [N, K] bf16 CUDA, contiguous (a linear
    layer's weight); out [..., N] bf16 (allocated if None).  K and N multiples of 64."""
    if x.dtype != torch.bfloat16 or w_o.dtype != torch.bfloat16:
        raise ValueError("x and w_o must be bfloat16")
    if not x.is_contiguous() or not w_o.is_contiguous() or w_o.dim() != 2:
        raise ValueError("x and w_o must be contiguous; w_o is [N, K]")
    K = x.shape[-1]
    N = w_o.shape[0]
    if w_o.shape[1] != K:
        raise ValueError(f"w_o is [{N}, {w_o.shape[1]}], x has K = {K}")
    T = x.numel() // K if K else 0
    if out is None:
        out = torch.empty(*x.shape[:-1], N, dtype=torch.bfloat16, device=x.device)
    elif out.dtype != torch.bfloat16 or not out.is_contiguous() or out.numel() != T * N:
        raise ValueError("out must be a contiguous bf16 tensor of T x N elements")
    st = _lib.load().gattn_o_proj(_ptr(x), _ptr(w_o), T, K, N, _ptr(out), _stream_handle(stream, x.device))
    check(st, "gattn_o_proj")
    return out


def _head_strides(t, name):
    """(token stride, head stride) in elements of a [B,S,H,*] or [B,S,H] view whose
    element (b,t,h,...) sits at (b*S + t)*token_stride + h*head_stride + ...."""
    if t.dim() not in (3, 4):
        raise ValueError(f"{name}: expected 3 or 4 dimensions")
    if t.dim() == 4 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    B, S = t.shape[0], t.shape[1]
    tok = t.stride(1) if S > 1 else t.stride(0)
    if B > 1 and S > 1 and t.stride(0) != S * t.stride(1):
        raise ValueError(f"{name}: batches must be evenly spaced tokens (stride(0) == S * stride(1))")
    return tok, t.stride(2)


def gattn_prefill(q, k, v, gate, qnorm_w, knorm_w, pos=None, *, rotary_dim, rope_base, eps=1e-6,
                  gate_mode="elementwise", gate_act="sigmoid", gate_additive=False, out=None, workspace=None,
                  stream=None):
    """Causal gated GQA attention over whole sequences.

    q [B,S,H,d] (may be a strided view, e.g. the query half of the packed q_proj
    output [B,S,H,2d]); k, v [B,S,G,d] contiguous; gate [B,S,H,d] (elementwise),
    [B,S,H] (headwise), [B,S,d] (head_shared: one vector for every head) or None;
    gate_act "sigmoid" | "ns_sigmoid" | "silu"; gate_additive: out = o + act(z)
    instead of o * act(z); qnorm_w, knorm_w [d]; pos [B,S] int32 or None.
    All on one CUDA device, bf16 or fp32 (all the same).  Returns out [B,S,H*d]."""
    mode = _mode(gate_mode, gate_act, gate_additive)
    B, S, H, d = q.shape
    G = k.shape[2]
    dt = DTYPES[q.dtype]
    qts, qhs = _head_strides(q, "q")
    if (mode & 0x0F) == GATE_MODES["head_shared"]:
        if gate.dim() != 3 or gate.stride(-1) != 1:
            raise ValueError("gate: a head-shared gate is [B,S,d] with a contiguous last dimension")
        if B > 1 and S > 1 and gate.stride(0) != S * gate.stride(1):
            raise ValueError("gate: batches must be evenly spaced tokens (stride(0) == S * stride(1))")
        gts, ghs = (gate.stride(1) if S > 1 else gate.stride(0)), 0
    elif mode & 0x0F:
        gts, ghs = _head_strides(gate, "gate")
    else:
        gate, gts, ghs = None, 0, 0
    if not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("k and v must be contiguous [B,S,G,d]")
    if pos is not None and (pos.dtype != torch.int32 or not pos.is_contiguous()):
        raise ValueError("pos must be a contiguous int32 [B,S] tensor")
    if out is None:
        out = torch.empty((B, S, H * d), dtype=q.dtype, device=q.device)
    need = gattn_prefill_workspace_size(B, S, H, G, d, q.dtype)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    st = _lib.load().gattn_prefill(
        _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(qnorm_w), _ptr(knorm_w), _ptr(pos), B, S, H, G, d,
        int(rotary_dim), float(rope_base), float(eps), mode, qts, qhs, gts, ghs, dt, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _stream_handle(stream, q.device))
    check(st, "gattn_prefill")
    return out


def gattn_prefill_varlen(q, k, v, gate, qnorm_w, knorm_w, cu_seqlens, pos=None, *, rotary_dim, rope_base,
                         eps=1e-6, gate_mode="elementwise", gate_act="sigmoid", gate_additive=False, out=None,
                         workspace=None, stream=None):
    """Causal gated GQA attention over packed variable-length sequences: sequence i
    is tokens [cu_seqlens[i], cu_seqlens[i+1]) of q [T,H,d] (last dimension
    contiguous), k, v [T,G,d] contiguous and gate [T,H,d] / [T,H] / [T,d]; it sees
    only its own keys and its positions restart at 0 unless pos [T] int32 is given.
    cu_seqlens: host int32 sequence (list, numpy array or CPU tensor).  Returns
    out [T,H*d]."""
    mode = _mode(gate_mode, gate_act, gate_additive)
    T, H, d = q.shape
    G = k.shape[1]
    cu = torch.as_tensor(cu_seqlens, dtype=torch.int32, device="cpu").contiguous()
    nseq = cu.numel() - 1
    if nseq < 1 or int(cu[-1]) != T:
        raise ValueError("cu_seqlens must have nseq+1 entries ending at T")
    if q.stride(-1) != 1:
        raise ValueError("q: the last dimension must be contiguous")
    if not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("k and v must be contiguous [T,G,d]")
    layout = mode & 0x0F
    if layout == 0:
        gate, gts, ghs = None, 0, 0
    elif layout == GATE_MODES["head_shared"]:
        gts, ghs = gate.stride(0), 0
    else:
        gts, ghs = gate.stride(0), gate.stride(1)
    if pos is not None and (pos.dtype != torch.int32 or not pos.is_contiguous()):
        raise ValueError("pos must be a contiguous int32 [T] tensor")
    if out is None:
        out = torch.empty((T, H * d), dtype=q.dtype, device=q.device)
    dt = DTYPES[q.dtype]
    need = _lib.load().gattn_prefill_varlen_workspace_size(T, nseq, H, G, d, dt)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    st = _lib.load().gattn_prefill_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(qnorm_w), _ptr(knorm_w), _ptr(pos), ctypes.c_void_p(cu.data_ptr()),
        nseq, H, G, d, int(rotary_dim), float(rope_base), float(eps), mode, q.stride(0), q.stride(1), gts, ghs, dt,
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out), _stream_handle(stream, q.device))
    check(st, "gattn_prefill_varlen")
    return out


def _check_decode_inputs(q_new, kv_cache, seqlens, gate, qnorm_w, mode, out):
    """The layout checks every contiguous-cache decode entry point makes before it
    hands pointers to the library: the kernels index these tensors as dense arrays."""
    for name, t in (("q_new", q_new), ("kv_cache", kv_cache), ("seqlens", seqlens), ("qnorm_w", qnorm_w)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if mode & 0x0F and not gate.is_contiguous():
        raise ValueError("gate must be contiguous")
    if seqlens.dtype != torch.int32:
        raise ValueError("seqlens must be int32")
    if q_new.dim() != 3 or kv_cache.dim() != 5 or kv_cache.shape[0] != 2 or kv_cache.shape[1] != q_new.shape[0]:
        raise ValueError("q_new must be [B,H,d] and kv_cache [2,B,G,Lmax,d]")
    if out is not None and (not out.is_contiguous() or out.numel() != q_new.numel()):
        raise ValueError("out must be a contiguous [B,H*d] tensor")


def gattn_decode(q_new, kv_cache, seqlens, gate, qnorm_w, *, rotary_dim, rope_base, eps=1e-6,
                 gate_mode="elementwise", gate_act="sigmoid", gate_additive=False, out=None, workspace=None,
                 stream=None):
    """One decode step.  q_new [B,H,d] raw; kv_cache [2,B,G,Lmax,d] (K normed and
    rotated, V raw); seqlens [B] int32 including the new token; gate [B,H,d]
    (elementwise), [B,H] (headwise), [B,d] (head_shared) or None; gate_act and
    gate_additive as for gattn_prefill; qnorm_w [d].  bf16.  Returns out [B,H*d]."""
    mode = _mode(gate_mode, gate_act, gate_additive)
    B, H, d = q_new.shape
    G, Lmax = kv_cache.shape[2], kv_cache.shape[3]
    _check_decode_inputs(q_new, kv_cache, seqlens, gate, qnorm_w, mode, out)
    if out is None:
        out = torch.empty((B, H * d), dtype=q_new.dtype, device=q_new.device)
    need = gattn_decode_workspace_size(B, H, G, d, Lmax)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q_new.device)
    st = _lib.load().gattn_decode(
        _ptr(q_new), _ptr(kv_cache), _ptr(seqlens), _ptr(gate if mode & 0x0F else None), _ptr(qnorm_w), B, H, G, d,
        Lmax, int(rotary_dim), float(rope_base), float(eps), mode, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _stream_handle(stream, q_new.device))
    check(st, "gattn_decode")
    return out


def gattn_decode_append(q_new, k_new, v_new, kv_cache, seqlens, gate, qnorm_w, knorm_w, *, rotary_dim, rope_base,
                        eps=1e-6, gate_mode="elementwise", gate_act="sigmoid", gate_additive=False, out=None,
                        workspace=None, stream=None):
    """One decode step that first writes the new token into the cache: k_new,
    v_new [B,G,d] raw (K is normed with knorm_w and rotated at position
    seqlens[b]-1); kv_cache [2,B,G,Lmax,d] is updated in place at row
    seqlens[b]-1; the rest as gattn_decode.  Returns out [B,H*d]."""
    mode = _mode(gate_mode, gate_act, gate_additive)
    B, H, d = q_new.shape
    G, Lmax = kv_cache.shape[2], kv_cache.shape[3]
    for name, t in (("q_new", q_new), ("k_new", k_new), ("v_new", v_new), ("kv_cache", kv_cache),
                    ("seqlens", seqlens), ("qnorm_w", qnorm_w), ("knorm_w", knorm_w)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if tuple(k_new.shape) != (B, G, d) or tuple(v_new.shape) != (B, G, d):
        raise ValueError("k_new and v_new must be [B,G,d]")
    if mode & 0x0F and not gate.is_contiguous():
        raise ValueError("gate must be contiguous")
    if seqlens.dtype != torch.int32:
        raise ValueError("seqlens must be int32")
    if out is None:
        out = torch.empty((B, H * d), dtype=q_new.dtype, device=q_new.device)
    need = gattn_decode_workspace_size(B, H, G, d, Lmax)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q_new.device)
    st = _lib.load().gattn_decode_append(
        _ptr(q_new), _ptr(k_new), _ptr(v_new), _ptr(kv_cache), _ptr(seqlens), _ptr(gate if mode & 0x0F else None),
        _ptr(qnorm_w), _ptr(knorm_w), B, H, G, d, Lmax, int(rotary_dim), float(rope_base), float(eps), mode,
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out),
        _stream_handle(stream, q_new.device))
    check(st, "gattn_decode_append")
    return out


def gattn_decode_paged(q_new, kv_pages, block_table, seqlens, gate, qnorm_w, *, rotary_dim, rope_base, eps=1e-6,
                       k_new=None, v_new=None, knorm_w=None, gate_mode="elementwise", gate_act="sigmoid",
                       gate_additive=False, out=None, workspace=None, stream=None):
    """One decode step against a paged cache: kv_pages [2,num_pages,G,page_size,d]
    bf16, block_table [B,max_pages] int32 (page of each page_size-token block of
    each sequence).  With k_new, v_new [B,G,d] and knorm_w the new token is first
    written into its page.  The rest as gattn_decode.  Returns out [B,H*d]."""
    mode = _mode(gate_mode, gate_act, gate_additive)
    B, H, d = q_new.shape
    num_pages, G, page_size = kv_pages.shape[1], kv_pages.shape[2], kv_pages.shape[3]
    max_pages = block_table.shape[1]
    for name, t in (("q_new", q_new), ("kv_pages", kv_pages), ("block_table", block_table), ("seqlens", seqlens),
                    ("qnorm_w", qnorm_w)) + ((("k_new", k_new), ("v_new", v_new), ("knorm_w", knorm_w))
                                             if k_new is not None else ()):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if block_table.dtype != torch.int32 or seqlens.dtype != torch.int32:
        raise ValueError("block_table and seqlens must be int32")
    if mode & 0x0F and not gate.is_contiguous():
        raise ValueError("gate must be contiguous")
    if out is None:
        out = torch.empty((B, H * d), dtype=q_new.dtype, device=q_new.device)
    need = gattn_decode_workspace_size(B, H, G, d, max_pages * page_size)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q_new.device)
    st = _lib.load().gattn_decode_paged(
        _ptr(q_new), _ptr(k_new), _ptr(v_new), _ptr(kv_pages), _ptr(block_table), num_pages, page_size, max_pages,
        _ptr(seqlens), _ptr(gate if mode & 0x0F else None), _ptr(qnorm_w), _ptr(knorm_w), B, H, G, d,
        int(rotary_dim), float(rope_base), float(eps), mode, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _stream_handle(stream, q_new.device))
    check(st, "gattn_decode_paged")
    return out


def gattn_decode_noalloc(q_new, kv_cache, seqlens, gate, qnorm_w, *, rotary_dim, rope_base, eps=1e-6,
                         gate_mode="elementwise", gate_act="sigmoid", gate_additive=False, out=None, stream=None):
    """gattn_decode without a workspace: the partial states live in the library's
    own fixed device array (GATTN_DECODE_NOALLOC_SCRATCH_BYTES).  For callers that
    must not allocate device memory while decoding; pass `out` to allocate nothing
    here either.  Calls that overlap on the GPU race on that array."""
    mode = _mode(gate_mode, gate_act, gate_additive)
    B, H, d = q_new.shape
    G, Lmax = kv_cache.shape[2], kv_cache.shape[3]
    _check_decode_inputs(q_new, kv_cache, seqlens, gate, qnorm_w, mode, out)
    if out is None:
        out = torch.empty((B, H * d), dtype=q_new.dtype, device=q_new.device)
    st = _lib.load().gattn_decode_noalloc(
        _ptr(q_new), _ptr(kv_cache), _ptr(seqlens), _ptr(gate if mode & 0x0F else None), _ptr(qnorm_w), B, H, G, d,
        Lmax, int(rotary_dim), float(rope_base), float(eps), mode, _ptr(out), _stream_handle(stream, q_new.device))
    check(st, "gattn_decode_noalloc")
    return out


# ------------------------------------------------------------------ 4-bit KV cache

def gattn_qcache_shape(num_pages, G, page_size, d):
    """Shape of a 4-bit KV cache, a uint8 tensor [2, num_pages, G, page_size/16, 10 d] (the
    layout is in gattn.h).  It needs no initialisation."""
    if page_size < 16 or page_size % 16 or d not in (64, 128, 256):
        raise ValueError("page_size must be a multiple of 16 and d one of 64, 128, 256")
    return (2, num_pages, G, page_size // 16, 10 * d)


# A decode step is a few microseconds on the GPU, so these wrappers stay lean: device
# indices instead of device objects, the raw handle of the current stream, no helper
# objects per call.

def _qcache_geometry(qcache, block_table):
    """(num_pages, G, page_size, d, B, max_pages, device index) of a cache and its table, checked."""
    if qcache.dim() != 5 or block_table.dim() != 2:
        raise ValueError("qcache is [2,num_pages,G,page_size/16,10 d], block_table [B,max_pages]")
    planes, num_pages, G, blocks, row = qcache.shape
    if planes != 2 or row % 10 or qcache.dtype is not torch.uint8 or not qcache.is_contiguous():
        raise ValueError("qcache must be a contiguous uint8 [2,num_pages,G,page_size/16,10 d] tensor")
    dev = qcache.get_device()
    if block_table.dtype is not torch.int32 or not block_table.is_contiguous() or block_table.get_device() != dev:
        raise ValueError("block_table must be a contiguous int32 [B,max_pages] tensor on the cache's device")
    B, max_pages = block_table.shape
    return num_pages, G, 16 * blocks, row // 10, B, max_pages, dev


def _qcache_index(name, t, n, dev):
    if t.shape != (n,) or t.dtype is not torch.int32 or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} on the cache's device")
    return t.data_ptr()


def _qcache_dense(name, t, shape, dtype, dev):
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on the cache's device")
    return t.data_ptr()


def _qcache_stride(size, stride, name):
    """A dimension's stride for the C call, where 0 selects the contiguous default: a
    dimension of one has no stride to speak of, and a broadcast one cannot be passed."""
    if size <= 1:
        return 0
    if stride == 0:
        raise ValueError(f"{name}: broadcast (stride 0) views are not supported; pass a contiguous copy")
    return stride


def _qcache_call(dev, stream, fn, *args):
    """fn(*args, stream handle) with device `dev` current."""
    if dev < 0:
        raise ValueError("the tensors must be on a CUDA device")
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        return fn(*args, s)
    with torch.cuda.device(dev):
        return fn(*args, s)


def _empty_on(stream, shape, dtype, device):
    """torch.empty whose memory belongs to the stream that will use it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def gattn_qcache_write(k, v, qcache, block_table, seqlens, knorm_w, cu_seqlens=None, *, rotary_dim, rope_base, eps=1e-6,
                       stream=None):
    """Write new tokens into a 4-bit KV cache (gattn_qcache_shape) in place and return it.

    k, v [T,G,d] raw projections, bf16 or fp32, the last dimension contiguous (views into
    a fused projection are fine); knorm_w [d] of the same dtype; K is normed and rotated.
    cu_seqlens [B+1] int32 on the device: sequence b's new tokens are rows cu_seqlens[b] ..
    cu_seqlens[b+1]-1 (rows past the last are ignored); None: one token per sequence, and a
    length of 0 marks an unused row.
    seqlens [B] int32 on the device: tokens in each sequence after the write.
    block_table [B,max_pages] int32: the page of each page_size-token stretch."""
    num_pages, G, page_size, d, B, max_pages, dev = _qcache_geometry(qcache, block_table)
    dtype = k.dtype
    if k.dim() != 3 or k.shape != v.shape or k.shape != (k.shape[0], G, d):
        raise ValueError(f"k and v must both be [T,{G},{d}], as the cache's heads")
    T = k.shape[0]
    (kt, kh, ke), (vt, vh, ve) = k.stride(), v.stride()
    if ke != 1 or ve != 1:
        raise ValueError("k and v: the last dimension must be contiguous")
    if dtype not in DTYPES or v.dtype is not dtype or k.get_device() != dev or v.get_device() != dev:
        raise ValueError("k and v must both be bfloat16 or both be float32, on the cache's device")
    if cu_seqlens is None and T != B:
        raise ValueError(f"without cu_seqlens every sequence gets one token: {T} tokens, {B} sequences")
    st = _qcache_call(
        dev, stream, _lib.load().gattn_qcache_write, k.data_ptr(), v.data_ptr(), qcache.data_ptr(),
        block_table.data_ptr(), num_pages, page_size, max_pages, _qcache_index("seqlens", seqlens, B, dev),
        None if cu_seqlens is None else _qcache_index("cu_seqlens", cu_seqlens, B + 1, dev),
        _qcache_dense("knorm_w", knorm_w, (d,), dtype, dev), T, B, G, d, rotary_dim, rope_base, eps,
        _qcache_stride(T, kt, "k"), _qcache_stride(G, kh, "k"), _qcache_stride(T, vt, "v"), _qcache_stride(G, vh, "v"),
        DTYPES[dtype])
    if st:
        check(st, "gattn_qcache_write")
    return qcache


def gattn_qcache_read(qcache, block_table, starts=None, cu_seqlens=None, *, total=None, dtype=torch.bfloat16,
                      k_out=None, v_out=None, stream=None):
    """Read cached tokens back: (k, v), each [total,G,d] in `dtype` (bf16 or fp32), K as the
    cache holds it (normed and rotated).

    Rows cu_seqlens[b] .. cu_seqlens[b+1]-1 receive the tokens starts[b], starts[b]+1, ... of
    sequence b; both are int32 on the device.  cu_seqlens None: one token per sequence
    (total = B); starts None: from token 0.  total is the number of rows, cu_seqlens[B] or
    more (rows past it are left as they were).  k_out, v_out: contiguous tensors to fill."""
    num_pages, G, page_size, d, B, max_pages, dev = _qcache_geometry(qcache, block_table)
    if total is None:
        if cu_seqlens is not None and k_out is None:
            raise ValueError("total (the number of rows) is needed with cu_seqlens")
        total = B if cu_seqlens is None else k_out.shape[0]
    if cu_seqlens is None and total != B:
        raise ValueError("without cu_seqlens one token of each sequence is read")
    if k_out is not None and v_out is not None:
        dtype = k_out.dtype
    elif k_out is not None or v_out is not None:
        raise ValueError("k_out and v_out go together")
    if dtype not in DTYPES:
        raise ValueError("the values are returned in bfloat16 or float32")
    if k_out is None:
        k_out = _empty_on(stream, (total, G, d), dtype, qcache.device)
        v_out = _empty_on(stream, (total, G, d), dtype, qcache.device)
        kp, vp = k_out.data_ptr(), v_out.data_ptr()
    else:
        kp = _qcache_dense("k_out", k_out, (total, G, d), dtype, dev)
        vp = _qcache_dense("v_out", v_out, (total, G, d), dtype, dev)
    st = _qcache_call(
        dev, stream, _lib.load().gattn_qcache_read, qcache.data_ptr(), block_table.data_ptr(), num_pages, page_size,
        max_pages, None if starts is None else _qcache_index("starts", starts, B, dev),
        None if cu_seqlens is None else _qcache_index("cu_seqlens", cu_seqlens, B + 1, dev), total, B, G, d,
        DTYPES[dtype], kp, vp)
    if st:
        check(st, "gattn_qcache_read")
    return k_out, v_out


def gattn_decode_qcache_workspace_size(B, H, G, d, Lmax) -> int:
    return _lib.load().gattn_decode_qcache_workspace_size(B, H, G, d, Lmax)


def gattn_decode_qcache(q_new, qcache, block_table, seqlens, gate, qnorm_w, *, rotary_dim, rope_base, eps=1e-6,
                        k_new=None, v_new=None, knorm_w=None, gate_mode="elementwise", gate_act="sigmoid",
                        gate_additive=False, out=None, workspace=None, stream=None):
    """One decode step against a 4-bit KV cache (gattn_qcache_shape): q_new [B,H,d] raw bf16
    queries and gate logits [B,H,d], [B,H], [B,d] or None, both possibly strided views with
    a contiguous last dimension (e.g. the halves of a packed [B,H,2d] projection).
    seqlens [B] int32 counts the new token; 0 marks an unused row.  With k_new, v_new
    [B,G,d] and knorm_w the new token is first written into the cache.  The rest as
    gattn_decode_paged.  Returns out [B,H*d]."""
    mode = _mode(gate_mode, gate_act, gate_additive)
    num_pages, G, page_size, d, B, max_pages, dev = _qcache_geometry(qcache, block_table)
    if q_new.dim() != 3 or q_new.dtype is not torch.bfloat16 or q_new.get_device() != dev:
        raise ValueError("q_new must be a bfloat16 [B,H,d] tensor on the cache's device")
    qb, H, qd = q_new.shape
    qs, qh, qe = q_new.stride()
    if qb != B or qd != d or qe != 1:
        raise ValueError(f"q_new must be [{B},H,{d}], as the table and the cache, its last dimension contiguous")
    layout = mode & 0x0F
    gp, gs, gh = None, 0, 0
    if layout:
        want = (B, H, d) if layout == 1 else (B, H) if layout == 2 else (B, d)
        if gate is None or gate.shape != want or gate.dtype is not torch.bfloat16 or gate.get_device() != dev:
            raise ValueError(f"gate must be a bfloat16 {list(want)} tensor on the cache's device")
        if layout != 2 and gate.stride(-1) != 1:
            raise ValueError("gate: the last dimension must be contiguous")
        gp, gs = gate.data_ptr(), _qcache_stride(B, gate.stride(0), "gate")
        if layout != 3:
            gh = _qcache_stride(H, gate.stride(1), "gate")
    kp = vp = wp = None
    if k_new is not None or v_new is not None or knorm_w is not None:
        if k_new is None or v_new is None or knorm_w is None:
            raise ValueError("an append needs k_new, v_new and knorm_w")
        kp = _qcache_dense("k_new", k_new, (B, G, d), torch.bfloat16, dev)
        vp = _qcache_dense("v_new", v_new, (B, G, d), torch.bfloat16, dev)
        wp = _qcache_dense("knorm_w", knorm_w, (d,), torch.bfloat16, dev)
    if out is None:
        out = _empty_on(stream, (B, H * d), torch.bfloat16, qcache.device)
        op = out.data_ptr()
    else:
        op = _qcache_dense("out", out, (B, H * d), torch.bfloat16, dev)
    if workspace is None:
        with torch.cuda.device(qcache.device):
            need = gattn_decode_qcache_workspace_size(B, H, G, d, max_pages * page_size)
        workspace = _empty_on(stream, (max(need, 1),), torch.uint8, qcache.device)
    elif not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    st = _qcache_call(
        dev, stream, _lib.load().gattn_decode_qcache, q_new.data_ptr(), kp, vp, qcache.data_ptr(),
        block_table.data_ptr(), num_pages, page_size, max_pages, _qcache_index("seqlens", seqlens, B, dev), gp,
        _qcache_dense("qnorm_w", qnorm_w, (d,), torch.bfloat16, dev), wp, B, H, G, d, rotary_dim, rope_base, eps, mode,
        _qcache_stride(B, qs, "q_new"), _qcache_stride(H, qh, "q_new"), gs, gh, workspace.data_ptr(), workspace.nbytes, op)
    if st:
        check(st, "gattn_decode_qcache")
    return out
