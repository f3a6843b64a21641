"""Plain references of the 4-bit KV cache in 64 bits, written from the format in gattn.h:
per-feature indexing into the byte layout, no step shared with the library."""
import numpy as np
import torch

BLOCK, GROUP = 16, 32


def bf16(x):
    """fp64 array rounded once to bfloat16, as fp64."""
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.bfloat16).double().numpy()


def layout(d):
    """For every feature: byte of token 0's code in a block, nibble shift, byte of its scale."""
    f = np.arange(d)
    byte = (f // 64) * (BLOCK * 32) + 4 * ((f % 32) // 4) + 2 * ((f % 64) // 32) + (f % 4) // 2
    return byte, 4 * (f % 2), 8 * d + (f // GROUP) * 2 * BLOCK


def _half(raw, at):
    bits = raw[..., at].astype(np.uint32) | (raw[..., at + 1].astype(np.uint32) << 8)
    return (bits << 16).view(np.float32).astype(np.float64)


def rows(cache, plane, page, g, slot):
    """(codes - 8 [d], scales [d/32], centres [d/32]) of one cached row; cache: numpy uint8 of the whole pool."""
    d = cache.shape[-1] // 10
    raw = cache[plane, page, g, slot // BLOCK]
    byte, shift, par = layout(d)
    t = slot % BLOCK
    code = (raw[byte + 32 * t].astype(np.int64) >> shift) & 15
    return code - 8, _half(raw, par[::GROUP] + 2 * t), _half(raw, par[::GROUP] + d + 2 * t)


def values(cache, table, b, lo, hi):
    """fp64 K and V [hi-lo, G, d] of tokens lo .. hi-1 of sequence b as the cache holds them."""
    _, _, G, blocks, row = cache.shape
    d, page = row // 10, BLOCK * blocks
    out = np.zeros((2, hi - lo, G, d))
    byte, shift, par = layout(d)
    for i, pos in enumerate(range(lo, hi)):
        pg, slot = int(table[b, pos // page]), pos % page
        t = slot % BLOCK
        raw = cache[:, pg, :, slot // BLOCK]  # [2, G, 10 d]
        code = (raw[..., byte + 32 * t].astype(np.int64) >> shift) & 15
        out[:, i] = _half(raw, par + d + 2 * t) + _half(raw, par + 2 * t) * (code - 8)
    return out[0], out[1]


def norm_rope(x, w, pos, rd, base, eps=1e-6):
    """fp64 [n,heads,d]: RMSNorm, rotate-half RoPE at positions pos [n]."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    h = rd // 2
    if h:
        a = np.asarray(pos, np.float64)[:, None] * np.power(float(base), -2.0 * np.arange(h) / rd)
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        y = np.concatenate([y[..., :h] * c - y[..., h:rd] * s, y[..., h:rd] * c + y[..., :h] * s, y[..., rd:]], -1)
    return y


def encode(x):
    """Codes - 8, scales and centres of float32 x [...,d], with the format's own roundings."""
    g = np.asarray(x, np.float32).reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    hi, lo = g.max(-1), g.min(-1)
    step = (np.float32(0.5) * hi - np.float32(0.5) * lo) * np.float32(2 / 15)
    s, c = bf16(step), bf16(lo + np.float32(8) * step)
    s = np.where(np.isfinite(step), s, np.nan)
    c = np.where(np.isfinite(step), c, np.nan)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        inv = np.where(s >= 2.0 ** -126, (np.float32(1) / s.astype(np.float32)).astype(np.float64), 0.0)
        n = np.clip(np.rint((g - c.astype(np.float32)[..., None]).astype(np.float64) * inv[..., None]), -8, 7)
    return n.reshape(x.shape), s, c


def decode(q, k, v, gate, w, L, rd, base, act=lambda z: 1 / (1 + np.exp(-z)), additive=False, eps=1e-6):
    """One sequence's step in fp64: q [H,d] raw, k, v [L,G,d], gate broadcastable to [H,d] or None."""
    H, d = q.shape
    o = np.zeros((H, d))
    if L:
        qn = norm_rope(q[None], w, [L - 1], rd, base, eps)[0]
        r = H // k.shape[1]
        for h in range(H):
            x = k[:, h // r] @ qn[h] / np.sqrt(d)
            p = np.exp(x - x.max())
            o[h] = p @ v[:, h // r] / p.sum()
    if gate is None:
        return o
    a = act(np.asarray(gate, np.float64))
    return o + a if additive else o * a
