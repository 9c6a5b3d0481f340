"""Plain references of the operators from the fused projection to attention over the 4-bit cache: the definitions in 64
bits, and the stated rules of codes step by step, on the CPU."""

from __future__ import annotations

import numpy as np
import torch

from tests.serve_util import HALF, half_step  # noqa: F401

F32 = np.float32


def frequencies(rot, base=500000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()


def angles(inv_freq, positions, axes):
    """float64 [tokens, rot / 2]; positions [tokens] or [axes, tokens]."""
    p = positions.cpu().numpy().astype(np.float64)
    p = p[None] if p.ndim == 1 else p
    which = np.zeros(inv_freq.shape[0], int) if axes is None else np.clip(axes.cpu().numpy(), 0, p.shape[0] - 1)
    return p[which].T * inv_freq.cpu().numpy().astype(np.float64)


def _pairs(rot, interleaved):
    half = rot // 2
    return (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half), slice(half, rot))


def rotated_ref(x, weight, eps, inv_freq, positions, axes, interleaved):
    """(x [tokens, heads, dim] normed and rotated in float64, what its f32 steps may be off by)."""
    y = x.double().cpu().numpy().copy()
    steps = 1
    if weight is not None:
        with np.errstate(divide="ignore", invalid="ignore"):
            y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight.double().cpu().numpy()
        steps += 3                                   # r, x * r, * w
    off = np.abs(y) * steps * 2.0 ** -24
    a = angles(inv_freq, positions, axes)[:, None]
    c, s = np.cos(a), np.sin(a)
    i, j = _pairs(2 * inv_freq.shape[0], interleaved)
    p, q = y[..., i].copy(), y[..., j].copy()
    y[..., i], y[..., j] = p * c - q * s, q * c + p * s
    # a cosine's or sine's rounding, a product's, the sum's
    off[..., i] = off[..., j] = (steps + 3) * 2.0 ** -24 * (np.abs(p) + np.abs(q))
    return y, off


def rotated_bits(x, weight, eps, inv_freq, positions, axes, interleaved):
    """The same by the stated f32 steps, rounded to x's type (CPU tensor)."""
    y = x.float().cpu().numpy().copy()
    if weight is not None:
        d = x.double().cpu().numpy()
        with np.errstate(divide="ignore", invalid="ignore"):
            r = (1 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)).astype(F32)
            y = (y * r) * weight.float().cpu().numpy()
    a = angles(inv_freq, positions, axes)[:, None]
    c, s = np.cos(a).astype(F32), np.sin(a).astype(F32)
    i, j = _pairs(2 * inv_freq.shape[0], interleaved)
    p, q = y[..., i].copy(), y[..., j].copy()
    y[..., i], y[..., j] = p * c - q * s, q * c + p * s
    assert y.dtype == F32
    return torch.from_numpy(y).to(x.dtype)


# ------------------------------------------------------------------------------------------------- 4 bits
def quantize4(x):
    """(codes uint32 [..., dim], scale words uint16 [...]) of values [..., dim] by the stated rule."""
    x = x.float().cpu().numpy()
    lo, hi = np.minimum(x.min(-1), 0), np.maximum(x.max(-1), 0)
    step = (hi.astype(np.float64) - lo.astype(np.float64)) / 15
    unit = 2.0 ** np.maximum(np.frexp(step)[1] - 7, -20)
    scale = np.minimum(np.ceil(step / unit) * unit, 4064.0)
    inv = np.where(scale > 0, 1 / np.where(scale > 0, scale, 1), 0).astype(F32)
    zero = np.minimum(np.rint(-lo * inv), F32(15))
    codes = np.clip(np.rint(x * inv[..., None]) + zero[..., None], 0, 15).astype(np.uint32)
    half = scale.astype(np.float16)
    assert np.array_equal(half.astype(np.float64), scale)
    bits = half.view(np.uint16)
    assert not (bits & 0x800F).any()                 # 7 significant bits, not negative
    return codes, bits | zero.astype(np.uint16)


def pack(codes):
    """uint32 words of 8 neighbours of the last dimension."""
    c = codes.reshape(*codes.shape[:-1], -1, 8).astype(np.uint64)
    return (c << (4 * np.arange(8, dtype=np.uint64))).sum(-1).astype(np.uint32)


def unpack(words):
    return ((words[..., None].astype(np.uint32) >> (4 * np.arange(8, dtype=np.uint32))) & 15).reshape(*words.shape[:-1], -1)


def values4(pool):
    """(k, v) [blocks, kv_heads, block, dim] float64 of a pool's tensors."""
    k, v, ks, vs = (t.cpu().numpy() for t in pool)
    ks, vs = ks.view(np.uint16), vs.view(np.uint16)

    def value(codes, words):
        with np.errstate(invalid="ignore"):
            return (codes - (words & 15).astype(np.float64)[..., None]) * (words & 0x7FF0).view(np.float16).astype(np.float64)[..., None]

    kc = unpack(k.view(np.uint32)).astype(np.float64)
    vw = v.view(np.uint32)                            # [blocks, hk, block / 8, dim]
    vc = np.moveaxis(unpack(np.moveaxis(vw, 2, 3)), 2, 3).astype(np.float64)
    return value(kc, ks), value(vc, vs)


def random_pool4(blocks, kv_heads, block, dim, gen, low=0.2, high=0.4):
    """Words at random; 7-bit scales of [low, high), any zero point."""
    def words(*shape):
        return torch.randint(-2 ** 31, 2 ** 31, shape, generator=gen, dtype=torch.int64).to(torch.int32)

    def scales(*shape):
        s = (low + (high - low) * torch.rand(shape, generator=gen)).half().view(torch.int16) & 0x7FF0
        return s | torch.randint(0, 16, shape, generator=gen, dtype=torch.int16)
    return (words(blocks, kv_heads, block, dim // 8), words(blocks, kv_heads, block // 8, dim), scales(blocks, kv_heads, block),
            scales(blocks, kv_heads, block))


def append4_ref(pool, k, v, table, lens, new, block):
    """The pool's arrays (uint32, uint32, uint16, uint16) with the new rows of k (as it is to be held) and v in their places."""
    kw, vw, ks, vs = (t.clone().cpu().numpy() for t in pool)
    kw, vw, ks, vs = kw.view(np.uint32), vw.view(np.uint32), ks.view(np.uint16), vs.view(np.uint16)
    kc, ksw = quantize4(k)
    vc, vsw = quantize4(v)
    kp = pack(kc)
    at = 0
    for s, (length, n) in enumerate(zip(lens, new)):
        for i in range(n):
            pos = max(length, 0) - n + i
            j = pos // block
            page = int(table[s, j]) if 0 <= pos and j < table.shape[1] else -1
            if not 0 <= page < kw.shape[0]:
                continue
            slot = pos % block
            kw[page, :, slot], ks[page, :, slot], vs[page, :, slot] = kp[at + i], ksw[at + i], vsw[at + i]
            shift = np.uint32(4 * (slot % 8))
            old = vw[page, :, slot // 8]
            vw[page, :, slot // 8] = (old & ~(np.uint32(15) << shift)) | (vc[at + i] << shift)
        at += n
    return kw, vw, ks, vs


def attention4_ref(q, pool, table, lens, new, window, scale):
    """(out, lse, error scale of out, of lse) of the definition in float64, row by row."""
    kv, vv = values4(pool)
    k_unit = (pool[2].cpu().numpy().view(np.uint16) & 0x7FF0).view(np.float16).astype(np.float64)
    n, heads, dim = q.shape
    blocks, hk, block, _ = kv.shape
    group = heads // hk
    qd = q.double().cpu().numpy()
    out, lse = np.zeros((n, heads, dim)), np.full((n, heads), -np.inf)
    off, loff = np.zeros((n, heads, dim)), np.zeros((n, heads))
    at = 0
    for s, (length, nn) in enumerate(zip(lens, new)):
        length = max(length, 0)
        pages = [int(table[s, j]) if j < table.shape[1] else -1 for j in range(-(-length // block))]
        there = np.array([0 <= p < blocks for p in pages], bool)
        ids = np.where(there, pages, 0).astype(int) if pages else np.zeros(0, int)
        seen_page = np.repeat(there, block)[:length]
        for h in range(hk):
            k, v, unit = kv[ids, h].reshape(-1, dim)[:length], vv[ids, h].reshape(-1, dim)[:length], k_unit[ids, h].reshape(-1)[:length]
            for i in range(nn):
                pos = length - nn + i
                j = np.arange(length)
                see = seen_page & (j <= pos) & ((j > pos - window) if window else True)
                if not see.any():
                    continue
                for g in range(group):
                    row = qd[at + i, h * group + g]
                    x = scale * (k[see] @ row)
                    top = x.max()
                    p = np.exp(x - top)
                    l = p.sum()
                    o = (at + i, h * group + g)
                    out[o] = p @ v[see] / l
                    lse[o] = top + np.log(l)
                    # sums of dim products with codes up to 15 and with the zero point in f32, their scale; a bf16 q's
                    # 2^-25 of its largest; the scores' roundings, exp2
                    a = abs(scale) * 15 * np.abs(row).sum() * unit[see].max()
                    aq = abs(scale) * np.abs(row).max() * np.abs(k[see]).sum(1).max()
                    d = (2 * dim + 32) * 2.0 ** -24 * a + 2.0 ** -24 * aq + 2.0 ** -18 + 2.0 ** -22 * np.abs(x).max()
                    off[o] = (2.0 ** -11 + 2 * d) * (p @ np.abs(v[see])) / l + 2.0 ** -39 * np.abs(v[see]).sum(0) / l
                    loff[o] = d + 2.0 ** -22 * (abs(lse[o]) + 20)
        at += nn
    return out, lse, off, loff


def check_attention(out, lse, ref, what):
    """out and lse within the reference's bounds and the storage type's rounding."""
    want, wlse, off, loff = ref
    half = half_step(out.dtype)
    tiny = torch.finfo(out.dtype).smallest_normal * half * 2
    got = out.double().cpu().numpy()
    err = np.abs(got - want)
    bound = off * (1 + half) + np.abs(want) * half + tiny
    assert np.all(err <= bound), (what, float((err / bound).max()))
    if lse is not None:
        got = lse.double().cpu().numpy()
        fin = np.isfinite(wlse)
        assert np.array_equal(fin, np.isfinite(got)) and np.all(got[~fin] == -np.inf), what
        assert np.all(np.abs(got[fin] - wlse[fin]) <= loff[fin]), (what, float((np.abs(got[fin] - wlse[fin]) / loff[fin]).max()))
