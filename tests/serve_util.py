"""Plain references of the serving operators, in 64 bits on the CPU, and their seeded inputs."""

from __future__ import annotations

import numpy as np
import torch

HALF = {"f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype) -> float:
    """The largest relative error of one rounding to `dtype`."""
    return torch.finfo(dtype).eps / 2


def rope_ref(x, inv_freq, positions, interleaved):
    """x [tokens, heads, dim] rotated, float64."""
    y = x.double().cpu().numpy().copy()
    half = inv_freq.shape[0]
    ang = positions.cpu().numpy().astype(np.float64)[:, None] * inv_freq.cpu().numpy().astype(np.float64)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    i, j = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    a, b = y[..., i].copy(), y[..., j].copy()
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    return y


def paging(lens, block, gen, extra_pages=3, width=None):
    """A shuffled pool large enough for `lens`, and its table (entries past a sequence's end are -1)."""
    counts = [-(-n // block) for n in lens]
    total = sum(counts) + extra_pages
    ids = torch.randperm(total, generator=gen)
    width = max(counts + [1]) if width is None else width
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for s, c in enumerate(counts):
        table[s, :c] = ids[at:at + c].to(torch.int32)
        at += c
    return total, table


def random_pool(blocks, kv_heads, block, dim, gen):
    k = torch.randint(-127, 128, (blocks, kv_heads, block, dim), generator=gen, dtype=torch.int32).to(torch.int8)
    v = torch.randint(-127, 128, (blocks, kv_heads, dim, block), generator=gen, dtype=torch.int32).to(torch.int8)
    ks = 0.01 + 0.02 * torch.rand((blocks, kv_heads), generator=gen)
    vs = 0.01 + 0.02 * torch.rand((blocks, kv_heads), generator=gen)
    return k, v, ks, vs


def append_ref(pool, k, v, table, lens, new, block):
    """The stated rule, page by page in numpy: quotients in f64 rounded to f32, products in f32."""
    kc, vc, ks, vs = (t.clone().numpy() for t in pool)
    out = {"k": (kc, ks, k.float().numpy()), "v": (vc, vs, v.float().numpy())}
    at = 0
    for s, (length, n) in enumerate(zip(lens, new)):
        first = length - n
        for j in range(first // block, -(-length // block) if n else 0):
            page = int(table[s, j]) if j < table.shape[1] else -1
            lo, hi = max(first, j * block), min(length, (j + 1) * block)
            if page < 0 or page >= kc.shape[0]:
                continue
            held = lo - j * block
            for h in range(kc.shape[1]):
                for name in ("k", "v"):
                    codes, scales, x = out[name]
                    rows = x[at + lo - first:at + hi - first, h]                 # [tokens, dim]
                    was = scales[page, h] if held else np.float32(0)
                    now = max(was, np.float32(np.float64(np.abs(rows).max()) / 127))
                    ratio = np.float32(np.float64(was) / np.float64(now)) if now > 0 else np.float32(0)
                    with np.errstate(over="ignore"):
                        inv = np.float32(1 / np.float64(now)) if now > 0 else np.float32(0)
                    inv = min(inv, np.finfo(np.float32).max)
                    fresh = np.clip(np.rint(rows * inv), -127, 127).astype(np.int8)
                    tile = codes[page, h] if name == "k" else codes[page, h].T    # [block, dim] view
                    if held and ratio != 1:
                        tile[:held] = np.rint(tile[:held].astype(np.float32) * ratio).astype(np.int8)
                    tile[held:hi - j * block] = fresh
                    scales[page, h] = now
        at += n
    return kc, vc, ks, vs
