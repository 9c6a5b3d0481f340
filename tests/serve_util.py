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


def attention_ref(q, pool, table, lens, new, window, scale):
    """(out, lse, error scale of out, of lse) of the definition in float64, row by row."""
    kc, vc, ks, vs = (t.double().numpy() for t in pool)
    n, heads, dim = q.shape
    blocks, hk, block, _ = kc.shape
    group = heads // hk
    qd = q.double().numpy()
    out, lse = np.zeros((n, heads, dim)), np.full((n, heads), -np.inf)
    off, loff = np.zeros((n, heads, dim)), np.zeros((n, heads))
    at = 0
    for s, (length, nn) in enumerate(zip(lens, new)):
        pages = [int(table[s, j]) if j < table.shape[1] else -1 for j in range(-(-length // block))]
        there = np.array([0 <= p < blocks for p in pages], bool)
        ids = np.where(there, pages, 0).astype(int) if pages else np.zeros(0, int)
        seen_page = np.repeat(there, block)[:length]
        for h in range(hk):
            k = (kc[ids, h] * ks[ids, h][:, None, None]).reshape(-1, dim)[:length]
            v = (vc[ids, h] * vs[ids, h][:, None, None]).transpose(0, 2, 1).reshape(-1, dim)[:length]
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
                    # f32: sums of dim products, the scores' roundings, exp2; q's own 2^-25 for bf16
                    a = abs(scale) * np.abs(k[see] * row).sum(1).max()
                    aq = abs(scale) * np.abs(row).max() * np.abs(k[see]).sum(1).max()
                    d = 2 * ((dim + 8) * 2.0 ** -24 * a + 2.0 ** -24 * aq + 2.0 ** -18)
                    off[o] = (2.0 ** -11 + 2 * d) * (p @ np.abs(v[see])) / l
                    loff[o] = d + 2.0 ** -22 * (abs(lse[o]) + 20)
        at += nn
    return out, lse, off, loff


def sample_ref(x, u, temperature, top_k, top_p, min_p):
    """(token, probability, distance of the nearest border) of one row in float64: the tokens in descending order,
    equals by index, cut to the kept prefix, one drawn in index order.  The distance, relative to the total, is that
    of u's border and of top_p's and min_p's."""
    x = x.astype(np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    order = np.argsort(-x, kind="stable")
    top = x[order[0]]
    if not temperature > 0 or not top_p > 0 or not min_p <= 1:
        return int(order[0]), 1.0, 1.0
    with np.errstate(invalid="ignore"):
        w = np.where(x == top, 1.0, np.exp((x - top) / np.float64(temperature)))
    s = w[order]
    keep = len(s) if top_k <= 0 else min(len(s), top_k)
    near = 1.0
    if top_p < 1:
        mass = np.cumsum(s[:keep])
        at = np.float64(top_p) * mass[-1]
        near = min(near, float(np.abs(mass - at).min() / mass[-1]))
        keep = 1 + int((mass[:-1] < at).sum())
    if min_p > 0:
        near = min(near, float(np.abs(s - np.float64(min_p)).min()))
        keep = max(1, min(keep, int((s >= np.float64(min_p)).sum())))
    ids = np.sort(order[:keep])
    mass = np.cumsum(w[ids])
    at = np.float64(u) * mass[-1]
    near = min(near, float(np.abs(mass - at).min() / mass[-1]))
    i = min(keep - 1, int((mass <= at).sum()))
    return int(ids[i]), float(w[ids[i]] / mass[-1]), near
