"""Attention over 4 bits: what a row's mask hides has no part in how its sums are held, however large its scale."""

import numpy as np
import pytest
import torch

from tests.gpu_util import note
from tests.serve4_util import HALF, attention4_ref, check_attention, random_pool4, unpack
from tests.test_serve_attention4 import _run

LARGEST = int(np.array([4064.0], np.float16).view(np.int16)[0])


def _problem(dim, block, t, lens, new, heads, kv, large, sink, seed):
    """Values of a few times 2^-20 but for a key with the largest scale there is (`large` of each sequence), and one that
    takes nearly all weight and whose value is 0 (`sink`): the output is what 2^-8 of the largest weight gives."""
    gen = torch.Generator().manual_seed(seed)
    width = -(-max(lens) // block)
    table = torch.randperm(len(lens) * width, generator=gen).view(len(lens), width).int()
    pool = random_pool4(len(lens) * width, kv, block, dim, gen)
    k, _, k_scale, v_scale = pool
    k[:], k_scale[:] = 0, 0
    v_scale.copy_((torch.randint(1, 8, v_scale.shape, generator=gen) * 16 + (v_scale & 15)).to(torch.int16))
    for s, n in enumerate(lens):
        page = lambda j: (int(table[s, j // block]), slice(None), j % block)  # noqa: E731
        v_scale[page(large(n))] = LARGEST | 7
        v_scale[page(sink(n))] = 5
        k[page(sink(n))] = 0x11111111                                    # 1 / 4 in every value
        k_scale[page(sink(n))] = int(np.array([0.25], np.float16).view(np.int16)[0])
    q = 8 * np.log(2) * 4 / dim ** 0.5 * (1 + 0.1 * torch.randn(sum(new), heads, dim, generator=gen))
    return q.to(HALF[t]), pool, table


def _weights_off(pool, table, lens, new, heads, window):
    """What the outputs may be off by where weights times scales leave f16's normal range.  A row holds weight * scale *
    2^(14 - k), with 2^k at most twice the largest scale S that it sees: below 2^-14 that is rounded by 2^-25 at most, so
    weight * scale by 2^-25 * 2^(k - 14) <= 2^-38 S, and a key's c - z takes it into the output.  Weights are relative to
    one that is at least 1, so dividing by their sum makes it no larger.  (attention4_ref has scales of one size in mind.)"""
    v, scales = pool[1].numpy().view(np.uint32), pool[3].numpy().view(np.uint16)
    codes = np.moveaxis(unpack(np.moveaxis(v, 2, 3)), 2, 3).astype(np.float64)         # [blocks, kv, block, dim]
    apart = np.abs(codes - (scales & 15)[..., None])
    unit = (scales & 0x7FF0).view(np.float16).astype(np.float64)
    hk, block, dim = codes.shape[1:]
    off, at = np.zeros((sum(new), heads, dim)), 0
    for s, (n, m) in enumerate(zip(lens, new)):
        pages = table[s, :-(-n // block)].numpy()
        for h in range(hk):
            a, u = apart[pages, h].reshape(-1, dim), unit[pages, h].reshape(-1)
            for i in range(m):
                last = n - m + i
                see = slice(max(last - window + 1, 0) if window else 0, last + 1)
                rows = slice(h * (heads // hk), (h + 1) * (heads // hk))
                off[at + i, rows] = 2.0 ** -38 * u[see].max() * a[see].sum(0)
        at += m
    return off


def _check(dim, block, t, lens, new, heads, kv, window, large, sink, what):
    q, pool, table = _problem(dim, block, t, lens, new, heads, kv, large, sink, dim + block)
    note(f"hidden scales: {what} dim={dim} block={block} {t} lens={lens} new={new} heads={heads}/{kv} window={window}")
    out, lse = _run(q, pool, table, lens, new, window, one=max(new) == 1)
    want, wlse, off, loff = attention4_ref(q, pool, table, lens, new, window, dim ** -0.5)
    check_attention(out, lse, (want, wlse, off + _weights_off(pool, table, lens, new, heads, window), loff), what)


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("dim,block", [(64, 16), (64, 128), (128, 32)])
def test_before_the_window(dim, block, t):
    """The key just before the window, in the chunk where it begins."""
    for window in (3, 41):
        for new, heads, kv in ((1, 4, 2), (1, 20, 1)):
            _check(dim, block, t, [60, 300, 3001], [new] * 3, heads, kv, window, lambda n: n - window - 1, lambda n: n - window, "window")
        # of a draft: hidden from its later tokens alone
        _check(dim, block, t, [60, 300, 3001], [3] * 3, 4, 2, window, lambda n: n - window - 1, lambda n: n - window, "window of a draft")


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("dim,block", [(64, 16), (64, 128), (128, 32)])
def test_later_tokens_of_a_draft(dim, block, t):
    """The draft's last token, which its earlier ones do not see."""
    for new, heads, kv in ((2, 2, 2), (5, 2, 1), (5, 8, 1), (60, 1, 1)):
        for sink in (lambda n: 3, lambda n: n - new - 1):
            _check(dim, block, t, [90, 300, 3001], [new] * 3, heads, kv, 0, lambda n: n - 1, sink, "draft")
