"""The append that rotates and attention over 4 bits at their edges: caches past 32 bits of words, norms on one side, head
counts that fill no block, scales that grow with every token, two streams at once."""

import numpy as np
import pytest
import torch

import dequant_matmul_qmv_amd as mxq
from tests.serve4_util import HALF, attention4_ref, check_attention, random_pool4
from tests.serve_util import random_pool
from tests.test_serve_rope_append import DEV, Problem, _i32, _tensors, note


def _large(bits, blocks, hk, block, dim, small):
    cache = (mxq.KvCache4 if bits == 4 else mxq.KvCache).empty(blocks, hk, block, dim, DEV)
    for big, part in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), small):
        big[blocks - 4:] = part.to(DEV)
    return cache


@pytest.mark.gpu
def test_attention_past_2_31_words():
    gen = torch.Generator().manual_seed(10)
    hk, block, dim = 4, 128, 128
    blocks = 2 ** 31 // (hk * block * dim // 8) + 5
    small = list(random_pool4(4, hk, block, dim, gen))
    cache = _large(4, blocks, hk, block, dim, small)
    tab = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32)
    for new in (1, 5, 90):
        q = torch.randn(new, 8, dim, generator=gen).bfloat16()
        ref = attention4_ref(q, small, tab, [430], [new], 0, dim ** -0.5)
        note(f"attention4 past 2^31 words, {new} new")
        out, lse = mxq.mxq_attention(q.to(DEV), cache, (tab + (blocks - 4)).to(DEV), _i32([430]), None if new == 1 else _i32([0, new]),
                                     return_lse=True)
        torch.cuda.synchronize()
        check_attention(out, lse, ref, f"large pool, {new}")


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
def test_append_past_32_bits(bits):
    """The same codes as in a small cache: 2^32 bytes of 8-bit codes, 2^31 words of 4-bit ones."""
    gen = torch.Generator().manual_seed(11)
    hk, block, dim = 4, 128, 128
    blocks = (2 ** 31 // (hk * block * dim // 8) if bits == 4 else 2 ** 32 // (hk * block * dim)) + 5
    pool = list(random_pool4(4, hk, block, dim, gen) if bits == 4 else random_pool(4, hk, block, dim, gen))
    small = (mxq.KvCache4 if bits == 4 else mxq.KvCache)(*[t.clone().to(DEV) for t in pool])
    large = _large(bits, blocks, hk, block, dim, pool)
    tab = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32).to(DEV)
    f = (10000.0 ** (-torch.arange(0, dim, 2) / dim)).to(DEV)
    for new, odd in ((1, 0), (1, 1), (150, 0), (150, 1)):     # aligned rows and others
        x = torch.randn(new, 8 + 2 * hk, dim + odd, generator=gen).bfloat16().to(DEV)[..., odd:]
        q, k, v = x[:, :8], x[:, 8:8 + hk], x[:, 8 + hk:]
        starts = None if new == 1 else _i32([0, new])
        note(f"append past 32 bits, {bits} bits, {new} new, odd={odd}")
        got = [mxq.mxq_rope_append(c, q, k, v, f, tab + t, _i32([430]), starts) for c, t in ((small, 0), (large, blocks - 4))]
        torch.cuda.synchronize()
        assert torch.equal(*got)
        for a, b in zip((small.k, small.v, small.k_scale, small.v_scale), (large.k, large.v, large.k_scale, large.v_scale)):
            assert torch.equal(a, b[blocks - 4:]), (new, odd)
    assert not bool(large.k_scale[:blocks - 4].any()) and not bool(large.v_scale[:blocks - 4].any())


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("side", [0, 1])
def test_norms_on_one_side(side, inter, bits):
    for one in (True, False):
        for f32 in (False, True):
            new = [1, 1, 1] if one else [33, 9, 1]
            p = Problem(bits, 128, 32, "bf16", [50, 9, 1], new, 20 + side, inter=inter, f32=f32)
            w = list(p.w)
            w[1 - side] = None
            p2 = Problem(bits, 128, 32, "bf16", [50, 9, 1], new, 20 + side, inter=inter, norm=False)   # the same values
            assert torch.equal(p.qkv, p2.qkv)
            # what the other side gives without a norm is what the whole call gives without norms
            if side == 0:
                p.want, p.held = p2.want, p2.held
            else:
                p.want_q = p2.want_q
            p.w = w
            note(f"rope_append, norm on side {side}, {bits} bits, one={one}, f32={f32}")
            p.check(*p.call(one=one), "one side")


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dim", [64, 128])
def test_head_counts(dim, bits):
    for heads, kv in ((1, 1), (5, 5), (7, 1), (15, 3), (33, 11), (64, 1)):
        for new in ([1, 1, 1], [29, 8, 3]):
            p = Problem(bits, dim, 16, "f16", [40, 8, 3], new, heads + kv, heads=heads, kv=kv)
            note(f"rope_append, {heads}/{kv} heads of {dim}, {bits} bits, new={new}")
            p.check(*p.call(one=new[0] == 1), f"{heads}/{kv}")


@pytest.mark.gpu
@pytest.mark.parametrize("dim,block", [(64, 16), (64, 128), (128, 32), (128, 64), (128, 128)])
def test_growing_scales(dim, block):
    """Every token larger than those before it: each append rescales the older codes, of every number of them.  The codes are
    those of the plain append."""
    gen = torch.Generator().manual_seed(dim + block)
    n, hk, heads = 2 * block + 3, 2, 6
    x = torch.randn(n, heads + 2 * hk, dim, generator=gen) * (1.03 ** torch.arange(n).float())[:, None, None]
    x = x.bfloat16().to(DEV)
    a, b = (mxq.KvCache.empty(4, hk, block, dim, DEV) for _ in range(2))
    tab = torch.tensor([[2, 0, 3]], dtype=torch.int32).to(DEV)
    f = torch.zeros(0, device=DEV)
    note(f"rope_append, growing scales, dim {dim}, block {block}")
    for i in range(n):
        row = x[i:i + 1]
        mxq.mxq_rope_append(a, row[:, :heads], row[:, heads:heads + hk], row[:, heads + hk:], f, tab, _i32([i + 1]))
        mxq.mxq_kv_append(b, row[:, heads:heads + hk], row[:, heads + hk:], tab, _i32([i + 1]))
        if i % 13 == 0 or i + 1 == n or i % block in (0, block - 1):
            torch.cuda.synchronize()
            for s, t in zip(_tensors(a), _tensors(b)):
                assert torch.equal(s, t), i


@pytest.mark.gpu
def test_two_streams_at_once():
    """Calls in flight on two streams: attention with partial results, and appends into caches of their own."""
    gen = torch.Generator().manual_seed(31)
    streams, state, want = [torch.cuda.Stream() for _ in range(2)], [], []
    hk, dim, block = 2, 128, 32
    for i in range(2):
        pool = [t.to(DEV) for t in random_pool4(260, hk, block, dim, gen)]
        q = torch.randn(3, 8, dim, generator=gen).to(HALF["f16"]).to(DEV)
        tab = torch.randperm(258, generator=gen)[:3 * 86].view(3, 86).int().to(DEV)
        state.append((mxq.KvCache4(*pool), q, tab, _i32([2700, 1900 + i, 40])))
        want.append(mxq.mxq_attention(*[state[i][j] for j in (1, 0, 2, 3)]).clone())
    torch.cuda.synchronize()
    note("attention4 on two streams")
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            c, q, tab, lens = state[i]
            got[i].append(mxq.mxq_attention(q, c, tab, lens, stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])
    problems = [Problem(4, dim, block, "bf16", [50, 90], [33, 1], 40 + i) for i in range(2)]
    cases = []
    for p in problems:
        cases.append(([x.to(DEV) for x in p.views(p.qkv)], (mxq.KvCache4(*[x.to(DEV) for x in p.pool])), p.f.to(DEV), p.table.to(DEV),
                      _i32(p.lens), _i32(np.cumsum([0] + p.new).tolist()), [w.to(DEV) for w in p.w]))
    torch.cuda.synchronize()
    note("rope_append on two streams")
    outs = [mxq.mxq_rope_append(c, *x, f, tab, lens, starts, *w, stream=s)
            for s, (x, c, f, tab, lens, starts, w) in zip(streams, cases)]
    torch.cuda.synchronize()
    for p, y, case in zip(problems, outs, cases):
        p.check(y, case[1], "two streams")
