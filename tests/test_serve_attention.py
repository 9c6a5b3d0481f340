"""Attention over the 8-bit paged cache: against the definition in 64 bits, and refusals.

The error bound counts the stated roundings: P to f16 (2^-11 of each term), the
f32 scores and weights, one rounding of the output (see attention_ref)."""

import numpy as np
import pytest
import torch

import dequant_matmul_qmv_amd as mxq
from tests.gpu_util import note
from tests.serve_util import HALF, attention_ref, half_step, paging, random_pool

DEV = "cuda:0"
P = 0x10000


def _call(pool=None, **kw):
    import dequant_matmul_qmv_amd._serve as serve
    lib = serve._load()
    c = dict(k=P, v=P, k_scale=P, v_scale=P, blocks=8, kv_heads=2, block=16, dim=64)
    c.update(pool or {})
    st = serve._CacheStruct(*[c[n] for n, _ in serve._CacheStruct._fields_])
    a = dict(q=P, qt=256, qh=64, table=P, stride=4, width=4, lens=P, starts=None, tokens=3, seqs=3, heads=4, window=0,
             scale=0.125, out=P, lse=None, dtype=mxq.MXQ_F16)
    a.update(kw)
    return lib.mxq_attention(a["q"], a["qt"], a["qh"], st, a["table"], a["stride"], a["width"], a["lens"], a["starts"],
                             a["tokens"], a["seqs"], a["heads"], a["window"], a["scale"], a["out"], a["lse"],
                             a["dtype"], None)


def test_refusals():
    assert _call(dict(block=24)) == mxq.MXQ_ERR_UNSUPPORTED
    assert _call(dict(dim=80)) == mxq.MXQ_ERR_UNSUPPORTED
    assert _call(dict(k=None)) == mxq.MXQ_ERR_INVALID_ARG
    assert _call(dict(v=P + 4)) == mxq.MXQ_ERR_MISALIGNED
    assert _call(dtype=mxq.MXQ_F32) == mxq.MXQ_ERR_UNSUPPORTED
    assert _call(heads=-1) == mxq.MXQ_ERR_INVALID_ARG
    assert _call(heads=3) == mxq.MXQ_ERR_UNSUPPORTED
    assert _call(dict(kv_heads=0)) == mxq.MXQ_ERR_UNSUPPORTED
    assert _call(window=-1) == mxq.MXQ_ERR_INVALID_ARG
    assert _call(scale=float("nan")) == mxq.MXQ_ERR_INVALID_ARG
    assert _call(scale=float("inf")) == mxq.MXQ_ERR_INVALID_ARG
    assert _call(tokens=4) == mxq.MXQ_ERR_INVALID_ARG
    assert _call(stride=2) == mxq.MXQ_ERR_INVALID_ARG
    assert _call(tokens=2 ** 24, seqs=1, starts=P, heads=256) == mxq.MXQ_ERR_UNSUPPORTED
    for name in ("q", "table", "lens", "out"):
        assert _call(**{name: None}) == mxq.MXQ_ERR_INVALID_ARG, name
        assert _call(**{name: P + 1}) == mxq.MXQ_ERR_MISALIGNED, name
    assert _call(q=P + 8) == mxq.MXQ_ERR_MISALIGNED
    assert _call(qt=132) == mxq.MXQ_ERR_MISALIGNED
    assert _call(qh=65) == mxq.MXQ_ERR_MISALIGNED
    assert _call(lse=P + 2) == mxq.MXQ_ERR_MISALIGNED
    assert _call(q=None, table=None, lens=None, out=None, tokens=0, seqs=0) == mxq.MXQ_OK
    assert _call(q=None, table=None, lens=None, out=None, heads=0) == mxq.MXQ_OK


def _check(out, lse, ref, what):
    want, wlse, off, loff = ref
    y = out.double().cpu().numpy()
    tiny = 2.0 ** -25 if out.dtype == torch.float16 else 2.0 ** -134
    bound = off + half_step(out.dtype) * (np.abs(want) + off) + tiny
    err = np.abs(y - want)
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), float((err / bound).max()))
    if lse is not None:
        got = lse.double().cpu().numpy()
        assert np.array_equal(np.isneginf(got), np.isneginf(wlse)), what
        fin = ~np.isneginf(wlse)
        assert np.all(np.abs(got - wlse)[fin] <= loff[fin]), (what, float((np.abs(got - wlse)[fin] / loff[fin]).max()))


def _run(lens, new, heads, kv_heads, dim, block, t, window=0, seed=0, table=None, spread=1.0, scale=None, strided=False):
    gen = torch.Generator().manual_seed(seed + 31 * dim + block)
    blocks, tab = paging(lens, block, gen)
    pool = random_pool(blocks, kv_heads, block, dim, gen)
    if table is not None:
        tab = table(tab)
    n = sum(new)
    q = (torch.randn(n, heads, dim, generator=gen) * spread).to(HALF[t])
    ref = attention_ref(q, pool, tab, lens, new, window, dim ** -0.5 if scale is None else scale)
    cache = mxq.KvCache(*[x.to(DEV) for x in pool])
    starts = None
    if any(x != 1 for x in new):
        starts = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=DEV)
    qd = q.to(DEV)
    if strided:   # heads outermost
        qd = qd.transpose(0, 1).contiguous().transpose(0, 1)
    what = f"attention lens={lens[:8]} new={new[:8]} heads={heads}/{kv_heads} dim={dim} block={block} window={window} {t}"
    note(what)
    args = (qd, cache, tab.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), starts)
    out, lse = mxq.mxq_attention(*args, window=window, return_lse=True, scale=scale)
    again = mxq.mxq_attention(*args, window=window, scale=scale)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)), what
    _check(out, lse, ref, what)


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_one_token(dim, block, t):
    lens = [1, 0, 2, 63, 64, 65, 255, 257, 700, 16, 1300]
    _run(lens, [1] * len(lens), 8, 2, dim, block, t)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (8, 1), (10, 2), (16, 1), (20, 1), (40, 1), (70, 1), (3, 3)])
def test_one_token_head_groups(heads, kv_heads):
    _run([37, 300, 5], [1, 1, 1], heads, kv_heads, 64, 32, "f16", seed=1)


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("window", [1, 64, 100])
def test_one_token_window(window, t):
    _run([1, 50, 64, 129, 700, 0], [1] * 6, 4, 2, 128, 16, t, window=window, seed=2)


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim,block,window", [
    (8, 1, 128, 16, 0), (10, 2, 64, 32, 0), (4, 4, 64, 64, 0), (16, 2, 128, 128, 50), (2, 2, 128, 32, 3)])
def test_drafts(heads, kv_heads, dim, block, window, t):
    """A few new tokens a sequence, of more sequences than a wave has lanes, some with none."""
    lens = [(37 * i) % 300 for i in range(70)]
    new = [min(n, i % 6) for i, n in enumerate(lens)]
    _run(lens, new, heads, kv_heads, dim, block, t, window=window, seed=3)


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim,block,window", [
    (4, 1, 64, 16, 0), (10, 2, 128, 32, 0), (2, 2, 64, 64, 77), (8, 1, 128, 128, 0), (5, 1, 64, 32, 9)])
def test_prompts(heads, kv_heads, dim, block, window, t):
    lens = [401, 130, 64, 333, 1, 0, 190]
    new = [401, 100, 64, 33, 1, 0, 70]
    _run(lens, new, heads, kv_heads, dim, block, t, window=window, seed=4)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[1, 1], [90, 90]])
def test_pages_missing(new):
    """Pages that do not exist hold no keys; a sequence without any gives zeros; a length past the table is cut."""
    def spoil(tab):
        tab[0, 1:3] = -1
        tab[1, :] = 10 ** 6
        return tab
    _run([200, 100], new, 4, 2, 64, 32, "f16", seed=5, table=spoil)
    _run([200, 100], new, 4, 2, 128, 16, "bf16", seed=5, table=lambda tab: tab[:, :5].contiguous())


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[1, 1], [70, 30]])
def test_spread_and_scale(new):
    """Scores far apart (one key takes all) and far below; all heads strided; another scale; stale table entries."""
    _run([150, 90], new, 4, 2, 64, 16, "f16", seed=6, spread=30.0, strided=True)
    _run([150, 90], new, 4, 2, 128, 32, "bf16", seed=7, spread=1e-3, scale=-3.0)
    _run([150, 90], new, 4, 2, 128, 32, "bf16", seed=7, spread=1e4, scale=1e-4)

    def stale(tab):
        tab[1, 3:] = tab[0, 3:]
        return tab
    _run([150, 90], new, 4, 2, 128, 32, "bf16", seed=8, table=stale)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 70])
def test_scales_of_any_size(new):
    """Pages whose scales differ by 2^40, and all-zero pages; unwritten pages behind the end hold NaN scales."""
    gen = torch.Generator().manual_seed(9)
    lens, block = [310, 77], 16
    blocks, tab = paging(lens, block, gen)
    pool = list(random_pool(blocks, 2, block, 64, gen))
    pool[3] = pool[3] * 2.0 ** torch.randint(-40, 1, pool[3].shape, generator=gen)
    pool[2][int(tab[0, 3])] = 0
    pool[3][int(tab[0, 4])] = 0
    pool[0][int(tab[0, 3])] = 0
    loose = [b for b in range(blocks) if b not in tab.flatten().tolist()]
    for b in loose:
        pool[2][b] = float("nan")
        pool[3][b] = float("nan")
    tab[1, 5:] = loose[0]
    n = [new, new]
    q = torch.randn(sum(n), 4, 64, generator=gen).half()
    ref = attention_ref(q, pool, tab, lens, n, 0, 0.125)
    cache = mxq.KvCache(*[x.to(DEV) for x in pool])
    note(f"attention scales of any size, {new} new")
    out, lse = mxq.mxq_attention(q.to(DEV), cache, tab.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                 torch.tensor([0, new, 2 * new], dtype=torch.int32, device=DEV), return_lse=True)
    torch.cuda.synchronize()
    _check(out, lse, ref, "scales")


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 1, 64), (2, 2, 128)])
def test_long_sequences(heads, kv_heads, dim, t):
    """Key axes split into many parts, beside short ones; one token and drafts."""
    _run([9000, 3, 2500, 0, 1024, 1025], [1] * 6, heads, kv_heads, dim, 32, t, seed=13)
    _run([7001, 40], [3, 2], heads, kv_heads, dim, 64, t, window=6000, seed=14)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 260])
@pytest.mark.parametrize("step", [1.0, -1.0])
def test_rising_and_falling_scores(new, step):
    """Scores whose largest grows (or falls) from page to page, far past what one reference can stand for."""
    gen = torch.Generator().manual_seed(15)
    block, length = 16, 400
    blocks, tab = paging([length], block, gen)
    pool = list(random_pool(blocks, 1, block, 64, gen))
    for j in range(length // block):
        pool[2][int(tab[0, j])] = 0.002 * 2.0 ** (0.25 * step * (j - 12))
    q = torch.randn(new, 3, 64, generator=gen).half()
    ref = attention_ref(q, pool, tab, [length], [new], 0, 1.0)
    cache = mxq.KvCache(*[x.to(DEV) for x in pool])
    note(f"attention scores by page, step {step}, {new} new")
    out, lse = mxq.mxq_attention(q.to(DEV), cache, tab.to(DEV), torch.tensor([length], dtype=torch.int32, device=DEV),
                                 torch.tensor([0, new], dtype=torch.int32, device=DEV), scale=1.0, return_lse=True)
    torch.cuda.synchronize()
    _check(out, lse, ref, "scores by page")


@pytest.mark.gpu
def test_no_pages_at_all():
    cache = mxq.KvCache.empty(0, 2, 16, 64, DEV)
    q = torch.ones(3, 4, 64, dtype=torch.float16, device=DEV)
    lens = torch.tensor([5, 0, 1], dtype=torch.int32, device=DEV)
    note("attention without pages")
    for width in (0, 2):
        out, lse = mxq.mxq_attention(q, cache, torch.zeros(3, width, dtype=torch.int32, device=DEV), lens, return_lse=True)
        torch.cuda.synchronize()
        assert int(torch.count_nonzero(out)) == 0 and bool(torch.isneginf(lse).all())


@pytest.mark.gpu
def test_cache_beyond_32_bits():
    """Codes past 2^31 bytes: the last pages of a large pool."""
    gen = torch.Generator().manual_seed(10)
    blocks, hk, block, dim = 2 ** 31 // (4 * 128 * 128) + 5, 4, 128, 128
    small = list(random_pool(4, hk, block, dim, gen))
    cache = mxq.KvCache.empty(blocks, hk, block, dim, DEV)
    for big, part in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), small):
        big[blocks - 4:] = part.to(DEV)
    tab = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32)
    for new in (1, 90):
        q = torch.randn(new, 8, dim, generator=gen).bfloat16()
        ref = attention_ref(q, small, tab, [430], [new], 0, dim ** -0.5)
        note(f"attention past 2^31 bytes, {new} new")
        out, lse = mxq.mxq_attention(q.to(DEV), cache, (tab + (blocks - 4)).to(DEV),
                                     torch.tensor([430], dtype=torch.int32, device=DEV),
                                     torch.tensor([0, new], dtype=torch.int32, device=DEV), return_lse=True)
        torch.cuda.synchronize()
        _check(out, lse, ref, "large pool")


@pytest.mark.gpu
def test_another_stream_and_graph():
    """On a side stream, and captured: each replay equals an eager call on the same inputs."""
    gen = torch.Generator().manual_seed(12)
    lens = [700, 90, 1]
    blocks, tab = paging(lens, 32, gen)
    pool = random_pool(blocks, 2, 32, 64, gen)
    cache = mxq.KvCache(*[x.to(DEV) for x in pool])
    tab, ln = tab.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = torch.randn(3, 8, 64, generator=gen).half().to(DEV)
    out = torch.empty_like(q)
    qp = torch.randn(91, 8, 64, generator=gen).half().to(DEV)
    outp = torch.empty_like(qp)
    st = torch.tensor([0, 20, 90, 91], dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()

    def work():
        mxq.mxq_attention(q, cache, tab, ln, None, out)
        mxq.mxq_attention(qp, cache, tab, ln, st, outp)

    side = torch.cuda.Stream()
    note("attention on a side stream")
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    first = out.clone(), outp.clone()
    g = torch.cuda.CUDAGraph()
    note("attention captured")
    with torch.cuda.graph(g):
        work()
    for rep in range(3):
        if rep:
            q.copy_(torch.randn(3, 8, 64, generator=gen).half())
            qp.copy_(torch.randn(91, 8, 64, generator=gen).half())
        out.zero_()
        outp.zero_()
        torch.cuda.synchronize()
        note(f"attention replay {rep}")
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), outp.clone()
        work()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], outp), rep
        if rep == 0:
            assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
