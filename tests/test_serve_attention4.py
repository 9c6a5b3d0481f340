"""Attention over the 4-bit cache against the definition in 64 bits (bounds in serve4_util.attention4_ref), and refusals."""

import numpy as np
import pytest
import torch

import dequant_matmul_qmv_amd as mxq
from tests.gpu_util import note
from tests.serve4_util import HALF, append4_ref, attention4_ref, check_attention, frequencies, random_pool4, rotated_bits
from tests.serve_util import paging

DEV = "cuda:0"
P = 0x10000


def _call(cache="default", **kw):
    import dequant_matmul_qmv_amd._serve as serve
    c = dict(k=P, v=P, ks=P, vs=P, blocks=4, kv=2, block=16, dim=64)
    a = dict(q=P, qt=256, qh=64, table=P, stride=3, width=3, lens=P, starts=None, tokens=2, seqs=2, heads=4, window=0, scale=0.1, out=P, lse=None,
             dtype=mxq.MXQ_F16)
    c.update({n: v for n, v in kw.items() if n in c})
    a.update({n: v for n, v in kw.items() if n in a})
    st = serve._CacheStruct(c["k"], c["v"], c["ks"], c["vs"], c["blocks"], c["kv"], c["block"], c["dim"]) if cache == "default" else cache
    return serve._load().mxq_attention4(a["q"], a["qt"], a["qh"], st, a["table"], a["stride"], a["width"], a["lens"], a["starts"], a["tokens"],
                                        a["seqs"], a["heads"], a["window"], a["scale"], a["out"], a["lse"], a["dtype"], None)


def test_refusals():
    bad, unsup, mis = mxq.MXQ_ERR_INVALID_ARG, mxq.MXQ_ERR_UNSUPPORTED, mxq.MXQ_ERR_MISALIGNED
    assert _call(cache=None) == bad
    for name in ("blocks", "kv", "tokens", "seqs", "width", "heads", "window"):
        assert _call(**{name: -1}) == bad, name
    for name in ("k", "v", "ks", "vs", "q", "out", "table", "lens"):
        assert _call(**{name: None}) == bad, name
    assert _call(tokens=3) == bad and _call(stride=2) == bad
    for scale in (float("nan"), float("inf"), 3.4e38):
        assert _call(scale=scale) == bad
    for kw in (dict(block=8), dict(block=24), dict(dim=96), dict(heads=3), dict(heads=65536), dict(dtype=mxq.MXQ_F32), dict(blocks=2 ** 31),
               dict(kv=65536), dict(width=2 ** 27, stride=2 ** 27), dict(tokens=2 ** 25, seqs=2 ** 25)):
        assert _call(**kw) == unsup, kw
    for name, at in (("k", 8), ("v", 8), ("ks", 2), ("vs", 8), ("q", 8), ("out", 4), ("lse", 2), ("table", 2), ("lens", 2), ("starts", 2)):
        assert _call(**{name: P + at}) == mis, name
    assert _call(qt=260) == mis and _call(qh=68) == mis
    assert _call(heads=0, q=None, out=None) == mxq.MXQ_OK
    assert _call(tokens=0, seqs=0, q=None, out=None, table=None, lens=None) == mxq.MXQ_OK


# ----------------------------------------------------------------------------------------------- GPU
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _poison(pool, table, lens, block):
    """Scale words that are no numbers in every place behind the sequences' ends (those pages were never written, or are
    others')."""
    for t in pool[2:]:
        keep = torch.zeros(t.shape, dtype=torch.bool)
        for s, n in enumerate(lens):
            for j in range(-(-max(n, 0) // block)):
                page = int(table[s, j]) if j < table.shape[1] else -1
                if 0 <= page < t.shape[0]:
                    keep[page, :, :min(block, n - j * block)] = True
        wrong = torch.tensor([0x7C0F, -1, 0x7E05, -1024], dtype=torch.int16)
        t.copy_(torch.where(keep, t, wrong[torch.arange(t.numel()) % 4].view(t.shape)))
    return pool


def _run(q, pool, table, lens, new, window=0, scale=None, one=False, lse=True, **kw):
    starts = None if one else _i32(np.cumsum([0] + new).tolist())
    got = mxq.mxq_attention(q.to(DEV), mxq.KvCache4(*[x.to(DEV) for x in pool]), table.to(DEV), _i32(lens), starts, window=window, scale=scale,
                            return_lse=lse, **kw)
    torch.cuda.synchronize()
    return got if lse else (got, None)


def _check(dim, block, t, lens, new, heads, kv, seed, window=0, scale=None, one=False, spread=1.0, what="", table=None, edit=None, **kw):
    gen = torch.Generator().manual_seed(seed)
    blocks, tab = paging([max(n, 0) for n in lens], block, gen)
    tab = tab if table is None else table(tab, blocks)
    pool = random_pool4(blocks, kv, block, dim, gen)
    if edit is not None:
        edit(pool)
    pool = _poison(list(pool), tab, lens, block)
    q = (torch.randn(sum(new), heads, dim, generator=gen) * spread)
    q = q.clamp(-torch.finfo(HALF[t]).max, torch.finfo(HALF[t]).max).to(HALF[t])   # (scores must be finite)
    note(f"attention4 dim={dim} block={block} {t} lens={lens[:6]} new={new[:6]} heads={heads}/{kv} window={window} {what}")
    out, lse = _run(q, pool, tab, lens, new, window, scale, one, **kw)
    ref = attention4_ref(q, pool, tab, lens, new, window, dim ** -0.5 if scale is None else scale)
    check_attention(out, lse, ref, what)


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_single_tokens(block, dim, t):
    """Lengths around pages, words, chunks and parts; groups of heads; windows."""
    for lens in ([1, 2, 7, 8, 9, 15, 16, 17], [31, 33, 63, 64, 65, 100], [0, 129, 257, 300], [1025, 3, 700], [2111]):
        for heads, kv, window in ((8, 2, 0), (5, 1, 20), (2, 2, 64), (16, 1, 1)):
            _check(dim, block, t, lens, [1] * len(lens), heads, kv, block + dim, window, one=True, what="one")


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_wide_groups_and_drafts(dim, t):
    for heads, kv, new in ((20, 1, 1), (64, 2, 1), (100, 1, 1), (8, 2, 5), (4, 1, 9), (16, 1, 3), (1, 1, 40)):
        lens = [40, 333, 1200]
        _check(dim, 32, t, lens, [new] * 3, heads, kv, heads, one=new == 1, what="group")
        _check(dim, 64, t, lens, [new] * 3, heads, kv, heads, window=37, what="group, window")


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("dim,block", [(64, 16), (64, 64), (128, 32), (128, 128)])
def test_prompts(dim, block, t):
    """Whole prompts and chunks over prefixes, ragged beside single tokens and sequences without new ones."""
    for lens, new, heads, kv, window in (([200], [200], 4, 1, 0), ([131, 64, 65, 1], [131, 64, 65, 1], 4, 2, 0), ([500, 300], [100, 170], 2, 1, 0),
                                         ([700, 20, 90, 33], [129, 1, 0, 33], 8, 2, 0), ([400, 129], [200, 129], 4, 1, 50),
                                         ([300], [270], 3, 3, 1), ([1500], [65], 4, 1, 0), ([1500, 9], [80, 9], 2, 2, 333)):
        _check(dim, block, t, lens, new, heads, kv, block, window, what="prompt")


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [1, 6, 150])
def test_missing_pages_and_empty_rows(new, dim):
    """Table entries that are none, rows that see no key, lengths past the table, more new tokens than keys, negative ones."""
    lens = [300, 90, 40, -3, 200]

    def table(tab, blocks):
        tab = tab.clone()
        tab[0, 3:7], tab[0, 9] = -1, blocks
        tab[1, :] = -1
        tab[4, 1::2] = 2 ** 31 - 1
        return tab[:, :11].contiguous()          # positions from 176 on have none
    for window in (0, 30):
        _check(dim, 16, "f16", lens, [new, new, min(new, 60), new, new], 4, 2, new, window, one=False, table=table, what="missing")
        if new == 1:
            _check(dim, 16, "f16", lens, [1] * 5, 4, 2, new, window, one=True, table=table, what="missing, one")


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("new", [1, 5, 90])
def test_scores_far_apart_and_rising(new, t):
    """Large queries, scores that rise along the keys, keys of all scales and zero points, scale 0 and below 0."""
    lens = [260, 1300]

    def rising(pool):
        unit = 2.0 ** torch.linspace(-16, 2, pool[2].shape[2] * pool[2].shape[0]).view(pool[2].shape[0], 1, -1).expand(pool[2].shape)
        for x in (pool[2], pool[3]):
            x.copy_((unit.half().view(torch.int16) & 0x7FF0) | (x & 15))
    for scale, spread, edit in ((None, 8.0, None), (-0.3, 1.0, None), (0.0, 1.0, None), (1e-3, 30.0, rising), (2.0, 1.0, rising), (1.0, 4.0, None)):
        for dim in (64, 128):
            _check(dim, 16, t, lens, [new, new], 4, 1, 5, scale=scale, spread=spread, one=new == 1, edit=edit, what=f"scale {scale}")


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 90])
def test_values_at_the_ends(new):
    """Scales of the largest and the smallest word, words of zero; queries of the types' largest and smallest values."""
    big = int(np.array([4064.0], np.float16).view(np.int16)[0])

    def largest(pool):
        pool[3][:] = (pool[3] & 15) | big
        pool[2][:] = pool[2] & 15                 # keys of zero: all scores are 0

    def smallest(pool):
        pool[3][:] = (pool[3] & 15) | 16          # 2^-20
        pool[2][:] = (pool[2] & 15) | 16

    def mixed(pool):
        pool[3][:, :, ::3] = 0
        pool[2][:, :, 1::3] = 0
    for edit in (largest, smallest, mixed):
        for t in ("f16", "bf16"):
            _check(64, 32, t, [300, 70], [new, min(new, 70)], 4, 2, 6, one=new == 1, edit=edit, what=edit.__name__)
    for t, spread, scale in (("bf16", 1e38, 1e-39), ("bf16", 1e-38, 1e36), ("f16", 2e4, 1e-5), ("f16", 1e-6, 1e5)):
        _check(128, 32, t, [300, 70], [new, min(new, 70)], 4, 2, 7, one=new == 1, spread=spread, scale=scale, what=f"queries of {spread}")


@pytest.mark.gpu
def test_long_keys():
    """More keys than one part has, in several sequences of different lengths, against sampled rows."""
    for dim, block, lens in ((128, 64, [30011, 17, 9000]), (64, 16, [20001, 20000])):
        _check(dim, block, "f16", lens, [1] * len(lens), 4, 1, 8, one=True, what="long")
    _check(64, 128, "bf16", [15000], [70], 1, 1, 9, what="long chunk")


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 5, 90])
def test_the_longest_sequence(new):
    """A sequence of nearly 2^31 tokens (a table as wide as is allowed): its last 1000 keys."""
    gen = torch.Generator().manual_seed(12)
    for dim, block in ((64, 128), (128, 16)):
        width, last = (2 ** 31 - 1) // block, 1500 // block
        pool = random_pool4(last + 1, 1, block, dim, gen)
        tab = torch.zeros(1, width, dtype=torch.int32)
        tab[0, -last:] = 1 + torch.arange(last, dtype=torch.int32)
        q = torch.randn(new, 3, dim, generator=gen).half()
        ref = attention4_ref(q, pool, tab[:, -last:], [last * block - 3], [new], 1000, dim ** -0.5)
        note(f"attention4, {new} new of {width * block - 3} tokens, dim {dim}")
        out, lse = _run(q, pool, tab, [width * block - 3], [new], window=1000, one=new == 1)
        check_attention(out, lse, ref, "longest")


@pytest.mark.gpu
def test_rows_strides_streams_and_determinism():
    gen = torch.Generator().manual_seed(13)
    lens, new, block, dim = [700, 30, 2000], [40, 2, 1], 32, 128
    blocks, tab = paging(lens, block, gen)
    pool = _poison(list(random_pool4(blocks, 2, block, dim, gen)), tab, lens, block)
    wide = torch.randn(50, 12, dim + 8, generator=gen).half().to(DEV)
    q = wide[:, 2:10, 8:]
    out = torch.full((50, 8, dim), 3.0, dtype=torch.float16, device=DEV)
    cache, starts = mxq.KvCache4(*[x.to(DEV) for x in pool]), _i32([0, 40, 42, 43])
    note("attention4, strided rows, rows behind the last sequence")
    y, lse = mxq.mxq_attention(q, cache, tab.to(DEV), _i32(lens), starts, out, return_lse=True)
    torch.cuda.synchronize()
    assert y.data_ptr() == out.data_ptr() and (out[43:] == 3).all()
    check_attention(out[:43], lse[:43], attention4_ref(q[:43].cpu(), pool, tab, lens, new, 0, dim ** -0.5), "strided")
    side = torch.cuda.Stream()
    args = tab.to(DEV), _i32(lens), starts
    torch.cuda.synchronize()
    note("attention4 on another stream, and again")
    z = mxq.mxq_attention(q, cache, *args, stream=side)
    side.synchronize()
    again = mxq.mxq_attention(q, cache, *args)
    torch.cuda.synchronize()
    assert torch.equal(z[:43], out[:43]) and torch.equal(again[:43], out[:43])


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 80])
def test_graph_replay(new):
    """A captured step whose lengths grow between the replays, eager calls with other workspaces beside it."""
    gen = torch.Generator().manual_seed(14)
    block, dim, width = 32, 64, 50
    pool = random_pool4(2 * width, 2, block, dim, gen)
    cache, tab = mxq.KvCache4(*[x.to(DEV) for x in pool]), torch.randperm(2 * width, generator=gen).view(2, width).int()
    q, table, lens = torch.empty(2 * new, 4, dim, dtype=torch.float16, device=DEV), tab.to(DEV), _i32([0, 0])
    starts = None if new == 1 else _i32([0, new, 2 * new])
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mxq.mxq_attention(q, cache, table, lens, starts, out)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mxq.mxq_attention(q, cache, table, lens, starts, out)
    for rep, n in enumerate(([90, 700], [1600, 81], [200, 1111])):
        x = torch.randn(q.shape, generator=gen).half()
        q.copy_(x)
        lens.copy_(_i32(n))
        torch.cuda.synchronize()
        note(f"attention4 replay {rep}")
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        eager = mxq.mxq_attention(q, cache, table, lens, starts)
        torch.cuda.synchronize()
        assert torch.equal(got, eager)
        check_attention(got, None, attention4_ref(x, pool, tab, n, [new, new], 0, dim ** -0.5), "replay")


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_from_the_projection_to_attention(t):
    """Prompts, then steps, as a decoder runs them: rope_append into the cache, attention over it, against the definitions
    on what the cache holds."""
    gen = torch.Generator().manual_seed(15)
    heads, kv, dim, block, prompts, steps = 8, 2, 64, 16, [37, 5, 100], 4
    tab = torch.randperm(3 * 8, generator=gen).view(3, 8).int()
    cache = mxq.KvCache4.empty(24, kv, block, dim, DEV)
    held = [x.cpu() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    f, w = frequencies(dim), [(1 + 0.3 * torch.randn(dim, generator=gen)).to(HALF[t]) for _ in range(2)]
    lens = [0, 0, 0]
    for step in range(steps):
        new = prompts if step == 0 else [1, 1, 1]
        lens = [a + b for a, b in zip(lens, new)]
        n = sum(new)
        qkv = (torch.randn(n, (heads + 2 * kv) * dim, generator=gen) * 1.5).to(HALF[t])
        views = lambda x: (x[:, :heads * dim].view(n, heads, dim), x[:, heads * dim:(heads + kv) * dim].view(n, kv, dim),  # noqa: E731
                           x[:, (heads + kv) * dim:].view(n, kv, dim))
        starts = _i32(np.cumsum([0] + new).tolist()) if step == 0 else None
        note(f"rope_append, attention4, step {step}")
        q = mxq.mxq_rope_append(cache, *views(qkv.to(DEV)), f.to(DEV), tab.to(DEV), _i32(lens), starts, w[0].to(DEV), w[1].to(DEV))
        out, lse = mxq.mxq_attention(q, cache, tab.to(DEV), _i32(lens), starts, return_lse=True)
        torch.cuda.synchronize()
        x, k, v = views(qkv)
        place = torch.cat([torch.arange(a - b, a) for a, b in zip(lens, new)]).int()
        held = append4_ref(held, rotated_bits(k, w[1], 1e-6, f, place, None, False), v, tab, lens, new, block)
        for a, b in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), held):
            assert np.array_equal(a.cpu().numpy().view(b.dtype), b), step
        held = [torch.from_numpy(a.view(np.int32 if a.dtype == np.uint32 else np.int16)) for a in held]
        want = rotated_bits(x, w[0], 1e-6, f, place, None, False)
        assert torch.equal(q.cpu().view(torch.int16), want.view(torch.int16))
        check_attention(out, lse, attention4_ref(want, held, tab, lens, new, 0, dim ** -0.5), f"step {step}")
