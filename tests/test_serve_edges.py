"""The serving operators at the ends of their ranges: lengths near 2^31, windows, scales and scores far apart, launches
past a grid's limit, values and settings at their borders.  References and bounds as in the operators' own tests."""

import numpy as np
import pytest
import torch

import dequant_matmul_qmv_amd as mxq
from tests.gpu_util import note
from tests.serve_util import HALF, append_ref, attention_ref, random_pool, rope_ref
from tests.test_serve_attention import _call as _attention_call
from tests.test_serve_attention import _check
from tests.test_serve_rope_kv import _append as _append_call
from tests.test_serve_sample import _check as _check_draw

DEV = "cuda:0"


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _attend(q, pool, tab, lens, new, **kw):
    """(out, lse) of a call on the pool's copy on the GPU."""
    cache = mxq.KvCache(*[x.to(DEV) for x in pool])
    starts = None if all(n == 1 for n in new) else _i32(np.cumsum([0] + new).tolist())
    out, lse = mxq.mxq_attention(q.to(DEV), cache, tab.to(DEV), _i32(lens), starts, return_lse=True, **kw)
    torch.cuda.synchronize()
    return out, lse


# ------------------------------------------------------------------------------------------- long sequences
@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 5, 90])
@pytest.mark.parametrize("dim,block", [(64, 128), (128, 16)])
def test_attention_of_the_longest_sequence(dim, block, new):
    """A sequence of nearly 2^31 tokens (a table as wide as is allowed, its early pages all one): the last 1000 keys
    are those of a short sequence that ends in the same pages."""
    gen = torch.Generator().manual_seed(block)
    width, last = (2 ** 31 - 1) // block, 1500 // block
    pool = random_pool(last + 1, 1, block, dim, gen)
    tab = torch.zeros(1, width, dtype=torch.int32)
    tab[0, -last:] = 1 + torch.arange(last, dtype=torch.int32)
    q = torch.randn(new, 3, dim, generator=gen).half()
    for cut in (0, 3):
        length = width * block - cut
        ref = attention_ref(q, pool, tab[:, -last:], [last * block - cut], [new], 1000, dim ** -0.5)
        note(f"attention, {new} new of {length} tokens, dim {dim}")
        out, lse = _attend(q, pool, tab, [length], [new], window=1000)
        _check(out, lse, ref, f"longest {length}")


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 70])
def test_append_to_the_longest_sequence(new):
    gen = torch.Generator().manual_seed(17)
    block, dim = 64, 64
    width, last = (2 ** 31 - 1) // block, 3
    pool = random_pool(last + 1, 2, block, dim, gen)
    tab = torch.zeros(1, width, dtype=torch.int32)
    tab[0, -last:] = 1 + torch.arange(last, dtype=torch.int32)
    k, v = (torch.randn(new, 2, dim, generator=gen).half() for _ in range(2))
    want = append_ref(pool, k, v, tab[:, -last:], [last * block - 5], [new], block)
    cache = mxq.KvCache(*[x.to(DEV) for x in pool])
    note(f"append of {new} at {width * block - 5}")
    mxq.mxq_kv_append(cache, k.to(DEV), v.to(DEV), tab.to(DEV), _i32([width * block - 5]), None if new == 1 else _i32([0, new]))
    torch.cuda.synchronize()
    for got, w in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), want):
        assert np.array_equal(got.cpu().numpy(), w)


# --------------------------------------------------------------------------------- small weights, small v scales
def _spread_pool(lens, heads, dim, block, gen, fall, v_bits):
    """(pool, table, q): scores that fall up to `fall` below a row's largest in small steps, pages whose v scales lie up
    to 2^v_bits apart, one of them below f32's normal range.  A key holds one code throughout, a query one value, so that
    the scores are exact but for their scaling."""
    counts = [-(-n // block) for n in lens]
    blocks = sum(counts)
    k, v, ks, vs = random_pool(blocks, heads, block, dim, gen)
    codes = torch.randint(-127, 128, (blocks, heads, block, 1), generator=gen, dtype=torch.int32)
    codes[:, :, 0] = 127                                       # every page holds a key of the largest score
    k = codes.to(torch.int8).expand(-1, -1, -1, dim).contiguous()
    ks[:] = fall / 254 / dim ** 0.5                            # score = dim^-0.5 * dim * ks * code
    vs = vs * 2.0 ** -torch.randint(0, v_bits + 1, vs.shape, generator=gen)
    tab = torch.full((len(lens), max(counts)), -1, dtype=torch.int32)
    ids, at = torch.randperm(blocks, generator=gen).int(), 0
    for s, c in enumerate(counts):
        tab[s, :c] = ids[at:at + c]
        at += c
    vs[int(tab[0, counts[0] // 2])] = 1e-39
    return (k, v, ks, vs), tab


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [1, 7, 150])
def test_small_weights_in_pages_of_small_scales(new, dim, t):
    """A weight times its page's share of the largest v scale passes below every f32 number."""
    gen = torch.Generator().manual_seed(dim + new)
    lens, block = [301, 1210], 16
    for fall, v_bits in ((110.0, 40), (95.0, 12), (60.0, 70)):
        pool, tab = _spread_pool(lens, 2, dim, block, gen, fall, v_bits)
        q = torch.ones(2 * new, 4, dim).to(HALF[t])
        ref = attention_ref(q, pool, tab, lens, [new, new], 0, dim ** -0.5)
        note(f"attention fall {fall} v scales 2^-{v_bits} {new} new, dim {dim} {t}")
        out, lse = _attend(q, pool, tab, lens, [new, new])
        _check(out, lse, ref, f"fall {fall} {v_bits}")


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [1, 6, 150])
def test_masked_pages_of_tiny_scales(new, dim):
    """Pages whose v scales' quotient is past f32's range, the small one's keys masked for the rows beside the large one."""
    gen = torch.Generator().manual_seed(3 * dim + new)
    block, length = 16, 150
    pool = list(random_pool(10, 1, block, dim, gen))
    pool[3][::3] *= 6000.0                         # up to 180
    pool[3][2::3] = 2.0 ** -126 * 1.5
    tab = torch.arange(10, dtype=torch.int32)[None]
    q = torch.randn(new, 8, dim, generator=gen).half() * 0.2
    for window in (0, 20):
        ref = attention_ref(q, pool, tab, [length], [new], window, dim ** -0.5)
        note(f"attention tiny v scales, {new} new, dim {dim}, window {window}")
        out, lse = _attend(q, pool, tab, [length], [new], window=window)
        _check(out, lse, ref, f"tiny scales {window}")


# ------------------------------------------------------------------------------------- windows, odd lengths
@pytest.mark.gpu
@pytest.mark.parametrize("window", [1, 2 ** 31 - 40, 2 ** 31 - 1, 2 ** 31, 2 ** 40])
def test_wide_windows_and_more_new_tokens_than_keys(window):
    """The first new tokens of a sequence shorter than they are have no keys, the others theirs, under any window."""
    gen = torch.Generator().manual_seed(18)
    block = 16
    for lens, new in (([5, 3, 40], [9, 12, 7]), ([50, 3, 70], [130, 100, 70]), ([60], [200]), ([0, 9], [4, 9])):
        pool = random_pool(12, 2, block, 64, gen)
        tab = torch.randperm(12, generator=gen)[:len(lens) * 4].view(len(lens), 4).int() if len(lens) < 3 else torch.arange(12).view(3, 4).int()
        tab = torch.cat((tab, tab[:, :1]), 1)
        q = torch.randn(sum(new), 4, 64, generator=gen).half()
        ref = attention_ref(q, pool, tab, lens, new, window, 0.125)
        note(f"attention {lens} {new} window {window}")
        out, lse = _attend(q, pool, tab, lens, new, window=window)
        _check(out, lse, ref, f"{lens} {new} {window}")


@pytest.mark.gpu
@pytest.mark.parametrize("length", [-1, -70, -2 ** 31])
def test_negative_lengths_are_empty(length):
    gen = torch.Generator().manual_seed(19)
    pool = random_pool(4, 1, 16, 64, gen)
    tab = torch.arange(4, dtype=torch.int32)[None]
    for new in (1, 6, 100):
        q = torch.randn(new, 2, 64, generator=gen).half()
        for window in (0, 5):
            note(f"attention of a length {length}, {new} new, window {window}")
            out, lse = _attend(q, pool, tab, [length], [new], window=window)
            assert int(torch.count_nonzero(out)) == 0 and bool(torch.isneginf(lse).all())
        cache = mxq.KvCache(*[x.to(DEV) for x in pool])
        kv = torch.randn(new, 1, 64, generator=gen).half().to(DEV)
        note(f"append to a length {length}, {new} new")
        mxq.mxq_kv_append(cache, kv, kv, tab.to(DEV), _i32([length]), None if new == 1 else _i32([0, new]))
        torch.cuda.synchronize()
        for got, was in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), pool):
            assert torch.equal(got.cpu(), was)


# ------------------------------------------------------------------------------------------------ the cache
@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "device", "blocks", "kv_heads", "block", "dim"])
def test_a_caches_parts_cannot_be_replaced(name):
    """The calls pass the addresses of the tensors that a cache was made of: another tensor in their place would leave
    them with memory that may be freed."""
    cache = object.__new__(mxq.KvCache)
    with pytest.raises(AttributeError):
        setattr(cache, name, None)


# ------------------------------------------------------------------------------------------------- sampling
DRAWS = [(1.0, 0, 1.0, 0.0), (0.8, 40, 0.95, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.02), (1.0, 2500, 1.0, 0.0),
         (3.0, 3000, 0.9, 0.1), (0.0, 0, 1.0, 0.0)]


def _draw(x, u, s, **kw):
    rows = x.shape[0]
    tok = torch.full((rows,), -7, dtype=torch.int32, device=DEV)
    prob = torch.full((rows,), -7.0, device=DEV)
    mxq.mxq_sample(x, u, tok, prob, temperature=s[0], top_k=s[1], top_p=s[2], min_p=s[3], **kw)
    torch.cuda.synchronize()
    return tok.cpu().tolist(), prob.cpu().tolist()


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 150])
@pytest.mark.parametrize("vocab", [300, 9001])
def test_uniform_numbers_outside_their_range(vocab, rows):
    """Below 0 as 0; 1, beyond it and NaN: the last kept token, by index."""
    gen = torch.Generator().manual_seed(50)
    x = (torch.randn(rows, vocab, generator=gen) * 0.7).half().to(DEV)
    full = lambda v: torch.full((rows,), v, device=DEV)  # noqa: E731
    for s in DRAWS:
        note(f"sample u outside, rows {rows} vocab {vocab} {s}")
        zero, last = _draw(x, full(0.0), s), _draw(x, full(1 - 2.0 ** -24), s)
        for v in (-0.0, -1e-30, -0.5, -3.0, -float("inf")):
            assert _draw(x, full(v), s) == zero, (s, v)
        for v in (1.0, 7.0, float("inf"), float("nan")):
            assert _draw(x, full(v), s) == last, (s, v)


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab", [9, 700, 5000, 128256])
def test_masked_tokens_are_never_drawn(vocab, t):
    """Rows without limits (and with), whose last tokens, or whole pieces of tokens, are -inf or NaN."""
    gen = torch.Generator().manual_seed(51)
    x = torch.randn(6, vocab, generator=gen).to({**HALF, "f32": torch.float32}[t])
    x[0, vocab // 2:] = -torch.inf
    x[1, 1:] = torch.nan
    x[2, :-1] = -torch.inf
    x[3, ::2] = -torch.inf
    x[4, vocab // 3:] = torch.nan
    x[4, -1] = -torch.inf
    ok = ~(torch.isneginf(x) | torch.isnan(x))
    last = [int(torch.nonzero(r).max()) for r in ok]
    xd = x.to(DEV)
    for s in DRAWS + [(1e30, 0, 1.0, 0.0), (float("inf"), 0, 1.0, 0.0), (1e30, 0, 0.9, 0.0)]:
        for v in (0.0, 0.3, 0.99, 1 - 2.0 ** -24, 1.0, float("nan")):
            note(f"sample masked {vocab} {t} {s} {v}")
            tok, prob = _draw(xd, torch.full((6,), v, device=DEV), s)
            assert all(bool(ok[r, i]) for r, i in enumerate(tok)), (s, v, tok)
            assert all(0 < p <= 1 for p in prob), (s, v, prob)
            if s == DRAWS[0] and not v < 1:
                assert tok == last, (s, v)


# --------------------------------------------------------------------------------------- queries of any size
@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [1, 5, 140])
def test_bf16_queries_at_the_ends_of_their_range(new, dim):
    """Rows whose largest value has bf16's highest exponent, or is below its normal range, over keys of the opposite
    size: the scores are ordinary."""
    gen = torch.Generator().manual_seed(dim + new)
    block, length = 32, 200
    tab = torch.randperm(7, generator=gen).int()[None]
    for size, key in ((2.0 ** 127, 2.0 ** -127), (2.0 ** -130, 2.0 ** 126)):
        pool = list(random_pool(7, 2, block, dim, gen))
        pool[2] *= key
        q = ((torch.rand(new, 4, dim, generator=gen) + 0.5).clamp(max=1.9) * size * torch.randn(new, 4, dim, generator=gen).sign()).bfloat16()
        assert bool(torch.isfinite(q).all())
        ref = attention_ref(q, pool, tab, [length], [new], 0, dim ** -0.5)
        note(f"attention bf16 q of {size}, {new} new, dim {dim}")
        out, lse = _attend(q, pool, tab, [length], [new])
        _check(out, lse, ref, f"q of {size}")


@pytest.mark.parametrize("scale", [2.4e38, -2.4e38, 3.4e38, float("nan"), float("-inf")])
def test_a_scale_that_overflows_is_refused(scale):
    assert _attention_call(scale=scale) == mxq.MXQ_ERR_INVALID_ARG


def test_numbers_past_32_bits_as_top_k():
    """A number that the library's int32 cannot hold stays what it means: no limit."""
    from dequant_matmul_qmv_amd import _serve
    for k in (2 ** 31, 2 ** 32 + 5, 2 ** 63, 10 ** 30):
        p, k_all = _serve._setting("mxq_sample", "top_k", k, 3, torch.int32, None)
        assert p is None and _serve._SamplingStruct(None, None, None, None, 1.0, k_all, 1.0, 0.0).top_k_all == 2 ** 31 - 1
    for k in (-1, -2 ** 31, -2 ** 32 + 5, -10 ** 30, 0):
        _, k_all = _serve._setting("mxq_sample", "top_k", k, 3, torch.int32, None)
        assert _serve._SamplingStruct(None, None, None, None, 1.0, k_all, 1.0, 0.0).top_k_all <= 0
    assert _serve._setting("mxq_sample", "top_k", 40, 3, torch.int32, None) == (None, 40)


# --------------------------------------------------------------------------------------------- large launches
@pytest.mark.gpu
@pytest.mark.parametrize("dim,rot", [(2, 2), (16, 16)])
def test_rope_of_more_tokens_than_a_grid_holds(dim, rot):
    """A workgroup of 256 threads a token: 2^24 of them are one grid's limit."""
    n = 2 ** 24 + 9
    gen = torch.Generator(device=DEV).manual_seed(60)
    q = torch.randn(n, 1, dim, generator=gen, device=DEV).half()
    positions = torch.randint(0, 131072, (n,), generator=gen, device=DEV, dtype=torch.int32)
    inv_freq = torch.logspace(0, -3, rot // 2, device=DEV)
    note(f"rope of {n} tokens, dim {dim}")
    out, _ = mxq.mxq_rope(q, None, inv_freq, positions)
    torch.cuda.synchronize()
    for at in (0, 2 ** 23 - 4, 2 ** 24 - 4, n - 8):
        part = slice(at, at + 8)
        want = rope_ref(q[part], inv_freq, positions[part], False)
        err = np.abs(out[part].double().cpu().numpy() - want)
        # a turn in f32 (2^-22 of the pair's size), rounded once to f16
        assert (err <= np.abs(want) * 2.0 ** -11 + 2.0 ** -25 + np.abs(want).max() * 2.0 ** -21).all(), at


@pytest.mark.gpu
def test_more_sequences_than_a_grid_holds_are_refused():
    """By an error that says so, before anything is launched; nothing is written."""
    n = 2 ** 23
    cache = mxq.KvCache.empty(1, 4, 16, 64, DEV)
    table, lens = torch.zeros(n, 1, dtype=torch.int32, device=DEV), torch.ones(n, dtype=torch.int32, device=DEV)
    starts = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    q = torch.ones(1, 4, 64, dtype=torch.float16, device=DEV)
    out = torch.full_like(q, 7.0)
    note("refused: too many sequences")
    with pytest.raises(mxq.MxqError) as e:
        mxq.mxq_attention(q, cache, table, lens, starts, out)
    assert e.value.status == mxq.MXQ_ERR_UNSUPPORTED and "split the call" in str(e.value)
    with pytest.raises(mxq.MxqError) as e:
        mxq.mxq_kv_append(cache, q, q, table, lens, starts)
    assert e.value.status == mxq.MXQ_ERR_UNSUPPORTED and "split the call" in str(e.value)
    torch.cuda.synchronize()
    assert bool((out == 7.0).all()) and int(torch.count_nonzero(cache.k_scale)) == 0


def test_append_of_more_sequences_than_a_grid_holds():
    assert _append_call(tokens=1, seqs=2 ** 23, starts=0x10000) == mxq.MXQ_ERR_UNSUPPORTED


# ---------------------------------------------------------------------------------------- values of any size
@pytest.mark.gpu
@pytest.mark.parametrize("size", [2.0 ** 118, 2.0 ** -110])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,new", [([900, 40], [1, 1]), ([5000, 300], [1, 1]), ([400, 30], [3, 5]), ([3001], [7]),
                                      ([700], [700]), ([5001], [80])])
def test_values_at_the_ends_of_their_range(lens, new, dim, size):
    """v near the largest and the smallest bf16 numbers, with the key axis in one part and in several."""
    gen = torch.Generator().manual_seed(len(lens) + dim + new[0])
    block, blocks = 64, sum(-(-n // 64) for n in lens)
    pool = list(random_pool(blocks, 1, block, dim, gen))
    pool[3] *= size
    tab, at = torch.full((len(lens), -(-max(lens) // block)), -1, dtype=torch.int32), 0
    for s, n in enumerate(lens):
        c = -(-n // block)
        tab[s, :c] = torch.arange(at, at + c)
        at += c
    q = torch.randn(sum(new), 4, dim, generator=gen).bfloat16() * 0.1      # flat: the sum of all weights is large
    ref = attention_ref(q, pool, tab, lens, new, 0, dim ** -0.5)
    assert np.abs(ref[0]).max() < 3e38
    note(f"attention v of {size}, {lens} {new}, dim {dim}")
    out, lse = _attend(q, pool, tab, lens, new)
    _check(out, lse, ref, f"v of {size}")


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("lens,new", [([300, 200, 90], [1, 1, 1]), ([300, 200, 90], [4, 3, 5]), ([300, 3000, 90], [150, 90, 80])])
def test_a_bad_query_row_stays_its_own(lens, new, t):
    """NaN and infinite queries beside others, in one wave and one workgroup: those keep their results."""
    gen = torch.Generator().manual_seed(70 + sum(new))
    block, blocks = 32, sum(-(-n // 32) for n in lens)
    pool = random_pool(blocks, 2, block, 64, gen)
    tab, at = torch.full((len(lens), -(-max(lens) // block)), -1, dtype=torch.int32), 0
    for s, n in enumerate(lens):
        c = -(-n // block)
        tab[s, :c] = torch.arange(at, at + c)
        at += c
    q = torch.randn(sum(new), 8, 64, generator=gen).to(HALF[t])
    bad = torch.rand(sum(new), 8, generator=gen) < 0.2
    bad[0, 0], bad[-1, -1] = True, False
    ref = attention_ref(q, pool, tab, lens, new, 0, 0.125)
    spoilt = q.clone()
    spoilt[bad] = torch.where(torch.rand(int(bad.sum()), 64, generator=gen) < 0.5, torch.nan, torch.inf).to(q.dtype)
    note(f"attention with bad rows {new} {t}")
    out, lse = _attend(spoilt, pool, tab, lens, new)
    assert bool(torch.isnan(out.cpu()[bad]).all()) and bool(torch.isnan(lse.cpu()[bad]).all())
    good = (~bad).numpy()
    want, wlse, off, loff = ref
    _check(out.cpu()[~bad], lse.cpu()[~bad], (want[good], wlse[good], off[good], loff[good]), "beside bad rows")


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("peaks", [40, 256, 257, 300, 1500, 2048, 2049])
def test_top_k_of_exactly_the_peaks(peaks, t):
    """One large token in each of `peaks` stretches of 64, the rest well below but with weight; top_k is their number,
    one less, one more: where all that was listed is kept, the rest must not be."""
    gen = torch.Generator().manual_seed(80 + peaks)
    vocab = 64 * 2100 - 5
    x = torch.rand(3, vocab, generator=gen)
    for r in range(3):
        at = torch.randperm(vocab // 64, generator=gen)[:peaks] * 64 + torch.randint(0, 64, (peaks,), generator=gen)
        x[r, at] = 4 + 2 * torch.rand(peaks, generator=gen)
    x = x.to({**HALF, "f32": torch.float32}[t])
    for k in (peaks - 1, peaks, peaks + 1):
        for p, m in ((1.0, 0.0), (0.9, 0.0), (1.0, 0.05)):
            for v in (0.0, 0.11, 0.5, 0.77, 0.999):
                u = torch.full((3,), v)
                _check_draw(x, u, 1.3, k, p, m, f"peaks {peaks} k {k} p {p} min_p {m} u {v} {t}")
