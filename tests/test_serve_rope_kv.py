"""Rotary positions and the 8-bit cache's append: values against plain
references in 64 bits (codes: against the stated rule, exactly), and refusals."""

import numpy as np
import pytest
import torch

import dequant_matmul_qmv_amd as mxq
from tests.gpu_util import note
from tests.serve_util import HALF, append_ref, half_step, paging, random_pool, rope_ref

DEV = "cuda:0"
P = 0x10000  # a 16-byte aligned non-null address; never dereferenced (the call is rejected first)


# ------------------------------------------------------------------------------------------------ refusals (CPU)
def _rope(**kw):
    a = dict(q=P, k=P, qo=P, ko=P, f=P, pos=P, tokens=4, heads=2, kv=1, dim=64, rot=64, dtype=mxq.MXQ_F16)
    a.update(kw)
    lib = mxq.load()
    import dequant_matmul_qmv_amd._serve as serve
    serve._load()
    return lib.mxq_rope(a["q"], 128, 64, a["k"], 64, 64, a["qo"], 128, 64, a["ko"], 64, 64, a["f"], a["pos"],
                        a["tokens"], a["heads"], a["kv"], a["dim"], a["rot"], 0, a["dtype"], None)


def test_rope_refusals():
    assert _rope(tokens=-1) == mxq.MXQ_ERR_INVALID_ARG
    assert _rope(rot=-2) == mxq.MXQ_ERR_INVALID_ARG
    assert _rope(dtype=mxq.MXQ_F32) == mxq.MXQ_ERR_UNSUPPORTED
    assert _rope(dim=257) == mxq.MXQ_ERR_UNSUPPORTED
    assert _rope(rot=63) == mxq.MXQ_ERR_UNSUPPORTED
    assert _rope(rot=66) == mxq.MXQ_ERR_UNSUPPORTED
    assert _rope(tokens=2 ** 31) == mxq.MXQ_ERR_UNSUPPORTED
    for name in ("q", "k", "qo", "ko", "f", "pos"):
        assert _rope(**{name: None}) == mxq.MXQ_ERR_INVALID_ARG, name
        assert _rope(**{name: P + 1}) == mxq.MXQ_ERR_MISALIGNED, name
    assert _rope(q=None, k=None, qo=None, ko=None, f=None, pos=None, tokens=0) == mxq.MXQ_OK
    assert _rope(q=None, k=None, qo=None, ko=None, heads=0, kv=0) == mxq.MXQ_OK


def _append(pool=None, null_cache=False, **kw):
    import dequant_matmul_qmv_amd._serve as serve
    lib = serve._load()
    c = dict(k=P, v=P, k_scale=P, v_scale=P, blocks=8, kv_heads=2, block=16, dim=64)
    c.update(pool or {})
    st = None if null_cache else serve._CacheStruct(*[c[n] for n, _ in serve._CacheStruct._fields_])
    a = dict(k=P, v=P, table=P, stride=4, width=4, lens=P, starts=None, tokens=3, seqs=3, dtype=mxq.MXQ_F16)
    a.update(kw)
    return lib.mxq_kv_append(st, a["k"], 128, 64, a["v"], 128, 64, a["table"], a["stride"], a["width"], a["lens"],
                             a["starts"], a["tokens"], a["seqs"], a["dtype"], None)


def test_append_refusals():
    assert _append(null_cache=True) == mxq.MXQ_ERR_INVALID_ARG
    assert _append(dict(blocks=-1)) == mxq.MXQ_ERR_INVALID_ARG
    assert _append(dict(block=48)) == mxq.MXQ_ERR_UNSUPPORTED
    assert _append(dict(block=8)) == mxq.MXQ_ERR_UNSUPPORTED
    assert _append(dict(dim=96)) == mxq.MXQ_ERR_UNSUPPORTED
    assert _append(dict(blocks=2 ** 31)) == mxq.MXQ_ERR_UNSUPPORTED
    for name in ("k", "v", "k_scale", "v_scale"):
        assert _append({name: None}) == mxq.MXQ_ERR_INVALID_ARG, name
        assert _append({name: P + 2}) == mxq.MXQ_ERR_MISALIGNED, name
    assert _append(dict(k=P + 8)) == mxq.MXQ_ERR_MISALIGNED
    assert _append(dtype=mxq.MXQ_F32) == mxq.MXQ_ERR_UNSUPPORTED
    assert _append(tokens=4) == mxq.MXQ_ERR_INVALID_ARG              # no starts: one token a sequence
    assert _append(tokens=-1, starts=P) == mxq.MXQ_ERR_INVALID_ARG
    assert _append(width=2 ** 27, stride=2 ** 27) == mxq.MXQ_ERR_UNSUPPORTED
    assert _append(stride=3) == mxq.MXQ_ERR_INVALID_ARG
    for name in ("k", "v", "table", "lens"):
        assert _append(**{name: None}) == mxq.MXQ_ERR_INVALID_ARG, name
        assert _append(**{name: P + 1}) == mxq.MXQ_ERR_MISALIGNED, name
    assert _append(k=None, v=None, table=None, lens=None, tokens=0, seqs=0) == mxq.MXQ_OK
    assert _append(dict(blocks=0, k=None, v=None, k_scale=None, v_scale=None)) == mxq.MXQ_OK


def test_tensor_refusals_on_the_cpu():
    """Host tensors, and shapes that do not fit, never reach the library."""
    x = torch.zeros(2, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="device tensor"):
        mxq.mxq_rope(x, x, torch.zeros(32), torch.zeros(2, dtype=torch.int32))
    pool = [t for t in random_pool(4, 2, 16, 64, torch.Generator().manual_seed(0))]
    with pytest.raises(ValueError, match="device tensor"):
        mxq.KvCache(*pool)
    with pytest.raises(ValueError, match="v must be"):
        mxq.KvCache(pool[0], pool[1].transpose(2, 3), pool[2], pool[3])
    with pytest.raises(TypeError, match="int8"):
        mxq.KvCache(pool[0].float(), *pool[1:])
    with pytest.raises(ValueError, match="k_scale"):
        mxq.KvCache(pool[0], pool[1], pool[2][:2], pool[3])


# ------------------------------------------------------------------------------------------------ rotary positions
# f32 arithmetic of a pair: the angle within half a turn rounds to 2^-26 turns (9.4e-8 rad), sine and cosine are
# within 2 units of 2^-24, two products and a sum round by 2^-24 each: under 2^-21 (|a| + |b|).
ROPE_F32 = 2.0 ** -21


def _check_rope(got, x, inv_freq, pos, interleaved, what):
    ref = rope_ref(x, inv_freq, pos, interleaved)
    rot = 2 * inv_freq.shape[0]
    xs = np.abs(x.double().cpu().numpy())
    pair = np.zeros_like(xs)
    if rot:
        if interleaved:
            pair[..., :rot] = np.repeat(xs[..., 0:rot:2] + xs[..., 1:rot:2], 2, -1)
        else:
            pair[..., :rot] = np.concatenate([xs[..., :rot // 2] + xs[..., rot // 2:rot]] * 2, -1)
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 2.0 ** -134   # half of the smallest subnormal step
    bound = ROPE_F32 * pair + half_step(x.dtype) * (np.abs(ref) + ROPE_F32 * pair) + tiny
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= bound), (what, float((err / bound).max()))
    assert np.array_equal(got[..., rot:].cpu().view(torch.int16).numpy(), x[..., rot:].cpu().view(torch.int16).numpy()), what


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot,heads,kv_heads,tokens", [
    (64, 64, 32, 8, 1), (128, 64, 8, 1, 37), (128, 32, 10, 2, 9), (64, 16, 1, 1, 130), (64, 0, 2, 1, 3),
    (80, 40, 3, 3, 5), (100, 6, 2, 1, 4), (256, 256, 2, 1, 3), (7, 2, 3, 1, 5)])
def test_rope_values(t, interleaved, dim, rot, heads, kv_heads, tokens):
    gen = torch.Generator().manual_seed(dim * 1000 + rot + tokens)
    n = (heads + 2 * kv_heads) * dim
    qkv = torch.randn(tokens, n, generator=gen).to(HALF[t]).to(DEV)
    q = qkv[:, :heads * dim].view(tokens, heads, dim)
    k = qkv[:, heads * dim:(heads + kv_heads) * dim].view(tokens, kv_heads, dim)
    pos = torch.randint(0, 131072, (tokens,), generator=gen).to(torch.int32).to(DEV)
    inv = (500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().to(DEV)
    before = qkv.clone()
    note(f"rope {t} interleaved={interleaved} dim={dim} rot={rot} heads={heads}/{kv_heads} tokens={tokens}")
    yq, yk = mxq.mxq_rope(q, k, inv, pos, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(qkv.view(torch.int16), before.view(torch.int16))
    _check_rope(yq, q, inv, pos, interleaved, "q")
    _check_rope(yk, k, inv, pos, interleaved, "k")
    # in place, in the fused projection's memory: the same bits, and nothing else touched
    mxq.mxq_rope(q, k, inv, pos, q, k, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(q.contiguous().view(torch.int16), yq.view(torch.int16))
    assert torch.equal(k.contiguous().view(torch.int16), yk.view(torch.int16))
    rest = (heads + kv_heads) * dim
    assert torch.equal(qkv[:, rest:].contiguous().view(torch.int16), before[:, rest:].contiguous().view(torch.int16))


@pytest.mark.gpu
def test_rope_layouts():
    """Transposed heads, one token broadcast over many, an odd base address, q alone, no tokens, far and negative positions."""
    gen = torch.Generator().manual_seed(5)
    inv = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().to(DEV)
    pos = torch.tensor([0, 1, 2 ** 30, 2 ** 31 - 1, -7], dtype=torch.int32, device=DEV)
    base = torch.randn(4, 5, 64, generator=gen).half().to(DEV)
    note("rope layouts")
    q = base.transpose(0, 1)                                          # [tokens, heads, dim] by strides
    yq, none = mxq.mxq_rope(q, None, inv, pos)
    assert none is None
    one = base[:1].expand(5, 5, 64)                                   # token stride 0
    yo, _ = mxq.mxq_rope(one, None, inv, pos)
    flat = torch.randn(5 * 2 * 64 + 1, generator=gen).bfloat16().to(DEV)
    odd = flat[1:].view(5, 2, 64)                                     # 2-byte aligned rows
    yd, _ = mxq.mxq_rope(odd, None, inv, pos)
    empty, _ = mxq.mxq_rope(base[:0], None, inv, pos[:0])
    torch.cuda.synchronize()
    _check_rope(yq, q, inv, pos, False, "transposed")
    _check_rope(yo, one, inv, pos, False, "broadcast")
    _check_rope(yd, odd, inv, pos, False, "odd base")
    assert empty.shape == (0, 5, 64)


# ------------------------------------------------------------------------------------------------ append
def _run_append(lens, new, kv_heads, block, dim, t, seed, spread=1.0, table=None, use_starts=True):
    gen = torch.Generator().manual_seed(seed)
    blocks, tab = paging(lens, block, gen)
    if table is not None:
        tab = table(tab)
    pool = random_pool(blocks, kv_heads, block, dim, gen)
    n = sum(new)
    kv = (torch.randn(n, 2, kv_heads, dim, generator=gen) * spread).to(HALF[t])
    k, v = kv[:, 0], kv[:, 1]
    want = append_ref(pool, k, v, tab, lens, new, block)
    cache = mxq.KvCache(*[x.to(DEV) for x in pool])
    kvd = kv.to(DEV)
    starts = None
    if use_starts:
        starts = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=DEV)
    note(f"append lens={lens[:6]} new={new[:6]} kv_heads={kv_heads} block={block} dim={dim} {t}")
    got = mxq.mxq_kv_append(cache, kvd[:, 0], kvd[:, 1], tab.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), starts)
    torch.cuda.synchronize()
    assert got is cache
    for name, g, w in zip(("k", "v", "k_scale", "v_scale"), (got.k, got.v, got.k_scale, got.v_scale), want):
        g = g.cpu().numpy()
        assert np.array_equal(g.view(np.uint8), w.view(np.uint8)), (name, np.argwhere(g != w)[:5], int((g != w).sum()))


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("block,dim", [(16, 64), (32, 128), (64, 64), (128, 128)])
@pytest.mark.parametrize("spread", [0.1, 1.0, 3.0])   # under the held scale, about it, over it
def test_append_one_token(block, dim, t, spread):
    lens = [1, 2, block, block + 1, 3 * block - 1, 200, 17, 16]
    _run_append(lens, [1] * len(lens), 3, block, dim, t, 11, spread, use_starts=False)


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("block,dim", [(16, 128), (32, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("spread", [0.1, 3.0])
def test_append_chunks(block, dim, t, spread):
    lens = [5 * block + 3, block, 0, 77, 2 * block, 300, 9]
    new = [4 * block + 5, block, 0, 77, 1, 0, 3]
    _run_append(lens, new, 2, block, dim, t, 13, spread)


@pytest.mark.gpu
def test_append_many_sequences():
    """More sequences than a wave has lanes, some without new tokens."""
    lens = [(7 * i) % 90 for i in range(150)]
    new = [min(n, (5 * i) % 23) for i, n in enumerate(lens)]
    _run_append(lens, new, 1, 16, 64, "bf16", 17)


@pytest.mark.gpu
def test_append_zeros_and_places_missing():
    """All-zero tokens (scale 0), f16's smallest and largest values, and tokens whose page does not exist."""
    _run_append([20, 40], [20, 8], 2, 16, 64, "f16", 19, spread=0.0)
    _run_append([20, 40], [20, 8], 2, 16, 64, "f16", 19, spread=1e-8)
    _run_append([20, 40], [20, 8], 2, 16, 64, "bf16", 19, spread=1e-37)

    def spoil(tab):
        tab[0, 1] = -1
        tab[1, 2] = 10 ** 6
        return tab
    _run_append([60, 60], [60, 30], 2, 16, 64, "f16", 23, table=spoil)
    _run_append([60, 60], [60, 50], 2, 16, 64, "f16", 23, table=lambda tab: tab[:, :2].contiguous())


# ------------------------------------------------------------------------------------------------ larger than the L2s
@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_beyond_the_caches(interleaved, t):
    """More bytes than the L2s hold, out of a fused projection and in place; more units a token than are loaded ahead."""
    gen = torch.Generator().manual_seed(51)
    n, heads, kv_heads, dim, half = 1100, 28, 4, 256, 48
    base = torch.randn(n, (heads + 2 * kv_heads) * dim, generator=gen).to(HALF[t])
    qkv = base.to(DEV)
    q = qkv[:, :heads * dim].view(n, heads, dim)
    k = qkv[:, heads * dim:(heads + kv_heads) * dim].view(n, kv_heads, dim)
    f = (10000.0 ** (-torch.arange(half) / half)).float().to(DEV)
    pos = torch.randint(0, 131072, (n,), generator=gen, dtype=torch.int32).to(DEV)
    note(f"rope beyond the caches interleaved={interleaved} {t}")
    q2, k2 = mxq.mxq_rope(q, k, f, pos, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(qkv.cpu(), base)
    _check_rope(q2, q, f, pos, interleaved, "q")
    _check_rope(k2, k, f, pos, interleaved, "k")
    mxq.mxq_rope(q, k, f, pos, q, k, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(k, k2)
    assert torch.equal(qkv[:, (heads + kv_heads) * dim:].cpu(), base[:, (heads + kv_heads) * dim:])
