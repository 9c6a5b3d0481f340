"""Keys normed, rotated and quantized into the caches of 8 and 4 bits, queries beside them: codes and scales against the
stated rules bit for bit, queries against the definition, and refusals."""

import numpy as np
import pytest
import torch

import dequant_matmul_qmv_amd as mxq
from tests.gpu_util import note
from tests.serve4_util import HALF, append4_ref, frequencies, pack, quantize4, random_pool4, rotated_bits, unpack, values4
from tests.serve_util import append_ref, paging, random_pool

DEV = "cuda:0"
P = 0x10000


# ----------------------------------------------------------------------------------------------- CPU
def test_quantized_values_are_near_and_exact_in_f16():
    """A code's value is at most half a scale from what it stands for, and a number of f16; 0 stays 0."""
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(400, 64, generator=gen) * torch.exp(3 * torch.randn(400, 1, generator=gen))
    x[0], x[1], x[2], x[3] = 0, 5.0, -7.0, 1e-9
    x[4] = 6e4
    x[5, ::2] = 0
    x = x.half()
    codes, words = quantize4(x)
    scale, zero = (words & 0x7FF0).view(np.float16).astype(np.float64)[:, None], (words & 15).astype(np.float64)[:, None]
    y = (codes - zero) * scale
    assert np.array_equal(y, y.astype(np.float16).astype(np.float64))
    assert np.all(np.abs(y - x.double().numpy()) <= scale * (0.5 + 1e-5))
    assert np.all(y[x.numpy() == 0] == 0) and not codes[0].any() and words[0] == 0
    assert np.array_equal(unpack(pack(codes)), codes)
    hand, word = quantize4(torch.tensor([[-1.0, 0.0, 0.5, 2.0, 2.75, 0.1, 0.124, 0.126]]))
    # range 3.75: scale 0.25, zero 4
    assert word[0] == (np.array([0.25], np.float16).view(np.uint16)[0] | 4)
    assert hand.tolist() == [[0, 4, 6, 12, 15, 4, 4, 5]]


def _rotation(**kw):
    from tests.test_serve_norm_rope import _rotation as make
    return make(**kw)


def _call(bits, rotation="default", cache="default", **kw):
    import dequant_matmul_qmv_amd._serve as serve
    c = dict(k=P, v=P, ks=P, vs=P, blocks=4, kv=2, block=16, dim=64)
    a = dict(q=P, qo=P, kx=P, vx=P, heads=4, dtype=mxq.MXQ_F16, table=P, stride=3, width=3, lens=P, starts=None, tokens=2, seqs=2)
    c.update({n: v for n, v in kw.items() if n in c})
    a.update({n: v for n, v in kw.items() if n in a})
    st = serve._CacheStruct(c["k"], c["v"], c["ks"], c["vs"], c["blocks"], c["kv"], c["block"], c["dim"]) if cache == "default" else cache
    r = _rotation(**kw["rot"]) if "rot" in kw else _rotation() if rotation == "default" else rotation
    lib = serve._load()
    f = lib.mxq_rope_append if bits == 8 else lib.mxq_rope_append4
    return f(st, a["q"], 256, 64, a["qo"], 256, 64, a["kx"], 128, 64, a["vx"], 128, 64, r, a["table"], a["stride"], a["width"], a["lens"],
             a["starts"], a["tokens"], a["seqs"], a["heads"], a["dtype"], None)


@pytest.mark.parametrize("bits", [8, 4])
def test_refusals(bits):
    bad, unsup, mis = mxq.MXQ_ERR_INVALID_ARG, mxq.MXQ_ERR_UNSUPPORTED, mxq.MXQ_ERR_MISALIGNED
    assert _call(bits, cache=None) == bad
    for name in ("blocks", "kv", "tokens", "seqs", "width", "heads"):
        assert _call(bits, **{name: -1}) == bad, name
    for name in ("k", "v", "ks", "vs", "q", "qo", "kx", "vx", "table", "lens"):
        assert _call(bits, **{name: None}) == bad, name
    assert _call(bits, tokens=3) == bad                       # without starts
    assert _call(bits, stride=2) == bad
    assert _call(bits, rot=dict(eps=-1.0)) == bad and _call(bits, rot=dict(axes=0)) == bad
    assert _call(bits, rot=dict(inv_freq=None)) == bad
    assert _call(bits, rot=dict(axes=2, stride=1)) == bad
    assert _call(bits, rotation=None) == bad                  # query heads to turn
    assert _call(8, rotation=None, heads=0) == bad
    for kw in (dict(block=48), dict(dim=96), dict(dim=256), dict(heads=3), dict(heads=65536 * 2), dict(dtype=mxq.MXQ_F32),
               dict(blocks=2 ** 31), dict(kv=65536, heads=0), dict(width=2 ** 27, stride=2 ** 27), dict(rot=dict(rot=66)),
               dict(rot=dict(rot=7)), dict(rot=dict(qw=P, wtype=mxq.MXQ_BF16))):
        assert _call(bits, **kw) == unsup, kw
    for name, at in (("k", 8), ("v", 8), ("q", 1), ("qo", 1), ("kx", 1), ("vx", 1), ("table", 2), ("lens", 2), ("starts", 2)):
        assert _call(bits, **{name: P + at}) == mis, name
    for name in ("ks", "vs"):
        assert _call(bits, **{name: P + (2 if bits == 8 else 8)}) == mis, name
    assert _call(bits, rot=dict(positions=P + 2)) == mis and _call(bits, rot=dict(kw=P + 2)) == mis
    ok = dict(q=None, qo=None, kx=None, vx=None, table=None, lens=None)
    assert _call(bits, tokens=0, seqs=0, **ok) == mxq.MXQ_OK
    assert _call(bits, heads=0, width=0, **{n: v for n, v in ok.items() if n != "lens"}) == mxq.MXQ_OK
    assert _call(bits, heads=0, blocks=0, k=None, v=None, ks=None, vs=None, **{n: v for n, v in ok.items() if n not in ("lens", "table")}) == mxq.MXQ_OK


@pytest.mark.parametrize("bits,tokens,seqs", [(4, 2 ** 31 - 1, 1), (4, 80000000, 1), (4, 2, 2 ** 31 - 1), (4, 2, 2 ** 30),
                                              (8, 2 ** 31 - 1, 1), (8, 2, 2 ** 31 - 1), (8, 2, 2 ** 30)])
def test_refusals_of_grids(bits, tokens, seqs):
    """A launch of 2^32 threads or more is refused by name before anything is enqueued."""
    assert _call(bits, tokens=tokens, seqs=seqs, starts=P) == mxq.MXQ_ERR_UNSUPPORTED


def test_cache_refusals_without_a_gpu():
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t)  # noqa: E731
    with pytest.raises(TypeError):
        mxq.KvCache4(z(2, 1, 16, 8, t=torch.int8), z(2, 1, 2, 64), z(2, 1, 16, t=torch.int16), z(2, 1, 16, t=torch.int16))
    with pytest.raises(ValueError, match="v must be"):
        mxq.KvCache4(z(2, 1, 16, 8), z(2, 1, 16, 64), z(2, 1, 16, t=torch.int16), z(2, 1, 16, t=torch.int16))
    with pytest.raises(ValueError, match="k_scale"):
        mxq.KvCache4(z(2, 1, 16, 8), z(2, 1, 2, 64), z(2, 1, t=torch.int16), z(2, 1, 16, t=torch.int16))
    with pytest.raises(ValueError, match="device tensor"):
        mxq.KvCache4(z(2, 1, 16, 8), z(2, 1, 2, 64), z(2, 1, 16, t=torch.int16), z(2, 1, 16, t=torch.int16))


# ----------------------------------------------------------------------------------------------- GPU
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cache(pool):
    return (mxq.KvCache4 if pool[0].dtype == torch.int32 else mxq.KvCache)(*[x.to(DEV) for x in pool])


def _tensors(cache):
    return [t.cpu() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]


def _places(lens, new):
    return torch.cat([torch.arange(max(a, 0) - n, max(a, 0)) for a, n in zip(lens, new)] + [torch.zeros(0, dtype=torch.int64)]).int()


class Problem:
    """q, k, v as views of a fused projection, a pool with older tokens, and what has to come out."""

    def __init__(self, bits, dim, block, t, lens, new, seed, heads=4, kv=2, rot=None, inter=False, norm=True, f32=False, axes=0, implied=True,
                 spread=1.0, extra=0):
        gen = torch.Generator().manual_seed(seed)
        rot = dim if rot is None else rot
        n = sum(new) + extra
        self.bits, self.lens, self.new, self.block, self.inter, self.heads, self.kv, self.dim = bits, lens, new, block, inter, heads, kv, dim
        qkv = (torch.randn(n, (heads + 2 * kv) * dim, generator=gen) * torch.exp(spread * torch.randn(n, 1, generator=gen))).to(HALF[t])
        self.qkv = qkv
        self.q, self.k, self.v = self.views(qkv)
        blocks, self.table = paging([max(x, 0) for x in lens], block, gen)
        self.pool = random_pool4(blocks, kv, block, dim, gen) if bits == 4 else random_pool(blocks, kv, block, dim, gen)
        self.f = frequencies(rot) if rot else torch.zeros(0)
        place = _places(lens, new)
        place = torch.cat((place, torch.zeros(extra, dtype=torch.int32)))
        self.axes, self.positions = None, None
        if axes:
            self.axes = (torch.arange(rot // 2) % axes).int()
            self.positions = torch.stack([place * (i + 1) + 17 * i for i in range(axes)]).int().contiguous()
        elif not implied:
            self.positions = torch.randint(0, 100000, (n,), generator=gen, dtype=torch.int32)
        self.w = [None, None]
        if norm:
            self.w = [(1 + 0.3 * torch.randn(dim, generator=gen)).to(torch.float32 if f32 else HALF[t]) for _ in range(2)]
        at = place if self.positions is None else self.positions
        self.want_q = rotated_bits(self.q, self.w[0], 1e-6, self.f, at, self.axes, inter) if heads else None
        self.held = rotated_bits(self.k, self.w[1], 1e-6, self.f, at, self.axes, inter)
        m = sum(new)
        if bits == 4:
            self.want = append4_ref(self.pool, self.held[:m], self.v[:m], self.table, lens, new, block)
        else:
            self.want = append_ref(self.pool, self.held[:m], self.v[:m], self.table, [max(x, 0) for x in lens], new, block)

    def views(self, qkv):
        n, h, kv, d = qkv.shape[0], self.heads, self.kv, self.dim
        return (qkv[:, :h * d].view(n, h, d), qkv[:, h * d:(h + kv) * d].view(n, kv, d), qkv[:, (h + kv) * d:].view(n, kv, d))

    def call(self, one=False, q_out=None, q="own", cache=None, **kw):
        dev = lambda x: None if x is None else x.to(DEV)  # noqa: E731
        cache = _cache(self.pool) if cache is None else cache
        q, k, v = self.views(self.qkv.to(DEV)) if q == "own" else q
        starts = None if one else _i32(np.cumsum([0] + self.new).tolist())
        got = mxq.mxq_rope_append(cache, q if self.heads else None, k, v, dev(self.f), dev(self.table), _i32(self.lens), starts,
                                  dev(self.w[0]), dev(self.w[1]), q_out, positions=dev(self.positions), axes=dev(self.axes),
                                  interleaved=self.inter, **kw)
        return got, cache

    def check(self, got, cache, what):
        torch.cuda.synchronize()
        for name, a, b in zip(("k", "v", "k_scale", "v_scale"), _tensors(cache), self.want):
            a = a.numpy().view(b.dtype)
            assert np.array_equal(a, b), (what, name, int((a != b).sum()))
        if self.heads:
            m = sum(self.new)
            assert torch.equal(got.cpu()[:m].view(torch.int16), self.want_q[:m].view(torch.int16)), (what, "q")


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dim,block", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 64), (128, 128)])
def test_single_tokens(dim, block, bits, t):
    """One new token a sequence: first tokens of pages and sequences, pages partly filled, scales that grow or stay."""
    lens = [1, 2, 15, 16, 17, 33, 64, 65, 127, 128, 129, 200]
    for kw in (dict(), dict(rot=dim // 2, inter=True, implied=False), dict(heads=0, norm=False), dict(heads=8, kv=1, f32=True, axes=3),
               dict(heads=10, kv=2, rot=20), dict(heads=3, kv=3, rot=0), dict(heads=32, kv=2, rot=16, implied=False, spread=2.0)):
        p = Problem(bits, dim, block, t, lens, [1] * len(lens), dim + block, **kw)
        note(f"rope_append one, {bits} bits, dim {dim}, block {block}, {t}, {kw}")
        p.check(*p.call(one=True), f"one {kw}")
        note("the same with starts")
        p.check(*p.call(), f"one with starts {kw}")


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dim,block", [(64, 16), (64, 32), (64, 128), (128, 16), (128, 64), (128, 128)])
def test_many_tokens(dim, block, bits, t):
    """Chunks that start and end inside pages and words of 8 tokens, sequences without new tokens, whole prompts."""
    lens, new = [1, 7, 8, 9, 40, 0, 130, 300, 20], [1, 3, 8, 2, 33, 0, 0, 171, 20]
    for kw in (dict(), dict(rot=dim // 4, inter=True), dict(heads=0, norm=False, rot=0), dict(heads=6, kv=3, axes=2, f32=True),
               dict(heads=5, kv=1, rot=36, implied=False, spread=2.0)):
        p = Problem(bits, dim, block, t, lens, new, dim + block + 1, **kw)
        note(f"rope_append many, {bits} bits, dim {dim}, block {block}, {t}, {kw}")
        p.check(*p.call(), f"many {kw}")


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
def test_many_heads(bits):
    """More kv heads than a workgroup takes at a time."""
    for heads, kv, dim in ((42, 21, 64), (19, 19, 128), (32, 16, 128)):
        p = Problem(bits, dim, 32, "f16", [50, 3, 11], [37, 3, 5], heads + dim, heads=heads, kv=kv)
        note(f"rope_append {heads}/{kv} heads, {bits} bits")
        p.check(*p.call(), "heads")
        p = Problem(bits, dim, 32, "f16", [50, 3, 11], [1, 1, 1], heads + dim, heads=heads, kv=kv)
        p.check(*p.call(one=True), "heads, one token")


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("one", [False, True])
def test_tokens_without_a_place(bits, one):
    """Pages that are missing, lengths past the table, more new tokens than the length, negative lengths: keys are dropped,
    queries are turned all the same."""
    lens = [40, 100, 20, -5, 7, 65, 0]
    new = [1] * 7 if one else [40, 37, 30, 3, 7, 9, 2]
    p = Problem(bits, 64, 16, "f16", lens, new, 5)
    p.table[0, 1], p.table[0, 2] = -1, p.pool[0].shape[0]     # no page, a page that is not there
    p.table = p.table[:, :5].contiguous()                     # positions from 80 on have none
    if bits == 4:
        p.want = append4_ref(p.pool, p.held, p.v, p.table, lens, new, 16)
    else:
        # (a sequence's rows without a place, taken off by hand)
        k, v, at, l2, n2, rows = p.held, p.v, 0, [], [], []
        for length, n in zip(lens, new):
            keep = [at + i for i in range(n) if 0 <= max(length, 0) - n + i < 80]
            rows += keep
            l2.append(min(max(length, 0), 80))
            n2.append(len(keep))
            at += n
        p.want = append_ref(p.pool, k[rows], v[rows], p.table, l2, n2, 16)
    note(f"rope_append without places, {bits} bits, one={one}")
    p.check(*p.call(one=one), "without places")


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
def test_rows_behind_the_last_sequence(bits):
    p = Problem(bits, 128, 32, "bf16", [50, 9], [33, 4], 6, extra=21)
    q_out = torch.full((58, 4, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    note("rope_append, rows behind")
    got, cache = p.call(q_out=q_out)
    p.check(got, cache, "behind")
    assert got.data_ptr() == q_out.data_ptr() and (q_out[37:] == 9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("new", [1, 19])
def test_in_place_odd_rows_and_streams(bits, new):
    p = Problem(bits, 128, 32, "f16", [50, 29, 70], [new] * 3, 7, heads=8, kv=2)
    dev = p.qkv.to(DEV)
    views = p.views(dev)
    note("rope_append in place")
    got, cache = p.call(one=new == 1, q=views, q_out=views[0])
    p.check(got, cache, "in place")
    assert torch.equal(dev[:, 8 * 128:].cpu(), p.qkv[:, 8 * 128:])
    note("rope_append, rows that are not 16-byte aligned")
    odd = torch.zeros(p.qkv.shape[0], p.qkv.shape[1] + 3, dtype=torch.float16, device=DEV)
    odd[:, 1:-2] = p.qkv.to(DEV)
    out = torch.full((8, 3 * new, 131), 5.0, dtype=torch.float16, device=DEV)
    views = tuple(odd[:, 1 + i * 128:1 + j * 128].unflatten(1, (j - i, 128)) for i, j in ((0, 8), (8, 10), (10, 12)))
    got, cache = p.call(one=new == 1, q=views, q_out=out.transpose(0, 1)[:, :, 1:129])
    p.check(got, cache, "odd rows")
    assert (out[:, :, 0] == 5).all() and (out[:, :, 129:] == 5).all()
    note("rope_append on another stream")
    side = torch.cuda.Stream()
    cache, views = _cache(p.pool), p.views(p.qkv.to(DEV))
    args = [x.to(DEV) for x in (p.f, p.table, p.w[0], p.w[1])]
    lens, starts = _i32(p.lens), None if new == 1 else _i32(np.cumsum([0] + p.new).tolist())
    torch.cuda.synchronize()
    got = mxq.mxq_rope_append(cache, *views, args[0], args[1], lens, starts, args[2], args[3], stream=side)
    side.synchronize()
    p.check(got, cache, "stream")


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("new", [1, 45])
def test_one_after_the_other(bits, new):
    """The launch's codes and queries are those of a norm and rotation into memory and an append of it."""
    for kw in (dict(), dict(rot=32, inter=True, axes=3), dict(norm=False, implied=False)):
        p = Problem(bits, 64, 64, "bf16", [61, 100, 45], [new] * 3, 8, **kw)
        got, cache = p.call(one=new == 1)
        at = p.positions if p.positions is not None else _places(p.lens, p.new)
        q, k, v = p.views(p.qkv.to(DEV))
        dev = lambda x: None if x is None else x.to(DEV)  # noqa: E731
        q2, k2 = mxq.mxq_norm_rope(q, k, dev(p.f), dev(at), dev(p.w[0]), dev(p.w[1]), axes=dev(p.axes), interleaved=p.inter)
        other = mxq.mxq_kv_append(_cache(p.pool), k2, v, p.table.to(DEV), _i32(p.lens), None if new == 1 else _i32([0, new, 2 * new, 3 * new]))
        torch.cuda.synchronize()
        assert torch.equal(got, q2)
        assert all(torch.equal(a, b) for a, b in zip(_tensors(cache), _tensors(other)))


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_values_of_4_bits(t):
    """Rows of zeros, of one value, of the type's largest and smallest values, all positive, all negative; ties."""
    gen = torch.Generator().manual_seed(9)
    n, dim = 24, 64
    big, small = torch.finfo(HALF[t]).max, torch.finfo(HALF[t]).smallest_normal
    x = torch.randn(n, 1, dim, generator=gen)
    x[0], x[1], x[2] = 0, 3.0, -3.0
    x[3], x[4], x[5] = big, -big, small / 4
    x[6, :, ::2] = big
    x[7, :, ::2] = -big
    x[8], x[9] = x[8].abs() + 1, -x[9].abs() - 1
    x[10] *= small
    x[11] *= 1e-5
    x[12] *= 1e3
    x[13] = torch.arange(dim) % 16 - 7.0                      # scale 1: codes are the numbers
    x[14] = (torch.arange(dim) % 31) / 2 - 7.0                # ties between codes
    x[15, :, 5] = 60960.0
    x[16, :, 5] = -60960.0
    x[17] = 2.0 ** -20 * (torch.arange(dim) % 16)
    x = x.to(HALF[t])
    lens, new = [n + 5], [n]
    table = torch.tensor([[1, 0, 2]], dtype=torch.int32)
    pool = random_pool4(3, 1, 16, dim, gen)
    want = append4_ref(pool, x, x.flip(0), table, lens, new, 16)
    for one in (False, True):
        cache = _cache(pool)
        note(f"append of extreme values, one={one}")
        xd, vd = x.to(DEV), x.flip(0).to(DEV)
        if one:
            for i in range(n):
                mxq.mxq_kv_append(cache, xd[i:i + 1], vd[i:i + 1], table.to(DEV), _i32([6 + i]))
        else:
            mxq.mxq_kv_append(cache, xd, vd, table.to(DEV), _i32(lens), _i32([0, n]))
        torch.cuda.synchronize()
        for name, a, b in zip(("k", "v", "k_scale", "v_scale"), _tensors(cache), want):
            assert np.array_equal(a.numpy().view(b.dtype), b), (name, one)
    k, _ = values4(_tensors(cache))
    got = np.concatenate([k[1, 0], k[0, 0]])[5 + 13]
    assert np.array_equal(got, x[13, 0].double().numpy())


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [1, -1])
def test_every_scale_of_4_bits(sign):
    """Heads whose range is 15 times each scale there is, f16's values: the smallest steps, all mantissas and exponents.
    Their other values lie at and beside the middles between codes, where an inverse a step off would show."""
    dim, block = 64, 128
    scales = torch.cat([torch.arange(1, 64) * 2.0 ** -20] + [torch.arange(64, 128) * 2.0 ** e for e in range(-20, 6)]).double()
    scales = scales[scales <= 4064]
    middle = (torch.arange(dim) % 15 + 0.5).double()
    middle[15:30] *= 1 - 2.0 ** -11
    middle[30:45] *= 1 + 2.0 ** -11
    x = (scales[:, None] * middle).half()
    x[:, -1] = (15 * scales).half()                             # 11 bits at most: exact
    assert torch.equal(x[:, -1].double(), 15 * scales) and float(x.max()) < 65504
    x = sign * x[:, None]
    n = x.shape[0]
    blocks = -(-n // block)
    table = torch.arange(blocks, dtype=torch.int32)[None]
    pool = random_pool4(blocks, 1, block, dim, torch.Generator().manual_seed(2))
    want = append4_ref(pool, x, x.flip(0), table, [n], [n], block)
    cache = _cache(pool)
    mxq.mxq_kv_append(cache, x.to(DEV), x.flip(0).to(DEV), table.to(DEV), _i32([n]), _i32([0, n]))
    torch.cuda.synchronize()
    for name, a, b in zip(("k", "v", "k_scale", "v_scale"), _tensors(cache), want):
        assert np.array_equal(a.numpy().view(b.dtype), b), name
    held = _tensors(cache)[2].numpy().view(np.uint16).reshape(-1)[:n] & 0xFFF0
    assert np.array_equal(held.view(np.float16).astype(np.float64), scales.numpy())


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("new", [1, 70])
def test_the_longest_sequence(bits, new):
    """Positions near 2^31 in a table as wide as is allowed."""
    block, dim = 64, 64
    width, last = (2 ** 31 - 1) // block, 3
    p = Problem(bits, dim, block, "f16", [last * block - 5], [new], 18, heads=2, kv=2, norm=False, implied=False)
    tab = torch.zeros(1, width, dtype=torch.int32)
    tab[0, -last:] = p.table[0, :last]
    note(f"rope_append of {new} at {width * block - 5}")
    cache, views = _cache(p.pool), p.views(p.qkv.to(DEV))
    got = mxq.mxq_rope_append(cache, *views, p.f.to(DEV), tab.to(DEV), _i32([width * block - 5]), None if new == 1 else _i32([0, new]),
                              positions=p.positions.to(DEV))
    p.check(got, cache, "longest")


@pytest.mark.gpu
def test_no_pages_at_all():
    """A cache of no pages, a table of none: queries are turned, nothing else happens."""
    for bits in (8, 4):
        for new in ([1, 1], [5, 3]):
            p = Problem(bits, 64, 16, "f16", [30, 9], new, 19)
            empty = (mxq.KvCache4 if bits == 4 else mxq.KvCache).empty(0, 2, 16, 64, DEV)
            note(f"rope_append without pages, {bits} bits, {new}")
            got, _ = p.call(one=new == [1, 1], cache=empty)
            torch.cuda.synchronize()
            assert torch.equal(got.cpu(), p.want_q)
            cache = _cache(p.pool)
            views = p.views(p.qkv.to(DEV))
            got = mxq.mxq_rope_append(cache, *views, p.f.to(DEV), torch.zeros(2, 0, dtype=torch.int32, device=DEV), _i32([30, 9]),
                                      None if new == [1, 1] else _i32([0, 5, 8]), p.w[0].to(DEV), p.w[1].to(DEV))
            torch.cuda.synchronize()
            assert torch.equal(got.cpu(), p.want_q)
            assert all(torch.equal(a, b) for a, b in zip(_tensors(cache), p.pool))


@pytest.mark.gpu
def test_python_refusals():
    p = Problem(4, 64, 16, "f16", [30, 9], [1, 1], 20)
    cache, (q, k, v) = _cache(p.pool), p.views(p.qkv.to(DEV))
    f, tab, lens, w = p.f.to(DEV), p.table.to(DEV), _i32(p.lens), p.w[0].to(DEV)
    pos = _i32([3, 4])
    for args, kw in (((cache, q, k.float(), v, f, tab, lens), {}), ((cache, q, k, v[:1], f, tab, lens), {}), ((cache, q[:1], k, v, f, tab, lens), {}),
                     ((cache, q, k[:, :1], v[:, :1], f, tab, lens), {}), ((cache, q.bfloat16(), k, v, f, tab, lens), {}),
                     ((cache, q[:, :3], k, v, f, tab, lens), {}), ((cache, q, k, v, f.half(), tab, lens), {}),
                     ((cache, q, k, v, f, tab.long(), lens), {}), ((cache, q, k, v, f, tab, lens[:1]), {}),
                     ((cache, q, k, v, f, tab, lens, _i32([0, 2])), {}), ((cache, q, k, v, f, tab, lens), dict(axes=_i32([0] * 32))),
                     ((cache, q, k, v, f, tab, lens), dict(positions=pos[:1])), ((cache, q, k, v, f, tab, lens), dict(positions=torch.stack((pos, pos)))),
                     ((cache, None, k, v, f, tab, lens, None, None, w, q), {}), ((cache, q, k, v, f, tab, lens, None, w[:32]), {}),
                     ((cache, q.cpu(), k, v, f, tab, lens), {}), ((cache, q, k, v, f, tab, lens, None, None, None, q[:, :2]), {})):
        with pytest.raises((TypeError, ValueError, mxq.MxqError)):
            mxq.mxq_rope_append(*args, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("new", [1, 13])
def test_graph_replay(bits, new):
    """Captured steps with lengths that change between the replays, eager calls on another cache beside them."""
    p = Problem(bits, 64, 16, "f16", [30, 9, 41], [new] * 3, 21, heads=4, kv=2)
    blocks = 40
    gen = torch.Generator().manual_seed(3)
    table = torch.randperm(36, generator=gen).view(3, 12).int().to(DEV)
    a, b = ((mxq.KvCache4 if bits == 4 else mxq.KvCache).empty(blocks, 2, 16, 64, DEV) for _ in range(2))
    dev, lens = p.qkv.to(DEV), _i32([new, new + 1, new + 2])
    starts = None if new == 1 else _i32([0, new, 2 * new, 3 * new])
    f, w = p.f.to(DEV), [x.to(DEV) for x in p.w]
    out = torch.empty(3 * new, 4, 64, dtype=torch.float16, device=DEV)

    def work(cache, q_out):
        mxq.mxq_rope_append(cache, *p.views(dev), f, table, lens, starts, *w, q_out)

    other = torch.empty_like(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work((mxq.KvCache4 if bits == 4 else mxq.KvCache).empty(blocks, 2, 16, 64, DEV), out)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work(a, out)
    for rep in range(4):
        dev.copy_(torch.randn(dev.shape, generator=gen).half())
        torch.cuda.synchronize()
        note(f"rope_append replay {rep}")
        g.replay()
        torch.cuda.synchronize()
        work(b, other)
        torch.cuda.synchronize()
        assert torch.equal(out, other)
        assert all(torch.equal(x, y) for x, y in zip(_tensors(a), _tensors(b)))
        lens.add_(new)
