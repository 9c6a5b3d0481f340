"""Heads normed and rotated in one pass: against the definition in 64 bits, against the stated f32 steps bit for bit,
and refusals."""

import numpy as np
import pytest
import torch

import dequant_matmul_qmv_amd as mxq
from tests.gpu_util import note
from tests.serve4_util import HALF, frequencies, half_step, rotated_bits, rotated_ref

DEV = "cuda:0"
P = 0x10000


def _rotation(**kw):
    import dequant_matmul_qmv_amd._serve as serve
    r = dict(inv_freq=P, positions=P, stride=8, axis=None, axes=1, rot=64, inter=0, wtype=mxq.MXQ_F32, qw=None, kw=None, eps=1e-6)
    r.update(kw)
    return serve._RotationStruct(r["inv_freq"], r["positions"], r["stride"], r["axis"], r["axes"], r["rot"], r["inter"], r["wtype"],
                                 r["qw"], r["kw"], r["eps"])


def _call(rotation="default", **kw):
    import dequant_matmul_qmv_amd._serve as serve
    a = dict(q=P, k=P, qo=P, ko=P, tokens=4, heads=2, kv_heads=1, dim=64, dtype=mxq.MXQ_F16)
    a.update({n: v for n, v in kw.items() if n in a})
    r = _rotation(**{n: v for n, v in kw.items() if n not in a}) if rotation == "default" else rotation
    side = (a["heads"] * a["dim"], a["dim"])
    return serve._load().mxq_norm_rope(a["q"], *side, a["k"], *side, a["qo"], *side, a["ko"], *side, r, a["tokens"], a["heads"],
                                       a["kv_heads"], a["dim"], a["dtype"], None)


def test_refusals():
    bad, unsup, mis = mxq.MXQ_ERR_INVALID_ARG, mxq.MXQ_ERR_UNSUPPORTED, mxq.MXQ_ERR_MISALIGNED
    for name in ("tokens", "heads", "kv_heads", "dim", "rot"):
        assert _call(**{name: -1}) == bad, name
    assert _call(rotation=None) == bad
    assert _call(axes=0) == bad and _call(axes=65537) == bad
    assert _call(axes=2, stride=3) == bad
    for eps in (-1e-9, float("nan"), float("inf")):
        assert _call(eps=eps) == bad
    for name in ("q", "k", "qo", "ko", "inv_freq", "positions"):
        assert _call(**{name: None}) == bad, name
    assert _call(dim=272, rot=64) == unsup and _call(rot=66) == unsup and _call(rot=63) == unsup
    assert _call(dtype=mxq.MXQ_F32) == unsup
    assert _call(heads=65536) == unsup and _call(tokens=2 ** 31) == unsup
    assert _call(qw=P, wtype=mxq.MXQ_BF16) == unsup and _call(kw=P, wtype=7) == unsup
    for name, at in (("q", 1), ("k", 1), ("qo", 1), ("ko", 1), ("inv_freq", 2), ("positions", 2), ("axis", 2), ("qw", 2), ("kw", 1)):
        assert _call(**{name: P + at}) == mis, name
    assert _call(qw=P + 1, wtype=mxq.MXQ_F16) == mis
    assert _call(tokens=0, q=None, k=None, qo=None, ko=None, positions=None) == mxq.MXQ_OK
    assert _call(heads=0, kv_heads=0) == mxq.MXQ_OK and _call(dim=0, rot=0) == mxq.MXQ_OK
    with pytest.raises(ValueError, match="device tensor"):
        mxq.mxq_norm_rope(torch.zeros(1, 1, 64, dtype=torch.float16), None, torch.zeros(4), torch.zeros(1, dtype=torch.int32))


def _inputs(n, heads, kv, dim, t, seed, scale=1.5):
    gen = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(n, (heads + 2 * kv) * dim, generator=gen) * scale).to(HALF[t])
    w = [(1 + 0.3 * torch.randn(dim, generator=gen)) for _ in range(2)]
    return qkv, w, gen


def _check(got, x, weight, eps, inv_freq, positions, axes, inter, what):
    want, off = rotated_ref(x, weight, eps, inv_freq, positions, axes, inter)
    half = half_step(x.dtype)
    y = got.double().cpu().numpy()
    bound = off + half * (np.abs(want) + off) + torch.finfo(x.dtype).smallest_normal * half * 2
    assert np.all(np.abs(y - want) <= bound), (what, float((np.abs(y - want) / bound).max()))
    bits = rotated_bits(x, weight, eps, inv_freq, positions, axes, inter)
    assert torch.equal(got.cpu().view(torch.int16), bits.view(torch.int16)), (what, int((got.cpu() != bits).sum()))


SHAPES = [(64, 64), (128, 128), (128, 64), (256, 256), (256, 64), (64, 32), (96, 96), (80, 48), (48, 16), (16, 16), (32, 32), (64, 0),
          (128, 20), (66, 66), (33, 32), (2, 2), (250, 18), (1, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot", SHAPES)
def test_shapes(dim, rot, inter, t):
    """Every path, views of a fused projection, norms of both, one or none, in the type or in f32."""
    for n, heads, kv, norms, wide in ((1, 1, 1, 3, False), (5, 4, 2, 3, True), (3, 17, 1, 1, False), (37, 8, 8, 2, True), (2, 3, 0, 1, False),
                                      (4, 5, 2, 0, False), (70, 2, 1, 3, False)):
        qkv, w, gen = _inputs(n, heads, kv, dim, t, dim + n)
        f = frequencies(rot) if rot else torch.zeros(0)
        pos = torch.randint(0, 131072, (n,), generator=gen, dtype=torch.int32)
        w = [x if wide else x.to(HALF[t]) for x in w]
        qw, kw = w[0] if norms & 1 else None, w[1] if norms & 2 else None
        dev = qkv.to(DEV)
        q, k = dev[:, :heads * dim].view(n, heads, dim), dev[:, heads * dim:(heads + kv) * dim].view(n, kv, dim)
        note(f"norm_rope dim={dim} rot={rot} inter={inter} {t} n={n} heads={heads}/{kv} norms={norms}")
        y, z = mxq.mxq_norm_rope(q, k if kv else None, f.to(DEV), pos.to(DEV), None if qw is None else qw.to(DEV),
                                 None if kw is None else kw.to(DEV), interleaved=inter)
        torch.cuda.synchronize()
        _check(y, q.cpu(), qw, 1e-6, f, pos, None, inter, "q")
        if kv:
            _check(z, k.cpu(), kw, 1e-6, f, pos, None, inter, "k")


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (64, 32), (96, 36)])
def test_axes(dim, rot, inter):
    """Each pair by its own axis, in sections or in turn; axes that are none count as the nearest."""
    n, heads, kv = 29, 6, 2
    qkv, w, gen = _inputs(n, heads, kv, dim, "bf16", rot)
    f, half = frequencies(rot), rot // 2
    pos = torch.stack((torch.randint(0, 5000, (n,), generator=gen), torch.arange(n) * 3, torch.randint(-7, 90, (n,), generator=gen))).int()
    dev = qkv.to(DEV)
    q, k = dev[:, :heads * dim].view(n, heads, dim), dev[:, heads * dim:(heads + kv) * dim].view(n, kv, dim)
    w = [x.bfloat16() for x in w]
    for axes in (torch.arange(half) % 3, torch.arange(half) * 3 // half, torch.zeros(half), torch.arange(half) % 9 - 3):
        axes = axes.int()
        note(f"norm_rope axes dim={dim} rot={rot} {inter}")
        y, z = mxq.mxq_norm_rope(q, k, f.to(DEV), pos.to(DEV), w[0].to(DEV), w[1].to(DEV), axes=axes.to(DEV), interleaved=inter)
        torch.cuda.synchronize()
        _check(y, q.cpu(), w[0], 1e-6, f, pos, axes, inter, "q")
        _check(z, k.cpu(), w[1], 1e-6, f, pos, axes, inter, "k")


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_values(t):
    """Zeros, the type's largest and smallest values, one value alone, rows with infinities and NaN beside others."""
    dim, n = 128, 12
    x = torch.zeros(n, 2, dim, dtype=HALF[t])
    big, small = torch.finfo(HALF[t]).max, torch.finfo(HALF[t]).smallest_normal
    gen = torch.Generator().manual_seed(1)
    x[1] = big / 512
    x[2] = small / 4
    x[3, :, 5] = 1.0
    x[4] = torch.randn(2, dim, generator=gen) * small
    x[5] = torch.randn(2, dim, generator=gen) * (big / 64)
    x[6:] = torch.randn(n - 6, 2, dim, generator=gen)
    f, w = frequencies(dim), (1 + torch.rand(dim, generator=gen)).to(HALF[t])
    pos = torch.arange(n, dtype=torch.int32) * 1000
    for eps in (1e-6, 1e-30, 0.5):
        note(f"norm_rope values {t} eps={eps}")
        y, _ = mxq.mxq_norm_rope(x.to(DEV), None, f.to(DEV), pos.to(DEV), w.to(DEV), eps=eps)
        torch.cuda.synchronize()
        _check(y, x, w, eps, f, pos, None, False, f"values {eps}")
    odd = x.clone()
    odd[7, 0, 3], odd[8, 1, 100] = torch.inf, torch.nan
    note(f"norm_rope inf, nan {t}")
    y0, _ = mxq.mxq_norm_rope(x.to(DEV), None, f.to(DEV), pos.to(DEV), w.to(DEV))
    y1, _ = mxq.mxq_norm_rope(odd.to(DEV), None, f.to(DEV), pos.to(DEV), w.to(DEV))
    y2, _ = mxq.mxq_norm_rope(odd.to(DEV), None, f.to(DEV), pos.to(DEV))
    torch.cuda.synchronize()
    for y in (y1, y2):
        assert y[7, 0, 3].isnan() or y[7, 0, 3].isinf()
        assert y[8, 1, 100].isnan()
    same = torch.ones(n, 2, dtype=torch.bool)
    same[7, 0] = same[8, 1] = False
    assert torch.equal(y0.cpu()[same], y1.cpu()[same])
    assert y1[8, 1].isnan().all()
    # norms alone, and a head of zeros with eps = 0 (0 / 0)
    y, _ = mxq.mxq_norm_rope(x.to(DEV), None, torch.zeros(0, device=DEV), pos.to(DEV), w.to(DEV), eps=0.0)
    assert y[0].isnan().all() and y[6:].isfinite().all()


@pytest.mark.gpu
def test_far_positions():
    """Positions up to 2^31 and below 0 with the highest frequency."""
    dim, n = 64, 9
    qkv, _, gen = _inputs(n, 3, 0, dim, "f16", 3)
    q = qkv.view(n, 3, dim)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 131071, -131071, 2 ** 24 + 1, 1000003], dtype=torch.int32)
    f = frequencies(dim)
    note("norm_rope far")
    y, _ = mxq.mxq_norm_rope(q.to(DEV), None, f.to(DEV), pos.to(DEV))
    torch.cuda.synchronize()
    _check(y, q, None, 0, f, pos, None, False, "far")


@pytest.mark.gpu
def test_in_place_strides_streams_and_other_rows():
    n, heads, kv, dim = 33, 6, 2, 128
    qkv, w, gen = _inputs(n, heads, kv, dim, "bf16", 11)
    f, pos = frequencies(dim).to(DEV), torch.randint(0, 9000, (n,), generator=gen, dtype=torch.int32).to(DEV)
    w = [x.bfloat16().to(DEV) for x in w]
    dev = qkv.to(DEV)
    view = lambda b: (b[:, :heads * dim].view(n, heads, dim), b[:, heads * dim:(heads + kv) * dim].view(n, kv, dim))  # noqa: E731
    want = mxq.mxq_norm_rope(*view(dev), f, pos, *w)
    note("norm_rope in place")
    mine = dev.clone()
    q, k = view(mine)
    a, b = mxq.mxq_norm_rope(q, k, f, pos, *w, q, k)
    assert a.data_ptr() == q.data_ptr() and torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert torch.equal(mine[:, (heads + kv) * dim:], dev[:, (heads + kv) * dim:])
    note("norm_rope on rows that are not 16-byte aligned")
    odd = torch.zeros(n, heads, dim + 3, dtype=torch.bfloat16, device=DEV)
    odd[:, :, 1:dim + 1] = view(dev)[0]
    out = torch.full((heads, n, dim + 1), 7.0, dtype=torch.bfloat16, device=DEV)
    a, _ = mxq.mxq_norm_rope(odd[:, :, 1:dim + 1], None, f, pos, w[0], None, out.transpose(0, 1)[:, :, :dim])
    assert torch.equal(a, want[0]) and (out[:, :, dim] == 7).all()
    note("norm_rope on another stream")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = mxq.mxq_norm_rope(*view(dev), f, pos, *w, stream=side)
    side.synchronize()
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    note("norm_rope of nothing")
    a, b = mxq.mxq_norm_rope(view(dev)[0][:0], view(dev)[1][:0], f, pos[:0], *w)
    assert a.shape == (0, heads, dim)


@pytest.mark.gpu
def test_python_refusals():
    x, f, p = torch.zeros(2, 3, 64, dtype=torch.float16, device=DEV), torch.ones(32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    ok = torch.ones(64, dtype=torch.float16, device=DEV)
    for args, kw in (((x, None, f, None), {}), ((x, None, f.double(), p), {}), ((x, None, torch.ones(33, device=DEV), p), {}),
                     ((x, None, f, p.long()), {}), ((x, None, f, p[:1]), {}), ((x, None, f, torch.stack((p, p))), {}),
                     ((x, None, f, torch.stack((p, p))), dict(axes=p)), ((x, None, f, p, ok[:63]), {}), ((x, None, f, p, ok.bfloat16()), {}),
                     ((x, x, f, p, ok, ok.float()), {}), ((x, x[:1], f, p), {}), ((x, None, f, p, None, None, None, x), {}),
                     ((x.float(), None, f, p), {}), ((x, x, f, p, None, None, x[:, :1]), {}), ((x, None, f.cpu(), p), {})):
        with pytest.raises((TypeError, ValueError)):
            mxq.mxq_norm_rope(*args, **kw)


@pytest.mark.gpu
def test_graph_replay():
    n, heads, kv, dim = 7, 8, 2, 64
    qkv, w, gen = _inputs(n, heads, kv, dim, "f16", 2)
    dev, f = qkv.to(DEV), frequencies(dim).to(DEV)
    pos = torch.zeros(3, n, dtype=torch.int32, device=DEV)
    axes = (torch.arange(32) % 3).int().to(DEV)
    w = [x.half().to(DEV) for x in w]
    q, k = dev[:, :heads * dim].view(n, heads, dim), dev[:, heads * dim:(heads + kv) * dim].view(n, kv, dim)
    yq, yk = torch.empty(n, heads, dim, dtype=torch.float16, device=DEV), torch.empty(n, kv, dim, dtype=torch.float16, device=DEV)

    def work(a, b):
        mxq.mxq_norm_rope(q, k, f, pos, *w, a, b, axes=axes)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(yq, yk)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work(yq, yk)
    for rep in range(3):
        dev.copy_((torch.randn(dev.shape, generator=gen)).half())
        pos.copy_(torch.randint(0, 5000, (3, n), generator=gen, dtype=torch.int32))
        torch.cuda.synchronize()
        note(f"norm_rope replay {rep}")
        g.replay()
        torch.cuda.synchronize()
        a, b = torch.empty_like(yq), torch.empty_like(yk)
        work(a, b)
        torch.cuda.synchronize()
        assert torch.equal(a, yq) and torch.equal(b, yk)
