"""mxq_norm_rope on enough tokens that a workgroup takes several, at a time and one after the other."""

import pytest
import torch

import dequant_matmul_qmv_amd as mxq
from tests.gpu_util import note
from tests.serve4_util import HALF, frequencies
from tests.test_serve_norm_rope import DEV, _check, _inputs

GUARD = 3  # tokens before and behind an output that have to stay


def _guarded(n, heads, dim, dtype):
    """(an output of n tokens, all of its memory), filled with a NaN that no result has."""
    whole = torch.full((n + 2 * GUARD, heads, dim), -3, dtype=torch.int16, device=DEV).view(dtype)
    return whole[GUARD:GUARD + n], whole


def _run(n, heads, kv, dim, rot, inter, t, norms=3, f32=False, axes=0, far=131072):
    qkv, w, gen = _inputs(n, heads, kv, dim, t, n + dim + heads)
    f = frequencies(rot) if rot else torch.zeros(0)
    pos = torch.randint(-far, far, (axes, n) if axes else (n,), generator=gen, dtype=torch.int32)
    which = (torch.arange(rot // 2) * axes // (rot // 2)).int() if axes else None
    w = [x if f32 else x.to(HALF[t]) for x in w]
    qw, kw = w[0] if norms & 1 else None, w[1] if norms & 2 else None
    on = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    dev = qkv.to(DEV)
    q, k = dev[:, :heads * dim].view(n, heads, dim), dev[:, heads * dim:(heads + kv) * dim].view(n, kv, dim)
    (y, y_all), (z, z_all) = _guarded(n, heads, dim, HALF[t]), _guarded(n, kv, dim, HALF[t])
    what = f"norm_rope n={n} heads={heads}/{kv} dim={dim} rot={rot} inter={inter} {t} norms={norms} axes={axes}"
    note(what)
    mxq.mxq_norm_rope(q, k if kv else None, f.to(DEV), on(pos), on(qw), on(kw), y, z if kv else None, axes=on(which), interleaved=inter)
    torch.cuda.synchronize()
    _check(y, q.cpu(), qw, 1e-6, f, pos, which, inter, what + ", q")
    if kv:
        _check(z, k.cpu(), kw, 1e-6, f, pos, which, inter, what + ", k")
    for x in (y_all, z_all):
        x = x.view(torch.int16)
        assert bool((x[:GUARD] == -3).all()) and bool((x[GUARD + n:] == -3).all()), what


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("rot", [0, 16])
def test_one_head_of_16_values(rot, t):
    """A token has one lane: its lanes' number divides by nothing."""
    for n in (1, 63, 513, 1023, 1024, 1500, 5003, 40001):
        for heads, kv in ((1, 0), (0, 1)):
            _run(n, heads, kv, 16, rot, n % 2 == 1, t)


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,heads,kv,dim,rot", [
    (513, 3, 0, 16, 16), (1024, 2, 1, 16, 16), (40001, 2, 1, 16, 0),                    # up to 64 tokens at a time
    (513, 4, 2, 64, 64), (1023, 5, 1, 80, 48), (1025, 3, 1, 48, 32), (1500, 2, 0, 32, 32), (5003, 16, 4, 64, 32),
    (777, 4, 2, 256, 256), (5000, 4, 2, 256, 256),                                      # the table of turns sets how many
    (1100, 56, 14, 128, 64),                                                            # a token of more than a workgroup's lanes
    (600, 3, 1, 250, 18), (1300, 2, 1, 128, 20)])                                       # one token a workgroup
def test_many_tokens(n, heads, kv, dim, rot, inter):
    """Tokens at a time, one after the other, and last ones that fill neither; no norm, one, both, in f32 and in the type."""
    for norms, f32, t in ((3, False, "bf16"), (n % 3, True, "f16")):
        _run(n, heads, kv, dim, rot, inter, t, norms, f32)


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_many_tokens_on_several_axes(inter):
    for n, heads, kv, dim, rot in ((1500, 3, 1, 64, 32), (5003, 16, 4, 64, 64), (700, 5, 1, 128, 100)):
        _run(n, heads, kv, dim, rot, inter, "f16", axes=3, far=5000)


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("n,heads,kv,dim,rot,inter", [(8191, 8, 2, 128, 128, False), (2500, 32, 8, 128, 128, True),
                                                      (9001, 12, 4, 64, 32, False), (33333, 12, 4, 16, 16, True)])
def test_more_than_the_caches_hold(n, heads, kv, dim, rot, inter, t):
    """Calls of more than 32 MB, which pass the L2s by."""
    assert 4 * n * (heads + kv) * dim > 32 << 20
    _run(n, heads, kv, dim, rot, inter, t)


@pytest.mark.gpu
def test_more_tokens_than_a_launch_takes():
    """2^23 tokens and some: the second launch's rows, with its positions on each axis, and the seam."""
    n, dim, rot = 2 ** 23 + 70, 16, 16
    gen = torch.Generator().manual_seed(4)
    f = frequencies(rot)
    rows = torch.cat((torch.arange(0, 40), torch.arange(2 ** 23 - 40, n)))
    x = torch.randn(rows.shape[0], 1, dim, generator=gen).half()
    pos = torch.randint(-5000, 5000, (2, rows.shape[0]), generator=gen, dtype=torch.int32)
    w = (1 + 0.3 * torch.randn(dim, generator=gen)).half()
    axes = (torch.arange(rot // 2) % 2).int()
    q = torch.ones(n, 1, dim, dtype=torch.float16, device=DEV)
    at = torch.zeros(2, n, dtype=torch.int32, device=DEV)
    q[rows.to(DEV)], at[:, rows.to(DEV)] = x.to(DEV), pos.to(DEV)
    out, whole = _guarded(n, 1, dim, torch.float16)
    note("norm_rope past 2^23 tokens")
    mxq.mxq_norm_rope(q, None, f.to(DEV), at, w.to(DEV), None, out, axes=axes.to(DEV))
    torch.cuda.synchronize()
    _check(out[rows.to(DEV)], x, w, 1e-6, f, pos, axes, False, "seam")
    middle = out[40:2 ** 23 - 40]                     # tokens alike
    assert bool((middle == middle[:1]).all())
    _check(middle[:1], torch.ones(1, 1, dim, dtype=torch.float16), w, 1e-6, f, torch.zeros(2, 1, dtype=torch.int32), axes, False, "middle")
    whole = whole.view(torch.int16)
    assert bool((whole[:GUARD] == -3).all()) and bool((whole[GUARD + n:] == -3).all())
