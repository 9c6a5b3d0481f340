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
