"""The next token's draw: against the rule in 64 bits, and refusals.

Tokens are whole numbers and have to be equal.  A weight is off by 2^-44 of the
largest, so a sum of n by n 2^-44 at most: the inputs' borders are checked to be
further away than that.  The probability is one f32 rounding (2^-24) of a
quotient of such sums."""

import numpy as np
import pytest
import torch

import dequant_matmul_qmv_amd as mxq
from tests.gpu_util import note
from tests.serve_util import sample_ref

DEV = "cuda:0"
P = 0x10000
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _call(settings=None, null_settings=False, **kw):
    import dequant_matmul_qmv_amd._serve as serve
    lib = serve._load()
    s = dict(temperature=None, top_k=None, top_p=None, min_p=None)
    s.update(settings or {})
    st = None if null_settings else serve._SamplingStruct(s["temperature"], s["top_k"], s["top_p"], s["min_p"], 1.0, 0, 1.0, 0.0)
    a = dict(logits=P, stride=100, rows=2, vocab=100, dtype=mxq.MXQ_F16, u=P, tokens=P, probs=P)
    a.update(kw)
    return lib.mxq_sample(a["logits"], a["stride"], a["rows"], a["vocab"], a["dtype"], a["u"], st, a["tokens"],
                          a["probs"], None)


def test_refusals():
    assert _call(rows=-1) == mxq.MXQ_ERR_INVALID_ARG
    assert _call(vocab=-1) == mxq.MXQ_ERR_INVALID_ARG
    assert _call(vocab=0) == mxq.MXQ_ERR_INVALID_ARG
    assert _call(vocab=2 ** 20 + 1, stride=2 ** 21) == mxq.MXQ_ERR_UNSUPPORTED
    assert _call(rows=2 ** 25) == mxq.MXQ_ERR_UNSUPPORTED
    assert _call(dtype=5) == mxq.MXQ_ERR_UNSUPPORTED
    assert _call(stride=99) == mxq.MXQ_ERR_INVALID_ARG
    assert _call(null_settings=True) == mxq.MXQ_ERR_INVALID_ARG
    for name in ("logits", "u", "tokens", "probs"):
        assert _call(**{name: None}) == mxq.MXQ_ERR_INVALID_ARG, name
        assert _call(**{name: P + 1}) == mxq.MXQ_ERR_MISALIGNED, name
    for name in ("temperature", "top_k", "top_p", "min_p"):
        assert _call({name: P + 2}) == mxq.MXQ_ERR_MISALIGNED, name
    assert _call(logits=P + 2, dtype=mxq.MXQ_F32) == mxq.MXQ_ERR_MISALIGNED
    assert _call(logits=None, u=None, tokens=None, probs=None, null_settings=True, rows=0) == mxq.MXQ_OK
    with pytest.raises(ValueError, match="device tensor"):
        mxq.mxq_sample(torch.zeros(2, 5), torch.zeros(2))


def _check(x, u, t, k, p, m, what, slack=None):
    """Draw every row, with a setting given as a list (one a row) or a number."""
    rows, vocab = x.shape
    pick = lambda v, d: torch.tensor(v, dtype=d, device=DEV) if isinstance(v, list) else v  # noqa: E731
    at = lambda v, i: v[i] if isinstance(v, list) else v  # noqa: E731
    note(what)
    tok, prob = mxq.mxq_sample(x.to(DEV), u.to(DEV), temperature=pick(t, torch.float32), top_k=pick(k, torch.int32),
                               top_p=pick(p, torch.float32), min_p=pick(m, torch.float32))
    torch.cuda.synchronize()
    tok, prob = tok.cpu().tolist(), prob.cpu().double().tolist()
    xs = x.float().numpy()
    f = np.float32
    for r in range(rows):
        want, wp, near = sample_ref(xs[r], u[r].item(), f(at(t, r)), at(k, r), f(at(p, r)), f(at(m, r)))
        if near <= vocab * 2.0 ** -43:
            continue    # on a border: an exact tie of the sums is tested apart
        assert tok[r] == want, (what, r, tok[r], want, near)
        assert abs(prob[r] - wp) <= wp * (2.0 ** -24 + vocab * 2.0 ** -43) + 2.0 ** -43, (what, r, prob[r], wp)


def _logits(rows, vocab, t, seed, spread=2.5):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab, generator=gen) * spread
    likely = torch.randint(0, vocab, (rows, 12), generator=gen)
    x.scatter_add_(1, likely, 6 + 2 * torch.randn(rows, 12, generator=gen))
    return x.to(TYPES[t]), torch.rand(rows, generator=gen)


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.8, 40, 0.95, 0.0), (1.7, 0, 0.9, 0.0), (0.3, 0, 0.5, 0.0), (1.0, 500, 1.0, 0.0),
            (1.3, 0, 1.0, 0.02), (1.0, 20000, 0.99, 0.05), (0.0, 7, 0.9, 0.0), (1.0, 1, 1.0, 0.0), (30.0, 0, 0.9, 0.0),
            (1.5, 3, 0.6, 0.3), (0.01, 0, 0.9, 0.0), (100.0, 1000, 0.99, 0.5)]


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab", [1, 2, 63, 1000, 4097, 32003, 128256])
def test_settings(vocab, t):
    rows = len(SETTINGS) * (3 if vocab < 5000 else 1)
    x, u = _logits(rows, vocab, t, vocab)
    cols = [[s[j] for s in SETTINGS] * (rows // len(SETTINGS)) for j in range(4)]
    _check(x, u, *cols, f"sample vocab={vocab} {t}")


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "f32"])
@pytest.mark.parametrize("s", SETTINGS)
def test_one_row_numbers(s, t):
    """Settings as plain numbers, one row, several uniform numbers."""
    x, _ = _logits(1, 20011, t, 3)
    for u in (0.0, 0.37, 0.5, 0.999, 1 - 2.0 ** -24):
        _check(x, torch.tensor([u]), *s, f"sample one row {s} u={u} {t}")


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16", "f32"])
def test_ties(t):
    """Few distinct values: prefixes that end among equals, by index; sums are exact."""
    gen = torch.Generator().manual_seed(4)
    vocab = 5000
    x = torch.randint(0, 4, (64, vocab), generator=gen).float().mul(0.5).to(TYPES[t])
    u = torch.rand(64, generator=gen)
    for s in ((1.0, 700, 1.0, 0.0), (1.0, 2000, 0.5, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.5), (1.0, 5, 1.0, 0.0), (1.0, 0, 0.01, 0.0)):
        _check(x, u, *s, f"sample ties {s} {t}")
    same = torch.full((8, vocab), -3.0).to(TYPES[t])
    tok, prob = mxq.mxq_sample(same.to(DEV), torch.arange(8, device=DEV) / 8, top_k=4000)
    assert tok.tolist() == [500 * i for i in range(8)] and prob.tolist() == [float(np.float32(1 / 4000))] * 8
    tok, prob = mxq.mxq_sample(same.to(DEV), torch.arange(8, device=DEV) / 8, top_p=0.5)
    assert tok.tolist() == [i * 2500 // 8 for i in range(8)]
    zero = torch.tensor([[0.0, -0.0, 0.0, -1.0]]).to(TYPES[t])
    tok, _ = mxq.mxq_sample(zero.to(DEV), torch.tensor([0.9], device=DEV), top_k=2)
    assert tok.tolist() == [1]           # both zeros are equal: the first two by index


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16", "f32"])
def test_masked_rows(t):
    """-inf, the type's lowest value, NaN and +inf among the logits; a row of nothing but -inf."""
    vocab = 3001
    x, u = _logits(9, vocab, t, 5)
    low = torch.finfo(TYPES[t]).min
    x[0, 5:] = -torch.inf
    x[1, :] = -torch.inf
    x[2, 100:2900] = low
    x[3, ::3] = torch.nan
    x[4, 7] = torch.inf
    x[4, 2000] = torch.inf
    x[5, :] = low
    x[6, :] = low
    x[6, 77] = 0.0
    x[7, :] = torch.nan
    for s in SETTINGS:
        _check(x, u, *s, f"sample masked {s} {t}")


@pytest.mark.gpu
def test_settings_at_their_ends():
    x, u = _logits(8, 777, "f32", 6)
    big = 10 ** 9
    nan = float("nan")
    _check(x, u, [1.0, -1.0, nan, 1e-30, 1e30, 1.0, 1.0, 1.0], [big, 5, 5, 0, 0, -3, 776, 777],
           [1.0, 0.9, 0.9, 0.9, 0.9, 0.0, 1.5, nan], [0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 1.0, -1.0], "sample ends")
    _check(x, u, 1.0, 0, 1.0, [0.0, 1.0, 1.5, nan, -2.0, 1e-30, 0.999, 0.5], "sample min_p ends")
    tok, _ = mxq.mxq_sample(x.to(DEV), torch.ones(8, device=DEV), top_k=3)      # u = 1: the last kept token
    assert tok.tolist() == x.topk(3, 1).indices.max(1).values.tolist()


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(300, 9001), (1030, 2100), (40, 70001)])
def test_many_rows(rows, vocab, t):
    """More rows than one launch holds, and more than one last workgroup a row would serve; every row its own settings."""
    x, u = _logits(rows, vocab, t, 30 + rows, spread=1.5)
    cols = [[SETTINGS[(7 * r) % len(SETTINGS)][j] for r in range(rows)] for j in range(4)]
    _check(x, u, *cols, f"sample rows={rows} vocab={vocab} {t}")


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 200])
def test_wide_prefixes(rows):
    """Flat rows: prefixes of thousands of tokens by count, by weight, by both, and cut by min-p."""
    x, u = _logits(rows, 20000, "f32", 40, spread=0.7)
    for s in ((1.0, 0, 0.9, 0.0), (1.0, 9000, 1.0, 0.0), (2.0, 9000, 0.8, 0.0), (2.0, 9000, 0.8, 0.01), (1.0, 0, 1.0, 1e-4),
              (5.0, 0, 0.99, 0.02), (3.0, 19999, 0.999, 0.0)):
        _check(x, u, *s, f"sample wide rows={rows} {s}")


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [2, 150])
def test_wide_prefixes_of_equals(rows):
    """More equal logits than a list holds: the end of the prefix is found in the row itself."""
    gen = torch.Generator().manual_seed(41)
    x = torch.randint(0, 3, (rows, 15000), generator=gen).float().half()
    u = torch.rand(rows, generator=gen)
    for s in ((1.0, 7000, 1.0, 0.0), (1.0, 0, 0.7, 0.0), (1.5, 12000, 0.9, 0.3), (1.0, 6000, 0.5, 0.0)):
        _check(x, u, *s, f"sample equals rows={rows} {s}")


@pytest.mark.gpu
def test_odd_base_of_every_type():
    for t in ("f16", "bf16", "f32"):
        x, u = _logits(4, 3001, t, 42)
        wide = torch.full((4, 3011), 50.0).to(TYPES[t])
        wide[:, 5:3006] = x
        view = wide.to(DEV)[:, 5:3006]
        for s in ((0.9, 40, 0.9, 0.0), (1.7, 0, 0.95, 0.0), (1.0, 0, 1.0, 0.0), (1.0, 2500, 1.0, 0.0)):
            note(f"sample odd base {t} {s}")
            kw = dict(temperature=s[0], top_k=s[1], top_p=s[2], min_p=s[3])
            a, b = mxq.mxq_sample(view, u.to(DEV), **kw), mxq.mxq_sample(x.to(DEV), u.to(DEV), **kw)
            torch.cuda.synchronize()
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for n in (1, 5, 7, 8, 9):
        gen = torch.Generator().manual_seed(43 + n)
        x, u = torch.randn(4, n, generator=gen).half(), torch.rand(4, generator=gen)
        _check(x, u, 1.0, 0, 0.9, 0.0, f"sample vocab={n}")


@pytest.mark.gpu
def test_strided_rows_and_odd_base():
    x, u = _logits(6, 4001, "f16", 8)
    wide = torch.zeros(6, 4500, dtype=torch.float16)
    wide[:, 3:4004] = x
    view = wide.to(DEV)[:, 3:4004]
    tok, prob = mxq.mxq_sample(view, u.to(DEV), temperature=0.9, top_k=50, top_p=0.9)
    tok2, prob2 = mxq.mxq_sample(x.to(DEV), u.to(DEV), temperature=0.9, top_k=50, top_p=0.9)
    torch.cuda.synchronize()
    assert torch.equal(tok, tok2) and torch.equal(prob, prob2)
    _check(x, u, 0.9, 50, 0.9, 0.0, "sample strided")


@pytest.mark.gpu
def test_graph_replay():
    x, u = _logits(5, 32003, "f16", 9)
    xd, ud = x.to(DEV), u.to(DEV)
    tok, prob = torch.empty(5, dtype=torch.int32, device=DEV), torch.empty(5, device=DEV)
    k = torch.tensor([0, 40, 0, 1000, 1], dtype=torch.int32, device=DEV)

    def work():
        mxq.mxq_sample(xd, ud, tok, prob, temperature=0.9, top_k=k, top_p=0.95)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    note("sample captured")
    with torch.cuda.graph(g):
        work()
    for rep in range(3):
        x2, u2 = _logits(5, 32003, "f16", 20 + rep)
        xd.copy_(x2)
        ud.copy_(u2)
        torch.cuda.synchronize()
        note(f"sample replay {rep}")
        g.replay()
        torch.cuda.synchronize()
        got = tok.clone(), prob.clone()
        work()
        torch.cuda.synchronize()
        assert torch.equal(got[0], tok) and torch.equal(got[1], prob)
