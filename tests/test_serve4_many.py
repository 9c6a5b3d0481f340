"""The append that rotates and attention over 4 bits on calls of more work than one workgroup or one look takes: several
blocks of a row's heads a workgroup, more sequences than a wave has lanes, and grids that are refused."""

import numpy as np
import pytest
import torch

import dequant_matmul_qmv_amd as mxq
from tests.serve4_util import HALF, attention4_ref, check_attention, random_pool4
from tests.serve_util import paging
from tests.test_serve_attention4 import _poison, _run
from tests.test_serve_rope_append import Problem, note

P = 0x10000


# ----------------------------------------------------------------------------------------------- CPU
def _refused(bits, heads, kv, dim, tokens, seqs, starts, odd=0):
    """The error of a call on a cache of (never touched) pages, whose sizes are each allowed."""
    import dequant_matmul_qmv_amd._serve as serve
    from tests.test_serve_norm_rope import _rotation
    lib = serve._load()
    f = lib.mxq_rope_append if bits == 8 else lib.mxq_rope_append4
    cache = serve._CacheStruct(P, P, P, P, 4, kv, 16, dim)
    st = f(cache, P + odd, heads * dim, dim, P, heads * dim, dim, P + odd, kv * dim, dim, P, kv * dim, dim, _rotation(stride=tokens), P, 3, 3, P,
           starts, tokens, seqs, heads, mxq.MXQ_F16, None)
    return st, lib.mxq_last_error().decode()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("odd", [0, 2])
def test_grids_past_their_limit_are_refused(bits, odd):
    """2^24 sequences and tokens are within each limit of their own; 2^32 threads or more are not within a launch's."""
    for heads, kv, dim, tokens, starts in ((4, 2, 64, 2, P), (0, 1, 64, 2, P), (4, 2, 128, 2 ** 24, P), (28, 2, 128, 2 ** 24, None), (64, 1, 64, 2 ** 24, None)):
        st, text = _refused(bits, heads, kv, dim, tokens, 2 ** 24, starts, odd)
        assert st == mxq.MXQ_ERR_UNSUPPORTED and "split the call" in text, (heads, kv, dim, tokens, st, text)


# ----------------------------------------------------------------------------------------------- GPU
@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("heads,kv,dim,block,rot,new", [
    (32, 8, 128, 64, 128, 1400),    # 4 bits: two of 6 blocks of heads a workgroup
    (32, 8, 128, 128, 64, 3050),    # four, and the last two; 8 bits: three of 4 blocks of query heads, and the last
    (30, 6, 128, 32, 128, 4200),    # all of them
    (42, 21, 64, 16, 64, 3300),     # heads that fill no block
    (7, 7, 64, 64, 16, 4001)])
def test_several_blocks_of_heads(heads, kv, dim, block, rot, new, inter, bits):
    lens, news = [new + 37, 9, 1], [new, 6, 1]
    for t, kw in (("f16", dict()), ("bf16", dict(norm=False, implied=False)), ("bf16", dict(f32=True, axes=3))):
        p = Problem(bits, dim, block, t, lens, news, heads + new, heads=heads, kv=kv, rot=rot, inter=inter, **kw)
        note(f"rope_append, blocks of heads, {heads}/{kv} of {dim}, {bits} bits, new={new}, {inter}, {kw}")
        p.check(*p.call(), f"blocks {kw}")
        if t == "f16":
            dev = p.qkv.to("cuda:0")
            views = p.views(dev)
            note("the same in place")
            p.check(*p.call(q=views, q_out=views[0]), "blocks, in place")


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
def test_norms_on_one_side_of_several_blocks(bits):
    for side in (0, 1):
        kw = dict(heads=32, kv=8, rot=64)
        p = Problem(bits, 128, 64, "bf16", [3000], [2990], 3, **kw)
        plain = Problem(bits, 128, 64, "bf16", [3000], [2990], 3, norm=False, **kw)      # the same values
        assert torch.equal(p.qkv, plain.qkv)
        if side == 0:
            p.want, p.held = plain.want, plain.held
        else:
            p.want_q = plain.want_q
        p.w = [w if i == side else None for i, w in enumerate(p.w)]
        note(f"rope_append, blocks of heads, norm on side {side}, {bits} bits")
        p.check(*p.call(), "one side")


def _ragged(seqs, seed, longest):
    """Lengths of all sizes, every seventh sequence empty."""
    rng = np.random.default_rng(seed)
    lens = np.exp(rng.uniform(0, np.log(longest), seqs)).astype(int)
    lens[::7] = 0
    lens[seqs // 2], lens[-1] = longest, longest - 1
    return [int(n) for n in lens]


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("seqs", [64, 65, 96, 128, 129, 200])
def test_appends_of_many_sequences(seqs, bits):
    lens = _ragged(seqs, seqs, 300)
    rng = np.random.default_rng(seqs + 1)
    for heads, kv, dim, block in ((6, 2, 64, 16), (8, 8, 128, 64)):
        new = [min(n, int(rng.integers(0, 40))) for n in lens]
        p = Problem(bits, dim, block, "bf16", lens, new, seqs, heads=heads, kv=kv, extra=5)
        note(f"rope_append, {seqs} sequences, {bits} bits, dim {dim}")
        p.check(*p.call(), f"{seqs} sequences")
        p = Problem(bits, dim, block, "f16", [max(n, 1) for n in lens], [1] * seqs, seqs, heads=heads, kv=kv, implied=False)
        note("one token each")
        p.check(*p.call(one=True), f"{seqs} single tokens")
        p.check(*p.call(), f"{seqs} single tokens with starts")


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("seqs", [64, 65, 96, 128, 129, 200])
@pytest.mark.parametrize("kind", ["one", "drafts", "few and many"])
def test_attention_of_many_sequences(kind, seqs, t):
    """Tables that are split and tables that are not; empty sequences among the others."""
    gen = torch.Generator().manual_seed(seqs)
    rng = np.random.default_rng(seqs + 2)
    for dim, block, longest, heads, kv, window in ((64, 16, 900, 2, 1, 0), (128, 32, 2500, 2, 2, 0), (64, 64, 2500, 3, 1, 333)):
        lens = _ragged(seqs, seqs, longest)
        new = {"one": lambda n: 1, "drafts": lambda n: min(n, int(rng.integers(0, 6))),
               "few and many": lambda n: min(n, int(rng.choice([0, 1, 1, 3, 90])))}[kind]
        new = [new(n) for n in lens]
        blocks, table = paging(lens, block, gen)
        pool = _poison(list(random_pool4(blocks, kv, block, dim, gen)), table, lens, block)
        q = torch.randn(sum(new), heads, dim, generator=gen).to(HALF[t])
        note(f"attention4, {seqs} sequences, {kind}, dim {dim}, up to {longest} keys, {t}")
        out, lse = _run(q, pool, table, lens, new, window, one=kind == "one")
        check_attention(out, lse, attention4_ref(q, pool, table, lens, new, window, dim ** -0.5), f"{seqs} {kind}")


@pytest.mark.gpu
@pytest.mark.parametrize("seqs,longest", [(129, 5000), (200, 5000), (200, 4700), (130, 9000)])
def test_parts_of_many_sequences(seqs, longest):
    """More sequences than registers hold, tables on both sides of where long parts stop going first."""
    gen = torch.Generator().manual_seed(seqs + longest)
    lens = _ragged(seqs, seqs + 5, longest)
    blocks, table = paging(lens, 32, gen)
    pool = _poison(list(random_pool4(blocks, 1, 32, 64, gen)), table, lens, 32)
    for new in ([1] * seqs, [min(n, 1 + i % 3) for i, n in enumerate(lens)]):
        q = torch.randn(sum(new), 2, 64, generator=gen).half()
        note(f"attention4, {seqs} sequences of up to {longest} keys, new={new[:4]}")
        out, lse = _run(q, pool, table, lens, new, one=max(new) == 1)
        check_attention(out, lse, attention4_ref(q, pool, table, lens, new, 0, 64 ** -0.5), f"{seqs} of {longest}")
