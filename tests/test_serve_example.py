"""The serving operators together, as examples/generate.py runs them."""

import importlib.util
import os

import pytest
import torch

import dequant_matmul_qmv_amd as mxq
from tests.gpu_util import note

ROOT = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..")


def _example():
    spec = importlib.util.spec_from_file_location("generate_example", os.path.join(ROOT, "examples", "generate.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


PROMPTS = [[3, 1, 4, 1, 5, 9, 2, 6], [27], list(range(500, 570))]


@pytest.mark.gpu
def test_graph_and_eager_draw_the_same_tokens():
    ex = _example()
    note("example eager")
    eager = ex.generate(ex.Decoder(), PROMPTS, 24)
    note("example from a graph")
    graph = ex.generate(ex.Decoder(), PROMPTS, 24, graph=True)
    assert torch.equal(eager, graph)
    assert eager.shape == (3, 24) and int(eager.min()) >= 0 and int(eager.max()) < 4099
    assert len(set(eager.flatten().tolist())) > 20


@pytest.mark.gpu
def test_sequences_do_not_touch_each_other():
    """A sequence's greedy tokens are the same alone and in a batch.

    The projections of other row counts run other kernels, so logits may differ by their rounding: the largest
    logits compared are checked to lie further apart than that (2^-8 of the largest) before a difference counts."""
    ex = _example()
    note("example alone and in a batch")
    for i, prompt in enumerate(PROMPTS):
        ids = torch.tensor(prompt, device=ex.DEV)
        one, all_ = ex.Decoder(), ex.Decoder()
        n = len(prompt)
        table = torch.arange(6, dtype=torch.int32, device=ex.DEV)
        lens = torch.tensor([n], dtype=torch.int32, device=ex.DEV)
        alone = one(ids, torch.arange(n, dtype=torch.int32, device=ex.DEV), table[None], lens,
                    torch.tensor([0, n], dtype=torch.int32, device=ex.DEV))
        lengths = [len(p) for p in PROMPTS]
        starts = torch.tensor([sum(lengths[:j]) for j in range(4)], dtype=torch.int32, device=ex.DEV)
        batch = all_(torch.tensor([t for p in PROMPTS for t in p], device=ex.DEV),
                     torch.cat([torch.arange(m, dtype=torch.int32, device=ex.DEV) for m in lengths]),
                     torch.arange(18, dtype=torch.int32, device=ex.DEV).view(3, 6),
                     torch.tensor(lengths, dtype=torch.int32, device=ex.DEV), starts)[i:i + 1]
        top = alone.float().topk(2).values[0]
        margin = float(top[0] - top[1]) / float(alone.float().abs().max())
        assert bool(torch.isfinite(alone).all()) and bool(torch.isfinite(batch).all())
        u = torch.zeros(1, device=ex.DEV)
        a, b = mxq.mxq_sample(alone, u, temperature=0.0)[0], mxq.mxq_sample(batch, u, temperature=0.0)[0]
        if margin > 2.0 ** -8:
            assert int(a) == int(b), (i, margin)


def test_the_example_checks_its_cache():
    ex = _example()

    class Small:
        block = 16
        caches = [type("C", (), {"blocks": 2})()]

    with pytest.raises(ValueError, match="do not fit"):
        ex.generate(Small(), [[1], [2], [3]], 4)
