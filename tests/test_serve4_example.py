"""The operators from the projection to attention over either cache, as examples/generate.py runs them."""

import pytest
import torch

from tests.gpu_util import note
from tests.test_serve_example import PROMPTS, _example


@pytest.mark.gpu
@pytest.mark.parametrize("norms,bits", [(True, 8), (True, 4), (False, 4)])
def test_graph_and_eager_draw_the_same_tokens(norms, bits):
    ex = _example()
    note(f"example eager, norms={norms}, {bits} bits")
    eager = ex.generate(ex.Decoder(norms=norms, bits=bits), PROMPTS, 24)
    note("example from a graph")
    graph = ex.generate(ex.Decoder(norms=norms, bits=bits), PROMPTS, 24, graph=True)
    assert torch.equal(eager, graph)
    assert eager.shape == (3, 24) and int(eager.min()) >= 0 and int(eager.max()) < 4099
    assert len(set(eager.flatten().tolist())) > 20
