"""The cache, attention, router and experts together, as examples/decode_layer.py runs
them: prompts in one pass and graph-replayed steps against one token at a time.

Both ways compute the same function; they differ in the attention's order of sums (a
few 2^-21), which can move an int8 activation of the next product to its neighbour
(1/127 of its block's largest value) in a few places: far below 1e-4 of the energy."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_prompts_and_graph_steps_match_single_tokens():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_layer.py")
    spec = importlib.util.spec_from_file_location("decode_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    both, alone, _ = example.main(steps=5, prompts=(37, 70, 1, 16))
    for a, b in zip(both, alone):
        assert torch.isfinite(a).all()
        worst = ((a - b).square().sum(1) / b.square().sum(1)).max()
        assert float(worst) <= 1e-4
