"""Norms, adapters, rotation into the cache, attention, router, experts and log probabilities together, as
examples/decode_step.py runs them.

A graph's steps and the same calls without one are the same kernels on the same values: equal bit for bit.  A prompt in
one pass and its tokens one by one differ in orders of sums (a few 2^-21), which can move an int8 activation of the next
product to its neighbour (1/127 of its block's largest value) in a few places of each of two layers: below 1e-3 of the
energy.  Log probabilities against the same scaled logits' in 64 bits: a logit below 2^4 is off by 2^-20 in its scaling here and by
two such in the call's (difference and scaling), the logarithm of the sum by 2^-21: below 2^-18.  The entropy's mean of
values up to 2^5 below the largest has weights off by 2^-22 and as much from their sums: below 2^-17 with the logarithm."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_steps_run_together():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    both, alone, graph, eager, _ = example.main(steps=5, prompts=(37, 70, 1, 16))
    assert torch.isfinite(both).all()
    worst = ((both - alone).square().sum(1) / alone.square().sum(1)).max()
    assert float(worst) <= 1e-3
    for g, e in zip(graph, eager):
        for a, b in zip(g, e):
            assert torch.isfinite(a.float()).all() and torch.equal(a, b)
        x, lp, entropy, ids, top, logits = g
        assert torch.equal(lp, top[:, :1])  # the chosen token is the best one
        assert bool((top <= 0).all()) and bool((entropy >= 0).all()) and bool((top.diff(dim=1) <= 0).all())
        assert torch.equal(logits.gather(1, ids[:, :1].long()), logits.amax(1, keepdim=True))
        want = torch.log_softmax(logits.double(), 1)
        assert float(logits.abs().max()) < 16 and float((want.gather(1, ids.long()) - top).abs().max()) <= 2.0 ** -18
        assert float((-(want * want.exp()).sum(1) - entropy).abs().max()) <= 2.0 ** -17
