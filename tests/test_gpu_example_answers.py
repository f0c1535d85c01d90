"""The example's answers by beam search are what it says they are."""
from __future__ import annotations

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_answers_and_their_log_probabilities():
    import torch

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "preference_calibration.py")
    spec = importlib.util.spec_from_file_location("preference_calibration", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.main(steps=4, pairs=100, out=lambda *a: print(*a, flush=True))
    first, tokens, score = got["answers"]
    batch, beams, length = tokens.shape
    assert bool((score[:, :-1] >= score[:, 1:]).all())  # best first
    assert len({tuple(t) for t in tokens.view(-1, length).tolist()}) >= batch * beams - beams  # beams are different answers
    before = torch.cat([first.view(batch, 1, 1).expand(batch, beams, 1), tokens[:, :, :-1].long()], 2)
    logs = torch.log_softmax(got["model"].double(), 1)
    want = logs[before, tokens.long()].sum(2)
    # a step's score is rounded to f32, off by half a step, and so is its log-sum: 12 steps of a sum below 64
    assert float((score.double() - want).abs().max()) <= length * 2 * 64 * 2.0 ** -24
