"""The preference and calibration example runs and does what it says."""
from __future__ import annotations

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_preference_calibration():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "preference_calibration.py")
    spec = importlib.util.spec_from_file_location("preference_calibration", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.main(steps=20, pairs=500, out=lambda *a: print(*a, flush=True))
    assert abs(got["trained"][0] - 0.6931472) < 1e-5  # equal policies: log 2
    assert got["trained"][-1] < got["trained"][0]
    assert got["policy"][1] < got["policy"][0]
    xp, fp = got["curve"]
    assert bool((xp.diff() > 0).all()) and bool((fp.diff() >= 0).all()) and 0 <= float(fp[0]) and float(fp[-1]) <= 1
    assert got["brier"][1] <= got["brier"][0]  # the least-squares curve over the same pairs
