"""The Muon step's kernels in the index-checking debug build, and the example."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_debug_build_scenarios():
    r = subprocess.run([sys.executable, os.path.join(HERE, "muon_debug_scenario.py")], capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    assert r.stdout.strip().splitlines()[-1].endswith("ok"), r.stdout[-2000:]


def test_example_learns():
    sys.path.insert(0, os.path.join(os.path.dirname(HERE), "examples"))
    from train_muon import train
    losses = train(steps=40)
    # it starts near 2 (two independent outputs of equal size) and falls well below the target's own size
    assert losses[0] > 1.0 and losses[-1] < 0.5 * losses[0], losses
    assert losses == train(steps=40), "a run repeats bit for bit"
