"""The products' split and paired forms and several batches in the index-checking debug build."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_debug_build_scenarios():
    r = subprocess.run([sys.executable, os.path.join(HERE, "muon_debug_products_scenario.py")], capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    assert r.stdout.strip().splitlines()[-1].endswith("ok"), r.stdout[-2000:]
