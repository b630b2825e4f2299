"""Products whose blocks of a cluster share K store nothing where one of them has given up a wait: the
cases of tests/serving_debug_cases.py, in a child process that loads the debug build."""
import os
import subprocess
import sys

import pytest

from rmsnorm_fwd_bwd_gb300 import build as build_mod

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_cluster_with_a_block_that_gave_up_stores_nothing():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, RMSNORM_LIBRARY=build_mod.build(debug=True))
    res = subprocess.run([sys.executable, "-m", "tests.serving_debug_cases"], cwd=ROOT, env=env, capture_output=True, text=True,
                         timeout=900)
    print(res.stdout[-3000:], res.stderr[-3000:])
    assert res.returncode == 0
