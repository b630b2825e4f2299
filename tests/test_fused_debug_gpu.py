"""The residual addition's backward through the debug build (-DRMSNORM_DEBUG), whose TMA
copies are checked against the tensors they read: the tests with enough rows for its
ring, in a child process that loads that library, and the device error word after
them."""
import os
import subprocess
import sys

import pytest

from rmsnorm_fwd_bwd_gb300 import build as build_mod

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_ring_reads_stay_inside_their_tensors():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, RMSNORM_LIBRARY=build_mod.build(debug=True))
    res = subprocess.run([sys.executable, "-m", "pytest", "tests/test_fused_gpu.py", "-q", "-x", "-m", "gpu", "-k",
                          "add_bwd_many_rows or no_device_error"], cwd=ROOT, env=env, capture_output=True, text=True,
                         timeout=900)
    print(res.stdout[-3000:], res.stderr[-1000:])
    assert res.returncode == 0
