"""The selective block's operators and the loss over a vocabulary in the bounds-checked build: no index
check fails, and every result is within its type's tolerance of the float64 definition: 1e-5, and an
output stored in 16 bits its rounding (the loss's gradients have a second one, of d, held to what its
terms may add up to). In a child process, as test_gpu_bounds.py."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_index_check_fails_and_results_match():
    env = dict(os.environ, DLR_BOUNDS_CHECK="1")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "ssm_bounds_cases.py")], env=env,
                       capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stderr[-4000:]
    result = json.loads(r.stdout.strip().splitlines()[-1])
    assert result["checked"] is True
    assert len(result["cases"]) == 45 + 45 + 24
    for name, err, status, site in result["cases"]:
        assert status == 0 and site == 0, f"{name}: status {status}, site {site}"
        tol = 1e-5 + (2.0 ** -8 if "bfloat16" in name else 2.0 ** -11 if "float16" in name else 0)
        assert err <= tol, f"{name}: rel L2 {err:.3e}"
