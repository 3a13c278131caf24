"""The suite's own rules."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_fake_pointers_stay_off_a_device():
    """With a CUDA device the host executor's tests are skipped: the calls that pass their checks would go on to it."""
    run = ("import sys, torch, pytest; torch.cuda.is_available = lambda: True; "
           "sys.exit(pytest.main(['-q', '-p', 'no:cacheprovider', 'tests/test_host_executor.py']))")
    r = subprocess.run([sys.executable, "-c", run], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and "skipped" in r.stdout and "passed" not in r.stdout and "failed" not in r.stdout, r.stdout
