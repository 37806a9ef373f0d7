"""The operators around residual blocks after cudaDeviceReset, in a process of their own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_operators_after_a_device_reset():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from zero_sharded_mixed_02_gb300 import build
    build.build()
    program = os.path.join(os.path.dirname(os.path.abspath(__file__)), "reset_check.py")
    r = subprocess.run([sys.executable, program], capture_output=True, text=True, timeout=300)
    if r.returncode == 77:
        pytest.skip(r.stdout.strip())
    assert r.returncode == 0 and r.stdout.strip() == "OK", (r.returncode, r.stdout, r.stderr[-2000:])
