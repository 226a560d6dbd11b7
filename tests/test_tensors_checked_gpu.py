"""The tests of the step over a list of tensors again, through the
bounds-checked debug build: its kernels check that every tile lies in its
tensor, and the conftest fixture fails a test that leaves a record."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHECKED = os.path.join(ROOT, "mixed_precision_adam_gb300", "lib", "libdopt_checked.so")


def test_list_steps_under_the_bounds_checked_build():
    assert os.path.exists(CHECKED)
    out = subprocess.run([sys.executable, "-m", "pytest", os.path.join(ROOT, "tests", "test_tensors_gpu.py"), "-q", "-x",
                          "-m", "gpu", "-p", "no:cacheprovider"],
                         cwd=ROOT, env=dict(os.environ, DOPT_LIBRARY=CHECKED), capture_output=True, text=True, timeout=900)
    assert out.returncode == 0, out.stdout[-4000:] + out.stderr[-2000:]
    assert " passed" in out.stdout
