"""A memset that fails in an entry point is reported by that call and leaves
no error for the next one; against a stand-in for the runtime."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixed_precision_adam_gb300", "csrc")
CUDA = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")

PROGRAM = """
#include <cstdio>
#include "memset.h"
static cudaError_t last = cudaSuccess;
extern "C" cudaError_t CUDARTAPI cudaGetLastError(void) { const cudaError_t e = last; last = cudaSuccess; return e; }
extern "C" const char* CUDARTAPI cudaGetErrorString(cudaError_t) { return "because"; }
static std::string message;
namespace dopt { int fail(int status, const std::string& text) { message = text; return status; } }
int main() {
  if (dopt::check_memset(cudaSuccess, "call: ") != DOPT_OK || !message.empty()) return 1;
  last = cudaErrorInvalidValue;
  if (dopt::check_memset(last, "call: ") != DOPT_E_CUDA || message != "call: because") return 2;
  return cudaGetLastError() == cudaSuccess ? 0 : 3;
}
"""


def test_a_failed_memset_leaves_no_error(tmp_path):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(CUDA, "cuda_runtime_api.h")):
        pytest.skip("no C++ compiler or no CUDA headers")
    (tmp_path / "m.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, "-I", os.path.join(ROOT, "include"), "-I", CUDA, str(tmp_path / "m.cpp"), "-o",
                    str(tmp_path / "m")], check=True)
    assert subprocess.run([str(tmp_path / "m")]).returncode == 0
    # and every memset of the operators' entry points goes through it
    for name in ("matrix8_multiply.cu", "rms_norm.cu"):
        text = open(os.path.join(CSRC, name)).read()
        assert text.count("check_memset(cudaMemset") == text.count("cudaMemset") > 0
