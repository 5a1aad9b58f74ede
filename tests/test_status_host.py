"""A refused launch does not fail the thread's next call (csrc/status.h), on the host with a
stand-in for CUDA's last error; no entry point returns the CUDA status past it."""

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_expert_routed_b200", "csrc")
CUDA_INCLUDE = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")

PROGRAM = r"""
#include <stdio.h>
#include "status.h"

static cudaError_t last = cudaSuccess;
extern "C" cudaError_t cudaGetLastError() {
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}
static cudaError_t refused() { return last = cudaErrorInvalidValue; }
static cudaError_t launched() { return cudaGetLastError(); }

int main() {
    const moe_status a = moe::status_of(launched());
    const moe_status b = moe::status_of(refused());  // returned without asking for the last error
    const moe_status c = moe::status_of(launched());
    printf("%d %d %d\n", (int)a, (int)b, (int)c);
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(CUDA_INCLUDE, "cuda_runtime.h")),
                    reason="needs g++ and CUDA's headers")
def test_an_error_is_reported_once(tmp_path):
    src, exe = tmp_path / "status.cpp", tmp_path / "status"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-I", CSRC, "-I", os.path.join(ROOT, "include"), "-I", CUDA_INCLUDE,
                           str(src), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and out.stdout.split() == ["0", "4", "0"]


def test_entry_points_report_through_it():
    """MOE_ERR_CUDA stands in status.h, in its name's text and in the report of the device's own error word."""
    found = []
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            found += [(name, line.strip()) for line in f if re.search(r"\bMOE_ERR_CUDA\b", line)]
    assert [f for f in found if f[0] != "status.h"] == [
        ("api.cu", 'case MOE_ERR_CUDA: return "CUDA error";'), ("api.cu", "if (w & ERR_INTERNAL) return MOE_ERR_CUDA;")]
