"""Two threads that raise one kernel's dynamic shared memory limit (csrc/dyn_smem.h), on the
host with stand-ins for the two CUDA calls: the larger size stays, whichever comes first."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_routed_b200", "csrc")
CUDA_INCLUDE = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")

PROGRAM = r"""
#include <stdio.h>
#include <chrono>
#include <thread>
#include "dyn_smem.h"

static std::atomic<int> limit{0}, calls{0}, entered{0};
static void pause(int ms) { std::this_thread::sleep_for(std::chrono::milliseconds(ms)); }

extern "C" cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
// The call for the smaller size takes effect late.
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int bytes) {
    entered++;
    if (bytes == 50000) pause(300);
    limit = bytes;
    calls++;
    return cudaSuccess;
}

static void kernel() {}

int main() {
    static moe::SmemSet set;
    int ok = 0;
    std::thread small([&] { ok += moe::ensure_dyn_smem(kernel, 50000, set) == cudaSuccess; });
    while (!entered) pause(1);
    std::thread large([&] { moe::ensure_dyn_smem(kernel, 100000, set); });
    small.join();
    large.join();
    const int raised = limit;
    moe::ensure_dyn_smem(kernel, 70000, set);  // not lowered, no call
    printf("%d %d %d %d\n", ok, raised, (int)limit, (int)calls);
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(CUDA_INCLUDE, "cuda_runtime.h")),
                    reason="needs g++ and CUDA's headers")
def test_the_larger_limit_stays(tmp_path):
    src, exe = tmp_path / "smem.cpp", tmp_path / "smem"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-pthread", "-I", CSRC, "-I", CUDA_INCLUDE, str(src), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0
    assert out.stdout.split() == ["1", "100000", "100000", "2"]
