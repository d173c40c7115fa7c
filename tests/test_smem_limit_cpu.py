"""Two host threads that raise one kernel's shared-memory limit at once (csrc/internal.h against a fake CUDA runtime)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.path.join(os.path.dirname(os.path.dirname(os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc"))), "include")

PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include "internal.h"

std::atomic<int> limit{0};          // the kernel's attribute
std::atomic<bool> small_in{false}, large_done{false};

extern "C" cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int value) {
    if (value == 1000) {            // the smaller caller is slow: it waits for the larger one, half a second at most
        small_in = true;
        for (int i = 0; i < 500 && !large_done; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
    }
    limit = value;
    return cudaSuccess;
}

int main() {
    static int done[kvc::kMaxDevices];
    std::thread small([&] { kvc::dyn_smem_at_least(nullptr, 1000, done); });
    std::thread large([&] {
        while (!small_in) std::this_thread::yield();
        kvc::dyn_smem_at_least(nullptr, 2000, done);
        large_done = true;
    });
    small.join();
    large.join();
    std::printf("%d\n", (int)limit);  // what the larger caller launches under now
    return limit >= 2000 ? 0 : 1;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(CUDA, "cuda_runtime.h")),
                    reason="needs g++ and CUDA's headers")
def test_the_larger_limit_stays(tmp_path):
    src, exe = tmp_path / "limit.cpp", tmp_path / "limit"
    src.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "agent_kv_cache_lse_b200", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", f"-I{csrc}", f"-I{CUDA}", str(src), "-o", str(exe)], check=True,
                   capture_output=True, text=True)
    for _ in range(3):
        run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
        assert run.returncode == 0, f"limit at the larger launch: {run.stdout}"
