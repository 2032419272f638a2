"""First calls from several threads at once: what the library looks up once is there for every one of them."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NVCC = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"

# The runtime's lookup stands here in its place and takes its time.
PROGRAM = r"""
#include <cuda_runtime.h>
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>
#include "pipeline.cuh"

static int target;
extern "C" cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned, unsigned long long,
                                                        cudaDriverEntryPointQueryResult* result) {
    std::this_thread::sleep_for(std::chrono::milliseconds(200));
    *fn = &target;
    *result = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}

int main() {
    std::atomic<int> waiting{8}, missing{0};
    std::vector<std::thread> all;
    for (int i = 0; i < 8; ++i)
        all.emplace_back([&] {
            --waiting;
            while (waiting > 0) {}
            if (!gai4::encode_fn()) ++missing;
        });
    for (auto& t : all) t.join();
    std::printf("%d without it\n", missing.load());
    return missing.load();
}
"""


@pytest.mark.skipif(not os.path.exists(NVCC), reason="needs nvcc")
def test_tensor_map_entry_is_found_by_every_thread(tmp_path):
    (tmp_path / "first.cu").write_text(PROGRAM)
    program = str(tmp_path / "first")
    lib = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(NVCC))), "lib64")
    subprocess.run([NVCC, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-cudart", "shared", "-I",
                    os.path.join(ROOT, "gemm_affine_int4_gb300", "csrc"), str(tmp_path / "first.cu"), "-o", program,
                    "-Xlinker", "-rpath," + lib], check=True, capture_output=True)
    done = subprocess.run([program], capture_output=True, text=True, timeout=60)
    assert done.returncode == 0, done.stdout + done.stderr
