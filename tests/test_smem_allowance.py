"""CPU test of the shared-memory allowance that the launchers keep for a kernel: of two threads that
raise it at the same time the larger size has to stand, since later launches rely on the record."""
import os
import subprocess

from pagedattention_paged_kv_gb300 import _build

PROGRAM = r"""
#include <cuda_runtime.h>
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

static std::atomic<int> attribute{0}, small_is_in{0}, large_was_set{0};
static cudaError_t fake_device(int *d) { *d = 0; return cudaSuccess; }
template <typename K>
static cudaError_t fake_set(K, cudaFuncAttribute, int bytes) {
    if (bytes == 1000) {  // the smaller size: give the larger half a second to get ahead
        small_is_in = 1;
        for (int i = 0; i < 500 && !large_was_set; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
    }
    attribute = bytes;
    if (bytes == 2000) large_was_set = 1;
    return cudaSuccess;
}
#define cudaGetDevice fake_device
#define cudaFuncSetAttribute fake_set
#include "attn_block.cuh"

static void kernel() {}

int main() {
    static pkv::SmemAllowance allowed;
    std::thread small([] { pkv::allow_dynamic_smem(kernel, 1000, allowed); });
    while (!small_is_in) std::this_thread::yield();
    std::thread large([] { pkv::allow_dynamic_smem(kernel, 2000, allowed); });
    small.join();
    large.join();
    printf("%d %d\n", attribute.load(), allowed.bytes[0].load());
    pkv::allow_dynamic_smem(kernel, 1500, allowed);
    printf("%d\n", attribute.load());
    return 0;
}
"""


def test_the_larger_of_two_sizes_stands(tmp_path):
    src, exe = tmp_path / "allowance.cu", tmp_path / "allowance"
    src.write_text(PROGRAM)
    subprocess.run([_build._nvcc(), *_build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", _build.CSRC, "-I",
                    _build.INCLUDE, "-o", str(exe), str(src), "-Xcompiler", "-pthread"], check=True,
                   capture_output=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=30,
                         env={**os.environ, "CUDA_VISIBLE_DEVICES": ""}).stdout.split()
    assert out == ["2000", "2000", "2000"], out
