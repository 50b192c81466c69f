"""The limit of a kernel's dynamic shared memory (not gpu): host threads that launch one
kernel with different sizes raise it and never lower it.  The library's own header is
compiled with a stand-in for the runtime's attribute."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exl3_trellis_weight_gb300", "csrc")

PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>
#include "smem_limit.cuh"

static exl3::SmemLimits limits;
static std::atomic<int> attribute[2][2];          // kernel, device

static void wait_for(int value) {
    for (int i = 0; attribute[0][0] != value && i < 200; i++)
        std::this_thread::sleep_for(std::chrono::milliseconds(1));
}

// a launch: it fails when the attribute is below its size.  before, after: what the first
// kernel's attribute on the first device should be around the setting, if it comes to that
static bool launch(int kernel, int dev, int bytes, int before = 0, int after = 0) {
    const int e = limits.raise(&attribute[kernel], dev, bytes, [&] {
        if (before)
            wait_for(before);
        attribute[kernel][dev] = bytes;
        if (after) {
            wait_for(after);
            std::this_thread::sleep_for(std::chrono::milliseconds(20));
        }
        return 0;
    });
    return e == 0 && attribute[kernel][dev].load() >= bytes;
}

int main() {
    // the smaller size is set behind the larger one, and noted first, wherever the code lets it
    bool a = true, b = true;
    std::thread s([&] { b = launch(0, 0, 50, 100); });
    std::thread l([&] { a = launch(0, 0, 100, 0, 50); });
    s.join();
    l.join();
    if (!a || !b || !launch(0, 0, 100))
        return std::printf("a smaller size lowered the limit: %d\n", attribute[0][0].load()), 1;
    // many threads, sizes, kernels and devices
    std::atomic<int> failed{0};
    std::vector<std::thread> all;
    for (int t = 0; t < 8; t++)
        all.emplace_back([&, t] {
            for (int i = 0; i < 20000; i++)
                if (!launch(1 - (i & 1), t & 1, 100 + (i * 7919 + t * 104729) % 200 + i / 100))
                    failed++;
        });
    for (auto &t : all)
        t.join();
    if (failed)
        return std::printf("%d launches below their size\n", failed.load()), 1;
    // an error is handed on and leaves the limit to be set again
    if (limits.raise(&all, 0, 7, [] { return 3; }) != 3)
        return 1;
    int set = 0;
    return limits.raise(&all, 0, 7, [&] { return set++; }) == 0 && set == 1 &&
           limits.raise(&all, 0, 7, [&] { return set++; }) == 0 && set == 1 ? 0 : 1;
}
"""


def test_threads_never_lower_a_kernels_limit(tmp_path):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "limit.cpp", tmp_path / "limit"
    src.write_text(PROGRAM)
    subprocess.run([cc, "-std=c++17", "-O1", "-pthread", "-I", CSRC, "-x", "c++", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def test_every_product_kernel_goes_through_it():
    """No launch of the products sets the attribute by itself."""
    for name in sorted(os.listdir(CSRC)):
        if name.startswith("linear"):
            with open(os.path.join(CSRC, name)) as f:
                assert "cudaFuncAttributeMaxDynamicSharedMemorySize" not in f.read(), name
