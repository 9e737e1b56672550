"""The opt-in to large shared memory with several host threads: whatever their order, a size that was once
granted stays granted.  No GPU: the runtime's two calls are this test's own."""
import subprocess

from implicit_gemm_conv2d_gb300 import build

MAIN = r"""
#include <atomic>
#include <chrono>
#include <thread>
#include "internal.h"

extern std::atomic<int> limit, device, calls;
extern std::atomic<bool> together;
void kernel() {}

int main()
{
    using igc::ensure_smem;
    if (ensure_smem<kernel>(48 * 1024) != cudaSuccess || calls != 0) return 1;
    std::thread large([] { ensure_smem<kernel>(100 * 1024); });
    std::this_thread::sleep_for(std::chrono::milliseconds(100));
    std::thread small([] { ensure_smem<kernel>(60 * 1024); });
    large.join();
    small.join();
    if (ensure_smem<kernel>(100 * 1024) != cudaSuccess || limit < 100 * 1024) return 2;
    if (together) return 3;
    const int before = calls;
    if (ensure_smem<kernel>(90 * 1024) != cudaSuccess || calls != before || limit < 100 * 1024) return 4;
    if (ensure_smem<kernel>(120 * 1024) != cudaSuccess || limit != 120 * 1024) return 5;
    device = 1;  // a device of its own
    if (ensure_smem<kernel>(70 * 1024) != cudaSuccess || limit != 70 * 1024) return 6;
    device = 64;  // one beyond those that the library runs on
    return ensure_smem<kernel>(80 * 1024) == cudaErrorInvalidDevice ? 0 : 7;
}
"""
# The larger size takes effect at once and returns late, so that the smaller one's call falls between.
RUNTIME = r"""
#include <atomic>
#include <chrono>
#include <thread>

std::atomic<int> limit{0}, device{0}, calls{0}, inside{0};
std::atomic<bool> together{false};

extern "C" {
int cudaGetDevice(int* d)
{
    *d = device;
    return 0;
}
int cudaFuncSetAttribute(const void*, int, int bytes)
{
    if (inside.fetch_add(1) != 0) together = true;
    ++calls;
    limit = bytes;
    if (bytes == 100 * 1024) std::this_thread::sleep_for(std::chrono::milliseconds(300));
    --inside;
    return 0;
}
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
char __cudaInitModule(void**) { return 1; }
}
"""


def test_a_granted_size_is_not_taken_back(tmp_path):
    main, runtime = tmp_path / "main.cu", tmp_path / "runtime.cpp"
    main.write_text(MAIN)
    runtime.write_text(RUNTIME)
    exe = str(tmp_path / "main")
    r = subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", build.CSRC, "-I",
                        build.INCLUDE, "-cudart", "none", str(main), str(runtime), "-o", exe, "-Xlinker", "-lpthread"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([exe], timeout=60).returncode == 0
