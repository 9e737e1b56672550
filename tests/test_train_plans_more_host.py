"""The sequence operators' planners on the host, over their whole range of sizes, built with the
signed-overflow sanitizer: no plan's arithmetic overflows, and every launch is one that a GPU takes.  No
GPU: a plan is made for a described device (152 SMs)."""
import concurrent.futures as cf
import os
import shutil
import subprocess

import pytest

from implicit_gemm_conv2d_gb300 import build

from .test_train_plans_host import SANITIZE

SOURCES = ["kernels_scan.cu", "kernels_distill.cu", "kernels_ln.cu"]
MAIN = r"""
#include <cstdio>
#include "train_internal.h"
using namespace igc;

int main()
{
    DevInfo d;
    d.device = 0; d.sms = 152; d.smem_optin = 227 * 1024; d.cc_major = 10; d.cc_minor = 3;
    const int64_t most = (int64_t(1) << 31) - 1, last = most - (1 << 20);
    long plans = 0;
    for (int64_t B : {int64_t(1), int64_t(3), int64_t(152), int64_t(32768), int64_t(1) << 24, last})
        for (int64_t T : {int64_t(0), int64_t(1), int64_t(2), int64_t(8), int64_t(9), int64_t(77), int64_t(1024),
                          int64_t(65537), int64_t(1) << 27, last})
            for (int64_t D : {int64_t(1), int64_t(2), int64_t(31), int64_t(128), int64_t(1024), int64_t(4099),
                              int64_t(1) << 20, int64_t(1) << 28, last}) {
                if (B * D >= int64_t(1) << 37 || double(B) * double(T) * double(D) > 1.6e11) continue;
                for (int dt : {0, 1})
                    for (int64_t gap : {0, 1, 16}) {
                        conv_rows_t r = {T * (D + gap), D + gap};
                        conv_scan_desc_t e = {int32_t(B), int32_t(T), int32_t(D), dt, r, r, r, r, r, r};
                        for (bool bwd : {false, true}) {
                            for (int chunk : {dt ? 2 : 4, 8, 16}) {
                                const ScanPlan p = scan_plan(e, d, bwd, chunk);
                                if (p.blocks < 0 || p.blocks > most || p.threads < 0 || p.threads > 1024) return 1;
                                if (!p.walk && T > 0 && (p.cluster < 1 || p.cluster > 8)) return 2;
                                ++plans;
                            }
                            if (scan_workspace(e, d, bwd) > size_t(1) << 40) return 3;
                        }
                    }
            }
    for (int64_t N : {int64_t(1), int64_t(7), int64_t(153), int64_t(50021), (int64_t(1) << 27) - 1})
        for (int V : {1, 2, 3, 127, 128, 1000, 2049, 50021, 131071, 800003, 1 << 24, (1 << 30) - 1})
            for (int K : {1, 2, 33, 64, 257, 1024})
                for (int dt : {0, 1})
                    for (int it : {0, 1})
                        for (int64_t ld : {int64_t(V), int64_t(V) + 1, (int64_t(1) << 32) - 1}) {
                            if (double(N) * double(ld) > 1.6e11) continue;
                            conv_distill_desc_t e = {N, ld, V, K, dt, it, 0, 1.f};
                            for (int mode : {0, 1, 2}) {
                                const DistillPlan p = distill_plan(e, d, mode);
                                if (p.blocks < 1 || p.blocks > most || p.threads < 32 || p.threads > 1024) return 4;
                                if (p.smem < 0 || p.smem + 1024 > d.smem_optin) return 5;
                                ++plans;
                            }
                        }
    for (int64_t N : {int64_t(0), int64_t(1), int64_t(7), int64_t(153), int64_t(39001), int64_t(1) << 27, most})
        for (int D : {1, 2, 7, 8, 128, 1023, 1024, 4097, 8192, 8193, 50021, 1 << 20, (1 << 30) - 1})
            for (int dt : {0, 1})
                for (int rms : {0, 1}) {
                    if (double(N) * double(D) > 1.6e11) continue;
                    conv_ln_desc_t e = {N, D, rms, dt, 1e-5f};
                    for (bool bwd : {false, true}) {
                        const LnParams p = ln_plan(e, d, bwd);
                        if (N > 0 && (p.blocks < 1 || p.TL < 1 || int64_t(p.TL) * p.teams > 1024)) return 6;
                        ++plans;
                    }
                    if (ln_bwd_workspace(e, d) > size_t(1) << 42) return 7;
                }
    std::printf("%ld plans\n", plans);
    return 0;
}
"""


def test_plans_do_not_overflow(tmp_path):
    probe = tmp_path / "probe.cpp"
    probe.write_text("int main() { return 0; }")
    if not shutil.which("g++") or subprocess.run(["g++", "-fsanitize=signed-integer-overflow", str(probe), "-o",
                                                  str(tmp_path / "probe")], capture_output=True).returncode:
        pytest.skip("no sanitizer runtime")
    main = tmp_path / "plans_main.cu"
    main.write_text(MAIN)
    cc = build.nvcc()
    common = [cc, *build.ARCH, "-O0", "-Xcicc", "-O0", "-Xptxas", "-O0", "-std=c++17", "--expt-relaxed-constexpr",
              "-I", build.CSRC, "-I", build.INCLUDE, *SANITIZE]

    def compile_one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run(common + ["-c", src, "-o", obj], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return obj

    with cf.ThreadPoolExecutor(max_workers=4) as ex:
        objs = list(ex.map(compile_one, [str(main)] + [os.path.join(build.CSRC, s) for s in SOURCES]))
    exe = str(tmp_path / "plans")
    r = subprocess.run([cc, *build.ARCH, *objs, "-o", exe, "-cudart", "static", *SANITIZE, "-lubsan"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert int(r.stdout.split()[0]) > 3000
