"""What the sequence operators' plans promise to their launches, over their whole range of sizes and for rows that
begin at each alignment: a workspace that holds the pieces of time, the widths of copies that are compiled, and no
chain of additions longer than 256 vectors.  No GPU: a plan is made for a described device (152 SMs)."""
import concurrent.futures as cf
import os
import subprocess

import pytest

from implicit_gemm_conv2d_gb300 import build

SOURCES = ["kernels_scan.cu", "kernels_distill.cu", "kernels_ln.cu"]
MAIN = r"""
#include <cstdio>
#include "train_internal.h"
using namespace igc;

int main()
{
    DevInfo d;
    d.device = 0; d.sms = 152; d.smem_optin = 227 * 1024; d.cc_major = 10; d.cc_minor = 3;
    long pieces = 0, windows = 0, chains = 0;
    for (int64_t B : {1, 2, 3, 5, 40, 152, 3000, 32768})
        for (int64_t T : {1, 16, 17, 77, 1024, 2049, 5000, 9001, 20011, 55388, 65537, 1 << 22})
            for (int64_t D : {1, 6, 8, 9, 24, 31, 33, 70, 128, 260, 333, 777, 1022, 1024, 4099, 1 << 20}) {
                if (double(B) * double(T) * double(D) > 1.6e11) continue;
                for (int dt : {0, 1})
                    for (bool bwd : {false, true}) {
                        const int es = dt ? 2 : 4;
                        const conv_rows_t r = {T * D, D};
                        conv_scan_desc_t e = {int32_t(B), int32_t(T), int32_t(D), dt, r, r, r, r, r, r};
                        const size_t room = scan_workspace(e, d, bwd);
                        for (int chunk = es; chunk <= 16; chunk *= 2) {
                            const ScanPlan p = scan_plan(e, d, bwd, chunk);
                            if (p.pieces > 1) {
                                ++pieces;
                                if (size_t(p.pieces + 1) * size_t(B) * size_t(D) * 8 > room) return 1;
                                if (p.walk || p.cluster != 1) return 2;
                                if (int64_t(p.pieces) * p.piece < T || int64_t(p.pieces - 1) * p.piece >= T) return 3;
                                if (p.window && p.CB != 2) return 4;  // those that are compiled for pieces
                            }
                            if (p.walk) {
                                if (p.V * es > chunk || (p.V == 2 && D % 2 != 0)) return 5;
                                if (p.ring > 0 && es == 2 && p.V == 1) return 6;
                                continue;
                            }
                            if (p.CB > chunk && !(chunk < 2 * es && p.CB == es)) return 7;
                            if (p.window) {
                                ++windows;
                                if (bwd && es == 2) return 8;
                                if (p.CB != es && p.CB != 2 * es) return 9;
                            } else if (p.CB != 16 && p.CB != 4 && !(es == 2 && p.CB == 2)) {
                                return 10;
                            }
                        }
                    }
            }
    for (int64_t N : {int64_t(1), int64_t(24), int64_t(400), int64_t(8192), int64_t(1) << 20})
        for (int V : {1, 128, 2049, 50021, 1000003, 4000037, 4300001, 1 << 24, (1 << 30) - 1})
            for (int K : {1, 64, 1024})
                for (int dt : {0, 1})
                    for (int mode : {0, 1, 2}) {
                        if (double(N) * V > 1.6e11) continue;
                        conv_distill_desc_t e = {N, V, V, K, dt, 0, 0, 1.f};
                        const DistillPlan p = distill_plan(e, d, mode);
                        if (p.chains) {
                            ++chains;
                            if (p.warp || mode == 1 || p.stage_bytes > 0) return 11;
                        } else if (mode != 1) {
                            const int64_t vecs = int64_t(V) / (dt ? 8 : 4) / p.cluster;
                            if (vecs / (p.warp ? 32 : p.warps * 32) > 256) return 12;
                        }
                    }
    for (int64_t N : {int64_t(1), int64_t(153), int64_t(39001), int64_t(1) << 24})
        for (int D = 1; D < 70000; D += D < 300 ? 1 : D / 5 + 1)
            for (int dt : {0, 1})
                for (bool bwd : {false, true}) {
                    conv_ln_desc_t e = {N, D, 0, dt, 1e-5f};
                    const LnParams p = ln_plan(e, d, bwd);
                    if (p.NV == 0) continue;
                    if (p.edge && p.NV == 1 && !(bwd && dt)) return 13;  // not compiled
                    if (p.NV > (bwd ? (dt ? 2 : 4) : 8) || (p.NV & (p.NV - 1))) return 14;
                }
    if (pieces < 100 || windows < 100 || chains < 10) return 15;
    std::printf("%ld %ld %ld\n", pieces, windows, chains);
    return 0;
}
"""


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    folder = tmp_path_factory.mktemp("plans")
    main = folder / "main.cu"
    main.write_text(MAIN)
    cc = build.nvcc()
    common = [cc, *build.ARCH, "-O0", "-Xcicc", "-O0", "-Xptxas", "-O0", "-std=c++17", "--expt-relaxed-constexpr",
              "-I", build.CSRC, "-I", build.INCLUDE]

    def one(src):
        obj = str(folder / (os.path.basename(src) + ".o"))
        r = subprocess.run(common + ["-c", src, "-o", obj], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return obj

    with cf.ThreadPoolExecutor(max_workers=4) as ex:
        objs = list(ex.map(one, [str(main)] + [os.path.join(build.CSRC, s) for s in SOURCES]))
    exe = str(folder / "plans")
    r = subprocess.run([cc, *build.ARCH, *objs, "-o", exe, "-cudart", "static"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def test_plans_keep_their_promises(compiled):
    r = subprocess.run([compiled], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout)
