"""The training-step operators' planners on the host, over their whole range of sizes, built with the
signed-overflow sanitizer: no plan's arithmetic overflows.  No GPU: a plan is made for a described
device (152 SMs); the asked occupancy falls back to the SMs' count where there is none."""
import concurrent.futures as cf
import os
import shutil
import subprocess

import pytest

from implicit_gemm_conv2d_gb300 import build

SOURCES = ["kernels_embed.cu", "kernels_gn_fwd.cu", "kernels_gn_bwd.cu", "kernels_gn_cluster.cu", "kernels_gn_nhwc.cu",
           "kernels_grad.cu"]
MAIN = r"""
#include <cstdio>
#include <vector>
#include "train_internal.h"
using namespace igc;

int main()
{
    DevInfo d;
    d.device = 0; d.sms = 152; d.smem_optin = 227 * 1024; d.cc_major = 10; d.cc_minor = 3;
    const int64_t most = (int64_t(1) << 31) - 1;
    long plans = 0;
    for (int64_t T : {int64_t(1), int64_t(7), int64_t(512), int64_t(513), int64_t(65536), int64_t(65537),
                      int64_t(1540096), int64_t(100000003), most - (1 << 20)})
        for (int64_t V : {int64_t(1), int64_t(128), int64_t(300), int64_t(1799), int64_t(50021), int64_t(1) << 25, most})
            for (int D : {1, 2, 3, 32, 37, 1024, 1088, 4096, 1 << 20, (1 << 24) - 1, 1 << 24})
                for (int dt : {0, 1})
                    for (int it : {0, 1}) {
                        conv_embed_desc_t e = {T, int32_t(V), D, -1, it, dt, 1.f};
                        if (embed_bwd_workspace(e, d) > size_t(-1) / 2) return 1;
                        ++plans;
                    }
    const int64_t last = most - (1 << 20);
    for (int64_t C : {int64_t(1), int64_t(2), int64_t(27), int64_t(128), int64_t(320), int64_t(2051), int64_t(4096),
                      int64_t(65536), last - 1, last})
        for (int64_t P : {int64_t(1), int64_t(2), int64_t(12), int64_t(165), int64_t(5184), int64_t(1) << 20, last / C})
            for (int64_t G : {int64_t(1), int64_t(2), int64_t(3), int64_t(16), int64_t(32), C})
                for (int64_t B : {int64_t(1), int64_t(24), int64_t(32768), int64_t(100000007), most - (1 << 25)}) {
                    if (P < 1 || C * P > last || C % G != 0 || B * G > most) continue;
                    if (double(B) * double(C) * double(P) > 1.6e11) continue;  // no memory holds it
                    for (int layout : {0, 1})
                        for (int dt : {0, 1}) {
                            GnParams p;
                            p.B = int(B); p.C = int(C); p.P = int(P); p.G = int(G); p.Cg = int(C / G);
                            p.act = 0; p.layout = layout; p.M = C / G * P; p.N = C * P;
                            p.eps = 1e-5f; p.m = float(p.M); p.inv_m = float(1.0 / double(p.M));
                            if (gn_fwd_workspace(p, dt, d) > size_t(-1) / 2) return 2;
                            if (gn_bwd_workspace(p, dt, d) > size_t(-1) / 2) return 3;
                            ++plans;
                        }
                }
    std::vector<conv_grad_t> g;
    for (int64_t n : {int64_t(0), int64_t(1), int64_t(16384), int64_t(400000000), (int64_t(1) << 40) - 1}) {
        g.push_back({nullptr, nullptr, n, 0});
        g.insert(g.end(), 600, {nullptr, nullptr, n, 1});
        if (grad_workspace(g.data(), int(g.size()), d) > size_t(-1) / 2) return 4;
        ++plans;
    }
    std::printf("%ld plans\n", plans);
    return 0;
}
"""
SANITIZE = ["-Xcompiler", "-fsanitize=signed-integer-overflow,-fno-sanitize-recover=all"]


def test_plans_do_not_overflow(tmp_path):
    probe = tmp_path / "probe.cpp"
    probe.write_text("int main() { return 0; }")
    flags = ["-fsanitize=signed-integer-overflow"]
    if not shutil.which("g++") or subprocess.run(["g++", *flags, str(probe), "-o", str(tmp_path / "probe")],
                                                 capture_output=True).returncode:
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

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, [str(main)] + [os.path.join(build.CSRC, s) for s in SOURCES]))
    exe = str(tmp_path / "plans")
    r = subprocess.run([cc, *build.ARCH, *objs, "-o", exe, "-cudart", "static", *SANITIZE, "-lubsan"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert int(r.stdout.split()[0]) > 3000
