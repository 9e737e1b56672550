"""The kernels of the training-step operators are launched to overlap the kernel before them on the
stream, and only their wait for it (grid_dep_wait) makes what that one and those before it wrote
visible.  So no kernel reads or writes global memory in front of its wait: checked in the source."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "implicit_gemm_conv2d_gb300", "csrc")
FILES = [os.path.basename(f) for p in ("kernels_gn_*.cu", "kernels_embed.cu", "kernels_grad.cu")
         for f in sorted(glob.glob(os.path.join(CSRC, p)))]
WAIT = "tc::grid_dep_wait()"


def closing(text, at, pair="{}"):
    """The index behind the bracket that closes the one at ``at``."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i + 1
    raise AssertionError("unbalanced source")


def kernels(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\s*\([^;{]*?\)\s+)?(\w+)\s*\(", text):
        end = closing(text, m.end() - 1, "()")
        body = text.index("{", end)
        yield m.group(1), text[m.end():end - 1], text[body:closing(text, body)]


def without_lambdas(body):
    """The body without the lambdas that it names: their code runs where they are called."""
    while True:
        m = re.search(r"auto\s+\w+\s*=\s*\[&\]\s*\([^)]*\)\s*\{", body)
        if not m:
            return body
        body = body[:m.start()] + body[closing(body, m.end() - 1):]


@pytest.mark.parametrize("name", FILES)
def test_global_memory_is_touched_behind_the_wait(name):
    found = list(kernels(name))
    assert found
    for kernel, params, body in found:
        pointers = re.findall(r"\*\s*(?:__restrict__\s+)?(\w+)\s*(?:,|$)", params)
        if not pointers:
            continue
        body = without_lambdas(body)
        assert WAIT in body, f"{kernel} has no wait"
        front = body[:body.index(WAIT)]
        for p in pointers:
            use = re.search(rf"\b{p}\s*\[|\b(?:ld|ldg|st|load|store)\s*\(\s*{p}\b|\(\s*{p}\s*,|\*\s*{p}\b", front)
            assert not use, f"{kernel}: {p} is used in front of the wait: {use.group(0)!r}"
