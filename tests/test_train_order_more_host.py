"""The sequence operators' kernels, too, touch no global memory in front of their wait for the kernel
before them on the stream (grid_dep_wait), and none of them leaves before it: checked in the source."""
import re

import pytest

from .test_train_order_host import WAIT, kernels, without_lambdas

FILES = ["kernels_scan.cu", "kernels_distill.cu", "kernels_ln.cu"]


@pytest.mark.parametrize("name", FILES)
def test_global_memory_is_touched_behind_the_wait(name):
    found = list(kernels(name))
    assert found
    for kernel, params, body in found:
        pointers = re.findall(r"\*\s*(?:__restrict__\s+)?(\w+)\s*(?:,|$)", params)
        assert pointers
        body = without_lambdas(body)
        assert WAIT in body, f"{kernel} has no wait"
        front = body[:body.index(WAIT)]
        assert not re.search(r"\breturn\b", front), f"{kernel} may end in front of its wait"
        for p in pointers:
            use = re.search(rf"\b{p}\s*\[|\b(?:ld|ldg|st|load|store)\s*\(\s*{p}\b|\(\s*{p}\s*,|,\s*{p}\s*[,)]|\*\s*{p}\b",
                            front)
            assert not use, f"{kernel}: {p} is used in front of the wait: {use.group(0)!r}"
