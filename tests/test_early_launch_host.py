"""Kernels launched early (launch.cuh) wait for the kernels ahead of them before
they touch global memory: only a kernel's own wait makes what those wrote
visible to it.  Read from the sources: the wait stands at a kernel's outermost
level, and nothing ahead of it goes to global memory (no GPU needed)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gradient_allreduce_homomorphic_gb300",
                    "csrc")
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu") and '#include "launch.cuh"' in open(os.path.join(CSRC, f)).read())
# helpers that load, store or copy, and subscripts of the parameters' pointers
TOUCHES = re.compile(r"\b(fetch|choose|gradient|ld16|st16|load_f32|store_f32|tma_load\w*|bulk_load|copy_scales_async|__ldcg)\b"
                     r"|\bp\.\w+\[|\batomic\w+\(&?p\.")


def kernels(name):
    """(kernel, body) of every __global__ function of a source, comments taken out."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for m in re.finditer(r"__global__[^{;]*?(\w+_kernel)\(", text):
        begin = text.index("{", m.end())
        depth, at = 1, begin + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield m.group(1), text[begin + 1:at - 1]


def test_sources_are_found():
    assert {"balance.cu", "distill.cu", "matmul.cu", "quantize.cu"} <= set(FILES)
    assert sum(len(list(kernels(f))) for f in FILES) >= 9


@pytest.mark.parametrize("name", FILES)
def test_wait_comes_before_global_memory(name):
    for kernel, body in kernels(name):
        waits = [m.start() for m in re.finditer(r"\bafter_previous\(\);", body)]
        outer = [w for w in waits if body[:w].count("{") == body[:w].count("}")]
        assert outer, f"{kernel} has no wait at its outermost level"
        touched = TOUCHES.search(body[:outer[0]])
        assert touched is None, f"{kernel}: {touched.group(0)} before the wait"
