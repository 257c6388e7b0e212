"""A rule that the kernels' sources have to keep, checked as text (no GPU): a
kernel that starts while the kernel ahead of it still runs (griddep_wait)
reads nothing through the read-only path.  Its loads of what that kernel
writes could be moved ahead of the wait by the compiler, and the data is not
constant while it runs."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunked_prefill_hybrid_tau_gb300",
                    "csrc")
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def kernels(text):
    """(name, parameters, body) of each __global__ function."""
    for m in re.finditer(r"__global__", text):
        head = re.compile(r"(\w+)\s*\(([^()]*(?:\([^()]*\)[^()]*)*)\)\s*\{").search(text, m.end())
        depth, i = 1, head.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield head.group(1), head.group(2), text[head.end():i]


def test_the_kernels_are_found():
    waiting = [k for f in FILES for k, _, body in kernels(source(f)) if "griddep_wait" in body]
    assert {"kv_append_norm_kernel", "quant_groups_kernel", "rmsnorm_kernel", "quant_rows_kernel"} <= set(waiting)


@pytest.mark.parametrize("name", FILES)
def test_no_read_only_path_behind_a_wait(name):
    text = source(name)
    assert "__ldg(" not in text
    for kernel, params, body in kernels(text):
        if "griddep_wait" not in body:
            continue  # an ordinary launch: starts once the kernel ahead is complete
        bad = [p.strip() for p in params.split(",") if "const" in p and "__restrict__" in p]
        assert not bad, (kernel, bad)
