"""Rules that the kernels' sources have to keep, checked as text (no GPU).

A kernel that starts while the kernel ahead of it still runs (griddep_wait)
reads nothing through the read-only path: its loads of what that kernel
writes could be moved ahead of the wait by the compiler, and the data is not
constant while it runs.

A warp whose bounded wait has expired still meets the others at the named
barriers ahead of it: it leaves no loop that holds one, or the others wait
there for ever."""
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


def block_from(text, start):
    """The statement block whose opening brace follows position `start`."""
    i = text.index("{", start)
    depth, j = 1, i + 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        j += 1
    return text[i:j]


def test_no_warp_leaves_the_others_at_a_named_barrier():
    text = source("gemm_kernel.cuh")
    last = block_from(text, text.index("bool epilogue_last("))
    assert last.count("named_barrier_sync") == 3
    # one way out ahead of a barrier, taken by all threads or none (split_exchange meets them)
    assert last.count("return false") == 1
    assert last.index("split_exchange(") < last.index("return false") < last.index("named_barrier_sync")
    loops = [m.start() for m in re.finditer(r"for \(int un = ", text)]
    assert len(loops) == 2
    for at in loops:
        body = block_from(text, text.index(")", text.index("++t", at)))
        assert "epilogue_last<" in body and not re.search(r"\bbreak\b|\breturn\b", body)
    block = source("gemm_e4m3_block.cu")
    roles = [m.start() for m in re.finditer(r"for \(int [ut] = (?:first; u < units|blockIdx\.x; t < tiles); [ut] \+= \w+"
                                            r"(?:\.x)?\)", block)]
    met = [b for b in (block_from(block, at) for at in roles) if "named_barrier_sync" in b]
    assert len(met) == 2
    for body in met:
        # leaving the sums of a group past the last K block, and a lambda's value
        outer = body.replace("if (kb0 + g0 + g >= kblocks) break;", "").replace("{ return chunk_col(", "{ chunk_col(")
        assert not re.search(r"\bbreak\b|\breturn\b", outer)
