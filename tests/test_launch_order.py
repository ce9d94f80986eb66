"""Kernels that may start under their predecessor's end (cm_launch.cuh), read as source: nothing that an earlier
kernel wrote is promised to be visible before griddepcontrol.wait, so each waits in every thread, on no condition,
before its first access to global memory."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "collective_matmul_decomposition_gb300",
                    "csrc")
WAIT = "wait_for_previous();"
# what reads or writes global memory in these files; prefetches of a tensor map or of a box to L2 do not
ACCESS = re.compile(r"tma_load|tma_store|tma_reduce|copy16|copy_vec|copy_row8|load8|load_row8|load_param8|stage_param|"
                    r"store8|store_row8|param1|to_f\(|from_f\(|load_bias|cp\.async|ld\.global|st\.global|"
                    r"p\.(mean|rstd|x|dy|res|gamma|beta|out|partial|dgamma|dbeta)\b|\bget\(|\bput\(|\*t\.")


def plain(text):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def body(text, at):
    """The braces that open at or behind `at`, with what is between them."""
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start + 1:i]
    raise AssertionError("unbalanced braces")


def kernels():
    found = []
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith(".cu"):
            continue
        with open(os.path.join(CSRC, name)) as f:
            text = plain(f.read())
        if '"cm_launch.cuh"' not in text:
            continue
        helpers = {}   # functions that wait for their callers
        for m in re.finditer(r"__device__[^;{]*?\b(\w+)\([^;{]*?\)\s*\{", text):
            b = body(text, m.start())
            if "wait_for_previous" in b:
                helpers[m.group(1)] = b
        for m in re.finditer(r"__global__ void __launch_bounds__\([^)]*\)\s*(\w+)\(", text):
            b = body(text, m.end())
            for h, hb in helpers.items():
                b = re.sub(rf"[^;{{}}]*\b{h}(<\w+>)?\([^;]*\);", lambda _: hb, b, count=1)
            found.append(pytest.param(b, id=f"{name}:{m.group(1)}"))
    return found


def test_kernels_are_found():
    names = " ".join(p.id for p in kernels())
    for k in ("cm_adamw_kernel", "cm_linear_strip_kernel", "cm_linear_pair_kernel", "cm_linear_split_kernel",
              "cm_layer_norm_ring_kernel", "cm_layer_norm_backward_ring_kernel", "cm_colsum_kernel", "cm_sum_parts_kernel"):
        assert k in names


@pytest.mark.parametrize("text", kernels())
def test_waits_before_the_first_access(text):
    at = text.find(WAIT)
    assert at >= 0, "never waits"
    before = text[:at]
    # a statement of its own, outside of any block: in every thread, whatever the parameters
    assert before.rstrip()[-1:] in (";", "}", ""), before[-60:]
    assert before.count("{") == before.count("}")
    m = ACCESS.search(before)
    assert m is None, f"{m and m.group(0)} before the wait"
