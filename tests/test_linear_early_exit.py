"""The linear kernels' way out after a bounded wait has expired, read as source (no wait expires in a test: the kernels
wait for nothing but their own copies and products).  A CTA must not leave while a copy may still be writing its shared
memory."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "collective_matmul_decomposition_gb300",
                    "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_a_strips_loader_waits_for_what_it_issued():
    """Whether or not some other thread has given up by then: it may do so later."""
    text = source("cm_linear_strip.cu")
    kernel = text[text.index("cm_linear_strip_kernel("):]
    loop = re.search(r"([^;{}]*)for \(int i = 0; i < p\.stages && i < issued; \+\+i\)\s*drain_l\(", kernel)
    assert loop, "no drain of the issued loads"
    assert loop.group(1).strip() == ""


def test_an_aborting_pair_waits_for_loads_that_no_barrier_counts():
    text = source("cm_linear_pair.cu")
    close = text[text.index("void close_pair("):]
    close = close[:close.index("\n}\n")]
    synced, settled = close.find("cluster_sync();"), close.find("settle(")
    assert 0 <= synced < settled, "leaves without waiting"
