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


def test_waits_last_as_long_as_a_tile_of_many_slices():
    """A tile's products are waited for by its epilogue: 0.28 us a slice of 64 terms on the largest tiles, which for 2^30
    terms is more than the second that a small call's waits are bounded by."""
    text = source("cm_linear_api.cu")
    limit = re.search(r"uint64_t linear_timeout_ns\(int kblocks\) \{ return (\d+)ull \+ (\d+)ull \* uint64_t\(kblocks\); \}", text)
    assert limit and int(limit.group(1)) >= 10 ** 9
    for kblocks in (1, 1 << 12, 1 << 22, 1 << 24):
        assert int(limit.group(1)) + int(limit.group(2)) * kblocks > 1.5 * 281 * kblocks
    assert re.findall(r"timeout_ns = (.*?);", text) == ["linear_timeout_ns(p.kblocks)"] * 2
