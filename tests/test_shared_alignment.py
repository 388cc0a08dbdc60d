"""Shared memory that other CTAs of a cluster read or write in pairs lies on 8 bytes by its type, not by chance."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "latency_moe_decode_gb300", "csrc")


def test_paired_cluster_accesses_take_pairs():
    """Each such access stands in a function of its own that takes a pointer to pairs: what is passed to it is aligned
    by its declaration (an array of single words is only to 4 bytes, and where it lies beyond that is the compiler's)."""
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        lines = open(path).read().split("\n")
        for i, line in enumerate(lines):
            if re.search(r"shared::cluster\.v2", line):
                seen += 1
                head = next(lines[k] for k in range(i, -1, -1) if re.match(r"(template|__global__|__device__|static)", lines[k]))
                assert re.search(r"\((const )?(uint2|float2)\* at, uint32_t cta", head), (os.path.basename(path), i + 1, head)
    assert seen >= 3
