"""Properties of the kernel sources, without a GPU."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tensor_gemm_reduction_gb300", "csrc")


def sources():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h")):
            yield name, open(os.path.join(CSRC, name)).read()


def test_no_copy_lands_in_several_ctas():
    """The library also runs on every GPU of a job of several: its bulk copies write the
    shared memory of one CTA. (A commit may arrive on the barriers of a pair.)"""
    for name, text in sources():
        joined = re.sub(r'"\s*"', "", text)   # adjacent string literals of one instruction
        for copy in re.findall(r"cp\.async\.bulk[^\[;]*", joined):
            assert ".multicast" not in copy, (name, copy)
