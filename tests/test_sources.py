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


def test_no_load_is_non_coherent():
    """A kernel may be resident while the one before it in the stream still writes its
    inputs, and an output may be an input (the combine's base): a load that assumes
    memory which nothing writes for the kernel's whole duration may be moved before the
    wait for that kernel, or return what was there before."""
    for name, text in sources():
        code = re.sub(r"//[^\n]*", "", text)
        assert not re.search(r"__ldg\s*\(|ld\.global\S*\.nc\b|__restrict__", code), name
