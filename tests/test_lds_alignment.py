"""LDS arrays of the dense kernels that are accessed by vectors (reinterpreted,
or through helpers that do) are declared with a vector's alignment, not left to
what the compiler happens to place."""
import os
import re

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "sparse_memory_linear_sdm_amd", "csrc")
FILES = ["linear.hip", "linear_scan.h", "linear_backward.h", "norm.hip"]
ACCESS = (r"reinterpret_cast<[^>]*(?:f32x4|u32x4|bf16x4|bf16x8|f32x8)\*>\(\s*{n}\b"
          r"|\b(?:put8|weights8|store4|store4_parts|store)\(\s*{n}\b|(?:rows|cols)(?:<\w+>)?\(\s*{n}\b")


@pytest.mark.parametrize("name", FILES)
def test_arrays_accessed_by_vectors_are_aligned(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    seen = 0
    for words, names in re.findall(r"__shared__\s+([^;\[]*?)\s*(\w+\[[^;]*);", text):
        for array in re.findall(r"(?:^|,\s*)(\w+)\[", names):
            if re.search(ACCESS.format(n=array), text):
                seen += 1
                aligned = "__align__(16)" in words or re.search(r"\b(f32x4|u32x4)\b", words)
                assert aligned, f"{name}: {array} is accessed by vectors and declared as '{words}'"
    assert seen
