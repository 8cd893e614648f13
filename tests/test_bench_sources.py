"""The counter records that bench.py quotes are tied to the sources of the
kernels they were taken from: every file of the library that a kernel's file
includes, itself or through another, by the compiler's own account."""
import os
import subprocess

import pytest

import bench

KERNELS = {"SCAN_SOURCES": "scan.hip", "BWD_SOURCES": "backward.hip", "PROJ_SOURCES": "project.hip",
           "PLANNED_SOURCES": "scan_planned.hip", "DECODE_SOURCES": "decode.hip"}


def test_every_list_is_here():
    assert sorted(KERNELS) == sorted(k for k in vars(bench) if k.endswith("_SOURCES"))


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_a_kernels_sources_are_all_hashed(name):
    csrc = os.path.join(bench.ROOT, "sparse_memory_linear_sdm_amd", "csrc")
    # -MG: headers of the HIP runtime need not be found
    r = subprocess.run(["g++", "-x", "c++", "-std=c++17", "-MM", "-MG", os.path.join(csrc, KERNELS[name])],
                       capture_output=True, text=True, check=True)
    files = {os.path.realpath(f) for f in r.stdout.split(":", 1)[1].replace("\\\n", " ").split()}
    local = {f for f in files if os.path.dirname(f) == os.path.realpath(csrc)}
    listed = [os.path.realpath(f) for f in getattr(bench, name)]
    assert len(local) > 1 and set(listed) == local and len(listed) == len(local)
