"""Host check of the 8-bit tape's buffer descriptors (csrc/ranges.h, built with
g++ alone): every size below 2 GiB of codes has both descriptors in range, and
every offset the kernels form -- record number * 16 for codes, record number
for scales -- stays inside them."""
import itertools
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_tape8_descriptors(tmp_path):
    exe = str(tmp_path / "tape8_ranges")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror",
                    os.path.join(ROOT, "tests", "native", "tape8_ranges_check.cpp"), "-o", exe],
                   check=True)
    shapes = list(itertools.product([16, 32, 64, 128, 256],
                                    [0, 1, 7, 4096, 16384, 131071, 131072, 1 << 20, 1 << 24],
                                    [1, 13, 64], [1, 9, 64]))
    r = subprocess.run([exe], input="\n".join(" ".join(map(str, s)) for s in shapes),
                       capture_output=True, text=True, check=True)
    got = [int(x) for x in r.stdout.split()]
    assert len(got) == len(shapes)
    for (d_v, T, W, R), ok in zip(shapes, got):
        assert ok == (T * (W + R) * d_v < 1 << 31), (d_v, T, W, R)
        if ok and T:
            # last record of the last block's last step
            rec = (d_v // 16 - 1) * T * (W + R) + (T - 1) * (W + R) + W + R - 1
            assert rec * 16 + 16 == T * (W + R) * d_v and rec < (1 << 31) // 16
