"""The entry points of the dense recurrence and the norms (csrc/api_dense.hip,
with csrc/api.hip) built for the host alone with AddressSanitizer and
UndefinedBehaviorSanitizer, kernel launchers replaced by the stubs of
tests/native/api_dense_asan_driver.cpp."""
import os
import subprocess

import pytest

from tests.test_api_sanitized import CLANG, FLAGS, ROOT


@pytest.mark.skipif(not os.path.exists(CLANG), reason="ROCm clang not available")
def test_dense_entry_points_under_asan_and_ubsan(tmp_path):
    csrc = os.path.join(ROOT, "sparse_memory_linear_sdm_amd", "csrc")
    objs = []
    for src in (os.path.join(csrc, "api.hip"), os.path.join(csrc, "api_dense.hip"),
                os.path.join(ROOT, "tests", "native", "api_dense_asan_driver.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        subprocess.run([CLANG, *FLAGS, "-c", src, "-o", obj], check=True)
        objs.append(obj)
    exe = str(tmp_path / "api_dense_asan")
    subprocess.run([CLANG, "-Xarch_host", "-fsanitize=address,undefined", *objs, "-o", exe],
                   check=True)
    env = {k: v for k, v in os.environ.items() if k != "SDM_DEBUG_SYNC"}
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    assert r.stdout.strip() == "ok"
