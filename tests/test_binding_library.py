"""The binding says to rebuild a library that it does not fit: one of another
ABI version, or one built before calls were added."""
import subprocess

import pytest

import sparse_memory_linear_sdm_amd as sdm


def _library(tmp_path, version, exports):
    src, so = tmp_path / "stub.c", tmp_path / "libstub.so"
    src.write_text(f"int sdm_abi_version(void) {{ return {version}; }}\n" +
                   "".join(f"int {e}(void) {{ return 0; }}\n" for e in exports))
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    return str(so)


ALL = tuple(e for e in sdm.EXPORTS if e != "sdm_abi_version")


@pytest.mark.parametrize("version,exports,says", [
    (sdm.ABI_VERSION - 1, ALL, f"ABI {sdm.ABI_VERSION - 1}"),
    (sdm.ABI_VERSION - 1, ALL[:2], f"ABI {sdm.ABI_VERSION - 1}"),
    (sdm.ABI_VERSION, tuple(e for e in ALL if "mx4" not in e), "sdm_mx4_quantize"),
    (sdm.ABI_VERSION, tuple(e for e in ALL if e != "sdm_last_error"), "sdm_last_error")])
def test_a_stale_library(tmp_path, monkeypatch, version, exports, says):
    monkeypatch.setattr(sdm, "LIB_PATH", _library(tmp_path, version, exports))
    monkeypatch.setattr(sdm, "_lib", None)
    for _ in range(2):
        with pytest.raises(RuntimeError, match=f"{says}.*rebuild it"):
            sdm.lib()


def test_the_whole_set_loads(tmp_path, monkeypatch):
    monkeypatch.setattr(sdm, "LIB_PATH", _library(tmp_path, sdm.ABI_VERSION, ALL))
    monkeypatch.setattr(sdm, "_lib", None)
    assert sdm.lib().sdm_abi_version() == sdm.ABI_VERSION
