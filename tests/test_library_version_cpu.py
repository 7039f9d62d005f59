"""A library of another build than the binding: one message, whatever it lacks."""
import ctypes
import shutil
import subprocess

import pytest

import vocabulary_cross_entropy_row_amd as lce

pytestmark = pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")


def built(directory, source):
    c, so = directory / "old.c", directory / "liblce.so"
    c.write_text(source)
    subprocess.run(["gcc", "-shared", "-fPIC", str(c), "-o", str(so)], check=True)
    return str(so)


@pytest.mark.parametrize("source", [
    "int lce_abi_version(void) { return 2; }",                                          # another version
    f"int lce_abi_version(void) {{ return {lce.ABI_VERSION}; }}",                       # this version, before its entry points
    "const char *lce_last_error(void) { return \"\"; }",                                # not even that
], ids=["older version", "missing entry points", "no version"])
def test_another_build_asks_for_a_rebuild(source, tmp_path, monkeypatch):
    monkeypatch.setattr(lce, "_lib", None)
    monkeypatch.setattr(lce, "LIB_PATH", built(tmp_path, source))
    with pytest.raises(ImportError, match="rebuild it"):
        lce.lib()
    assert lce._lib is None   # a second call checks again


def test_this_build_loads(monkeypatch):
    monkeypatch.setattr(lce, "_lib", None)
    assert lce.lib().lce_abi_version() == lce.ABI_VERSION
    assert isinstance(lce.lib(), ctypes.CDLL)
