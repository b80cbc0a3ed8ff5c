"""The library is rebuilt when any file it is compiled from is newer (no GPU needed)."""
import os

import pytest

from quantized_linear_attention_sq_b200 import build


@pytest.mark.parametrize("name", ["csrc/a.cu", "csrc/a.cuh", "csrc/a.h", "include/a.h"])
def test_a_newer_source_makes_the_library_stale(name, tmp_path, monkeypatch):
    for sub in ("csrc", "include"):
        (tmp_path / sub).mkdir()
        monkeypatch.setattr(build, sub.upper(), str(tmp_path / sub))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    source, lib = tmp_path / name, tmp_path / "lib.so"
    source.write_text("")
    assert build._stale()
    lib.write_text("")
    os.utime(source, (100, 100))
    os.utime(lib, (200, 200))
    assert not build._stale()
    os.utime(source, (300, 300))
    assert build._stale()
