"""When the library counts as out of date."""

import glob
import os

import pytest


def test_every_source_is_an_input():
    from paged_kv_decode_mapping_gb300 import build

    here = {p for p in glob.glob(os.path.join(build.CSRC, "*")) if os.path.isfile(p)}
    assert here <= set(build._inputs())


@pytest.mark.parametrize("ending", ["cu", "cpp", "cuh", "h"])
def test_a_newer_source_makes_the_library_stale(tmp_path, monkeypatch, ending):
    from paged_kv_decode_mapping_gb300 import build

    lib, src = tmp_path / "libpkv.so", tmp_path / f"piece.{ending}"
    lib.touch()
    src.touch()
    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    monkeypatch.setattr(build, "INCLUDE", str(tmp_path))
    os.utime(src, (1000, 1000))
    os.utime(lib, (2000, 2000))
    assert not build.stale()
    os.utime(src, (3000, 3000))
    assert build.stale()
