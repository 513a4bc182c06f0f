"""Which files a library is rebuilt for."""
import glob
import os

from scale_deformable_attention_msda_gb300 import build


def test_every_file_that_a_translation_unit_includes():
    known = {os.path.realpath(f) for f in build._inputs()}
    for f in glob.glob(os.path.join(build.CSRC, "*")) + glob.glob(os.path.join(build.INCLUDE, "*")):
        if f.endswith((".cu", ".cuh", ".h")):
            assert os.path.realpath(f) in known, f


def test_a_header_that_changed_makes_the_library_stale(tmp_path, monkeypatch):
    library = tmp_path / "lib.so"
    library.write_text("")
    old = os.path.getmtime(os.path.abspath(build.__file__)) + 10 ** 6
    os.utime(library, (old, old))
    assert not build.stale(str(library))
    header = tmp_path / "new.h"
    header.write_text("")
    os.utime(header, (old + 1, old + 1))
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    assert build.stale(str(library))
