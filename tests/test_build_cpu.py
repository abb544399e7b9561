"""The build step's cache: what an object is compiled from decides whether it is compiled again."""
import os
import shutil

import pytest


@pytest.mark.parametrize("changed", ["csrc/*.cu", "csrc/*.cuh", "csrc/*.h", "include/*.h"])
def test_a_changed_source_or_header_compiles_its_objects_again(changed, tmp_path, monkeypatch, repo_root):
    from weight_sequence_mixing_b200 import build
    shutil.copytree(build.CSRC, tmp_path / "csrc")
    shutil.copytree(build.INCLUDE, tmp_path / "include")
    monkeypatch.setattr(build, "CSRC", str(tmp_path / "csrc"))
    monkeypatch.setattr(build, "INCLUDE", str(tmp_path / "include"))
    src = str(tmp_path / "csrc" / "scan.cu")
    before = build._digest(src, [])
    assert build._digest(src, []) == before != build._digest(src, ["-G"])
    folder, ending = changed.split("/")
    files = [src] if ending == "*.cu" else [str(f) for f in sorted((tmp_path / folder).glob(ending))]
    assert files
    for f in files:
        text = open(f).read()
        with open(f, "a") as fh:
            fh.write("\n// changed\n")
        assert build._digest(src, []) != before, os.path.basename(f)
        with open(f, "w") as fh:
            fh.write(text)
    assert build._digest(src, []) == before
