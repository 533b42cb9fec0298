"""The build's handling of object files, with a stand-in for the compiler."""
import stat
import subprocess

import pytest

from int8_w8a8_quantized_smoothed_b200 import build

# writes half an object and fails for the source named in FAIL, else writes "<source>: whole"
COMPILER = """#!/bin/sh
for a; do
  [ "$prev" = "-o" ] && out="$a"
  [ "$prev" = "-c" ] && src="$a"
  prev="$a"
done
if [ -n "$src" ] && [ "$(basename "$src")" = "$FAIL" ]; then
  printf half > "$out"
  exit 1
fi
printf '%s: whole' "$(basename "${src:-library}")" > "$out"
"""


@pytest.fixture
def fake(tmp_path, monkeypatch):
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(COMPILER)
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(build, "nvcc", lambda: str(nvcc))
    monkeypatch.setattr(build, "OBJ_DIR", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    return tmp_path


def test_a_compile_cut_short_leaves_no_object(fake, monkeypatch):
    monkeypatch.setenv("FAIL", "grad.cu")
    with pytest.raises(subprocess.CalledProcessError):
        build.build()
    obj = fake / "obj"
    assert (obj / "w8a8.cu.o").read_text() == "w8a8.cu: whole"
    assert not (obj / "grad.cu.o").exists() and not (fake / "lib.so").exists()
    monkeypatch.setenv("FAIL", "")
    build.build()  # and the next build makes it
    assert (obj / "grad.cu.o").read_text() == "grad.cu: whole"
    assert (fake / "lib.so").read_text() == "library: whole"


def test_an_older_object_survives_a_failed_build(fake, monkeypatch):
    monkeypatch.setenv("FAIL", "")
    build.build()
    monkeypatch.setenv("FAIL", "grad.cu")
    with pytest.raises(subprocess.CalledProcessError):
        build.build(force=True)
    assert (fake / "obj" / "grad.cu.o").read_text() == "grad.cu: whole"
