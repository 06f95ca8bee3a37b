"""The build keeps an object only while what made it is the same: its sources,
the compile flags and the compiler (a stand-in that notes its calls; no CUDA
compiler is run)."""
import os
import time

import pytest

from sparse_moe_transformer_router_b200 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    for folder in ("csrc", "include"):
        (tmp_path / folder).mkdir()
    (tmp_path / "csrc" / "a.cu").write_text('#include "shared.cuh"\n')
    (tmp_path / "csrc" / "b.cu").write_text("int b;\n")
    (tmp_path / "csrc" / "shared.cuh").write_text("int s;\n")
    for name, value in (("CSRC", "csrc"), ("INCLUDE", "include"), ("OBJ", "build"), ("LIB", "lib.so")):
        monkeypatch.setattr(build, name, str(tmp_path / value))
    compiler(tmp_path, monkeypatch, "1.0")
    return tmp_path


def compiler(folder, monkeypatch, version):
    """A compiler that writes its output file and notes what it compiled."""
    path = folder / f"nvcc-{version}"
    path.write_text(f'''#!/bin/sh
[ "$1" = --version ] && {{ echo "release {version}"; exit 0; }}
out= ; prev=
for a in "$@"; do
    [ "$prev" = -o ] && out="$a"
    [ "$prev" = -c ] && echo "$(basename $a)" >> "{folder}/compiled"
    prev="$a"
done
touch "$out"
''')
    path.chmod(0o755)
    monkeypatch.setenv("NVCC", str(path))


def compiled(folder):
    """The sources compiled since the last look."""
    log = folder / "compiled"
    names = sorted(log.read_text().split()) if log.exists() else []
    log.write_text("")
    return names


def change(path):
    later = time.time() + change.ahead
    change.ahead += 10
    os.utime(path, (later, later))


change.ahead = 10


def rebuild(folder, **kw):
    build.build(**kw)
    for name in ("lib.so", "build/a.o", "build/b.o"):  # newer than every change so far
        change(folder / name)
    return compiled(folder)


def test_an_object_is_kept_while_what_made_it_is_the_same(tree, monkeypatch):
    assert rebuild(tree) == ["a.cu", "b.cu"]
    assert rebuild(tree) == []
    change(tree / "csrc" / "b.cu")
    assert rebuild(tree) == ["b.cu"]
    change(tree / "csrc" / "shared.cuh")
    assert rebuild(tree) == ["a.cu"]
    assert rebuild(tree, force=True) == ["a.cu", "b.cu"]


def test_other_flags_compile_everything_again(tree, monkeypatch):
    rebuild(tree)
    monkeypatch.setattr(build, "ARCH", ["-gencode", "arch=compute_100a,code=[sm_100a,compute_100a]"])
    change(tree / "csrc" / "b.cu")
    assert rebuild(tree) == ["a.cu", "b.cu"]
    change(tree / "csrc" / "b.cu")
    assert rebuild(tree) == ["b.cu"]


def test_another_compiler_compiles_everything_again(tree, monkeypatch):
    rebuild(tree)
    compiler(tree, monkeypatch, "2.0")
    change(tree / "csrc" / "b.cu")
    assert rebuild(tree) == ["a.cu", "b.cu"]
    change(tree / "csrc" / "b.cu")
    assert rebuild(tree) == ["b.cu"]


def test_a_changed_folder_of_headers_compiles_everything_again(tree, monkeypatch):
    """(the flags name it)"""
    rebuild(tree)
    (tree / "other").mkdir()
    monkeypatch.setattr(build, "INCLUDE", str(tree / "other"))
    change(tree / "csrc" / "b.cu")
    assert rebuild(tree) == ["a.cu", "b.cu"]
