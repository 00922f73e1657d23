"""Which units the library's build compiles, with a compiler that only writes down its arguments."""
import os

import pytest

from token_recurrent_decoding_b200 import build as b

COMPILER = """#!/bin/sh
all="$*"
while [ $# -gt 0 ]; do
  case "$1" in
    -o) out="$2" ;;
    -MF) dep="$2" ;;
    -c) unit="$2" ;;
  esac
  shift
done
[ -n "$dep" ] && echo "x.o: $unit" > "$dep"
echo "$all" > "$out"
[ -z "$unit" ] || echo "$unit" >> "{log}"
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    csrc = tmp_path / "pkg" / "csrc"
    csrc.mkdir(parents=True)
    (tmp_path / "include").mkdir()
    for f in ("rlt_api.cu", "one.cu", "two.cu"):
        (csrc / f).write_text(f)
    (tmp_path / "include" / "rlt.h").write_text("")
    log = tmp_path / "log"
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(COMPILER.replace("{log}", str(log)))
    nvcc.chmod(0o755)
    for name, value in (("ROOT", tmp_path), ("CSRC", csrc), ("MAIN", csrc / "rlt_api.cu"),
                        ("LIB", tmp_path / "pkg" / "librlt.so"), ("NVCC", nvcc),
                        ("OBJ", tmp_path / "pkg" / "_build")):
        monkeypatch.setattr(b, name, str(value))

    def compiled():
        names = sorted(os.path.basename(x) for x in log.read_text().split()) if log.exists() else []
        log.write_text("")
        return names

    def objects():
        return {f: (tmp_path / "pkg" / "_build" / f).read_text() for f in
                ("rlt_api.o", "one.o", "two.o")}
    return csrc, compiled, objects


ALL = ["one.cu", "rlt_api.cu", "two.cu"]


def _touch(path):
    """As if `path` had changed since it was compiled."""
    old = os.path.getmtime(path) - 10
    os.utime(b.LIB, (old, old))
    os.utime(b._object(str(path)), (old, old))


def test_only_what_changed_is_compiled(tree):
    csrc, compiled, _ = tree
    b.build()
    assert compiled() == ALL
    b.build()
    assert compiled() == []
    _touch(csrc / "one.cu")
    b.build()
    assert compiled() == ["one.cu"]
    b.build(force=True)
    assert compiled() == ALL


def test_units_of_other_flags_are_compiled_again(tree):
    csrc, compiled, objects = tree
    b.build()
    compiled()
    b.build(extra=("-DPROBE",))
    assert compiled() == ALL and all("-DPROBE" in x for x in objects().values())
    _touch(csrc / "one.cu")
    b.build()
    assert compiled() == ALL and not any("-DPROBE" in x for x in objects().values())
    # also where no source changed
    b.build(extra=("-DPROBE",))
    compiled()
    b.build()
    assert compiled() == ALL and not any("-DPROBE" in x for x in objects().values())
    assert not b.stale()


def test_a_library_without_objects_is_taken_as_it_is(tree):
    csrc, compiled, _ = tree
    b.build()
    for f in os.listdir(b.OBJ):
        os.remove(os.path.join(b.OBJ, f))
    compiled()
    b.build()
    assert compiled() == []
