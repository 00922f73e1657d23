"""Build librlt.so (the C-ABI library) for sm_100a with nvcc, in-tree.

    python -m token_recurrent_decoding_b200.build [--force]
"""
from __future__ import annotations

import contextlib
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "librlt.so")
MAIN = os.path.join(CSRC, "rlt_api.cu")


def units():
    """Every translation unit of the library (rlt_api.cu first)."""
    extra = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu") and f != "rlt_api.cu")
    return [MAIN] + [os.path.join(CSRC, f) for f in extra]


NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
]
OBJ = os.path.join(PKG, "_build")  # one object and one dependency file per unit


def sources():
    out = [os.path.join(ROOT, "include", "rlt.h")]
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh", ".h")):
            out.append(os.path.join(CSRC, f))
    return out


def _object(unit: str) -> str:
    return os.path.join(OBJ, os.path.splitext(os.path.basename(unit))[0] + ".o")


def _flags_of(unit: str):
    """The flags the unit's object was compiled with; None where that is not known."""
    try:
        with open(_object(unit) + ".flags") as f:
            return f.read()
    except OSError:
        return None


def stale() -> bool:
    """Whether the library is older than its sources, or has units of other flags than FLAGS."""
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return (any(os.path.getmtime(s) > t for s in sources()) or
            any(_flags_of(u) not in (None, " ".join(FLAGS)) for u in units()))


def _object_stale(unit: str, flags) -> bool:
    """Whether the unit's object has other flags, or is older than a file of this tree that its last
    compilation read."""
    obj = _object(unit)
    if not (os.path.exists(obj) and os.path.exists(obj + ".d")) or \
            _flags_of(unit) != " ".join(flags):
        return True
    with open(obj + ".d") as f:
        deps = f.read().replace("\\\n", " ").split()[1:]
    deps = [d for d in deps if os.path.abspath(d).startswith(ROOT + os.sep)] + [unit, __file__]
    t = os.path.getmtime(obj)
    return any(not os.path.exists(d) or os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile the units that changed, side by side, and link them: all of FLAGS and `extra`."""
    if not force and not extra and not stale():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    flags = [*FLAGS, *extra]
    todo = [u for u in units() if force or _object_stale(u, flags)]

    def compile_unit(unit):
        obj = _object(unit)
        cmd = [NVCC, *flags, "-MD", "-MF", obj + ".d", "-c", unit, "-o", obj + ".tmp"]
        if verbose:
            print(" ".join(cmd), flush=True)
        with contextlib.suppress(FileNotFoundError):  # another build may have
            os.remove(obj + ".flags")
        subprocess.check_call(cmd)
        os.replace(obj + ".tmp", obj)
        with open(obj + ".flags", "w") as f:
            f.write(" ".join(flags))

    with ThreadPoolExecutor(max(1, min(len(todo), os.cpu_count() or 1))) as pool:
        list(pool.map(compile_unit, todo))
    tmp = LIB + ".tmp"
    subprocess.check_call([NVCC, *FLAGS, "-shared", *map(_object, units()), "-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=("-Xptxas", "-v") if "--ptxas" in sys.argv else ())
