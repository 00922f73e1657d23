"""How rlt_attend_paged cuts sequences into ranges (csrc/paged_plan.h, the header its kernels and its
host side run), checked without a GPU: tests/paged_plan_check.cpp over random batches, built with
the compiler's checks of undefined behaviour (a division by zero rows, an overflow)."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "token_recurrent_decoding_b200", "csrc")


@pytest.fixture(scope="module")
def checker(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("plan") / "paged_plan_check")
    subprocess.check_call([gxx, "-O1", "-std=c++17", "-fsanitize=undefined",
                           "-fno-sanitize-recover=all", "-I", CSRC,
                           os.path.join(HERE, "paged_plan_check.cpp"), "-o", exe])
    return exe


def _run(exe, off=0):
    r = subprocess.run([exe, str(off)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    m = re.search(r"cases (\d+) failing (\d+) tightest (\d+)", r.stdout)
    assert m, r.stdout
    return int(m.group(2)), int(m.group(3)), r.stdout


def test_ranges_and_their_partial_rows(checker):
    failing, _, out = _run(checker)
    assert failing == 0, out


def test_a_smaller_workspace_is_caught(checker):
    _, tightest, _ = _run(checker)
    assert _run(checker, tightest + 1)[0] > 0
