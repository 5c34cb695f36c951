"""The sizes and byte offsets of the row copies (csrc/ar_steps.h), walked on the host: no sum wraps for any row that the
entry points take, and a type with a sign in their place does not hold them."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "all_reduce_reduction_ring_amd", "csrc")
ROWS = [2 ** 31 - d for d in (1, 2, 4, 15, 16, 17, 127, 2048, 8176, 8191, 8192, 8193, 16384)] + [
    16, 17, 511, 513, 2047, 2048, 2049, 8192, 8193, 1 << 20]


def _build(tmp_path, include):
    exe = str(tmp_path / "row_steps")
    subprocess.run(["g++", "-std=c++17", "-O2", "-fwrapv", "-w", "-I", str(include), os.path.join(ROOT, "tests", "c", "row_steps.cpp"),
                    "-o", exe], check=True, capture_output=True, text=True)
    return exe


def test_every_row_size(tmp_path):
    r = subprocess.run([_build(tmp_path, CSRC), *map(str, ROWS)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("row", [2 ** 31 - 1, 2 ** 31 - 8191])
def test_a_sign_shows(tmp_path, row):
    """The walk itself: with signed offsets it does not end in the row."""
    header = open(os.path.join(CSRC, "ar_steps.h")).read()
    signed, n = re.subn(r"using row_bytes_t = uint32_t;", "using row_bytes_t = int32_t;", header)
    assert n == 1
    (tmp_path / "ar_steps.h").write_text(signed)
    r = subprocess.run([_build(tmp_path, tmp_path), str(row)], capture_output=True, text=True, timeout=120)
    assert r.returncode != 0
