"""The loads of the experts' products' operand tiles, walked on the host: none leaves its matrix, all elements come through;
and a bound that stops at the step or the row instead does not hold."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "all_reduce_reduction_ring_amd", "csrc")
# widths whose rows are multiples of 4 bytes, narrower and wider than a tile, with and without a chunk that the end cuts
SIZES = [(2, r, w) for r in (1, 3, 63, 64, 65, 130, 257, 300) for w in (2, 6, 8, 62, 64, 66, 130, 256, 322)] + [
    (4, r, w) for r in (1, 31, 33, 130, 257) for w in (1, 3, 4, 31, 33, 64, 77, 257)]


def _build(tmp_path, include):
    exe = str(tmp_path / "load_steps")
    subprocess.run(["g++", "-std=c++17", "-O2", "-w", "-I", str(include), os.path.join(ROOT, "tests", "c", "load_steps.cpp"), "-o", exe],
                   check=True, capture_output=True, text=True)
    return exe


def test_no_load_leaves_the_matrix(tmp_path):
    exe = _build(tmp_path, CSRC)
    for size in SIZES:
        r = subprocess.run([exe, *map(str, size)], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, (size, r.stdout)


@pytest.mark.parametrize("what,size", [
    (r"return static_cast<int64_t>\(rows - 1\) \* stride \+ static_cast<int64_t>\(sum - k\) \* size;", (2, 3, 66)),
    (r"return static_cast<int64_t>\(sum - k\) \* stride - static_cast<int64_t>\(first\) \* size;", (2, 130, 2))])
def test_a_bound_that_is_not_exact_shows(tmp_path, what, size):
    """The walk itself: without the bounds it finds loads outside."""
    header = open(os.path.join(CSRC, "ar_steps.h")).read()
    loose, n = re.subn(what, "return int64_t(1) << 30;", header)
    assert n == 1
    (tmp_path / "ar_steps.h").write_text(loose)
    r = subprocess.run([_build(tmp_path, tmp_path), *map(str, size)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 1 and "a load past the matrix" in r.stdout
