"""The experts' products' loads through registers, and those of the kernel for few rows, walked on the host: none leaves its
matrix, every element of a sum comes through once; and conditions that are loose or missing do not hold."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "all_reduce_reduction_ring_amd", "csrc")
# odd and even widths, narrower and wider than a tile and than a block of the few rows' kernel, at its ends and beside them
SIZES = [(2, r, w) for r in (1, 3, 17, 64, 65, 130) for w in (1, 2, 5, 7, 8, 9, 31, 33, 63, 64, 65, 127, 129, 255, 322, 577, 641)] + [
    (4, r, w) for r in (1, 17, 33, 130) for w in (1, 3, 4, 5, 31, 32, 33, 63, 65, 131, 257, 321)]


def _build(tmp_path, include):
    exe = str(tmp_path / "register_steps")
    subprocess.run(["g++", "-std=c++17", "-O2", "-w", "-I", str(include), os.path.join(ROOT, "tests", "c", "register_steps.cpp"), "-o", exe],
                   check=True, capture_output=True, text=True)
    return exe


def test_no_load_leaves_the_matrix(tmp_path):
    exe = _build(tmp_path, CSRC)
    for size in SIZES:
        r = subprocess.run([exe, *map(str, size)], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, (size, r.stdout)


@pytest.mark.parametrize("what,instead,size,shows", [
    (r"return at \+ 16 <= left;", "return true;", (2, 3, 65), "a load past the matrix"),
    (r"return at \+ 16 <= left;", "return at < left;", (2, 130, 1), "a load past the matrix"),
    (r"return at \+ v <= k;", "return true;", (2, 3, 65), "a load past the matrix or the row"),
    (r"return at \+ v <= k;", "return at + v < k;", (2, 3, 64), None),  # the elements one by one: right, only slower
    (r"return kFewUnits \* 4 \* v;", "return kFewUnits * 4 * v + v;", (2, 3, 577), "once")])
def test_a_condition_that_is_not_exact_shows(tmp_path, what, instead, size, shows):
    header = open(os.path.join(CSRC, "ar_steps.h")).read()
    loose, n = re.subn(what, instead, header)
    assert n == 1
    (tmp_path / "ar_steps.h").write_text(loose)
    r = subprocess.run([_build(tmp_path, tmp_path), *map(str, size)], capture_output=True, text=True, timeout=60)
    assert (r.returncode == 0) if shows is None else (r.returncode == 1 and shows in r.stdout), r.stdout
