"""The sizes and byte offsets of the row copies and the steps over choices and pad rows (csrc/ar_steps.h), walked on the host: no sum wraps for any row that the
entry points take, and a type with a sign in their place does not hold them."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "all_reduce_reduction_ring_amd", "csrc")
ROWS = [2 ** 31 - d for d in (1, 2, 4, 15, 16, 17, 127, 2048, 8176, 8191, 8192, 8193, 16384)] + [
    16, 17, 511, 513, 2047, 2048, 2049, 8192, 8193, 1 << 20]


def _build(tmp_path, include, name="row_steps", *flags):
    exe = str(tmp_path / name)
    subprocess.run(["g++", "-std=c++17", "-O2", "-fwrapv", "-w", *flags, "-I", str(include), os.path.join(ROOT, "tests", "c", name + ".cpp"),
                    "-o", exe], check=True, capture_output=True, text=True)
    return exe


def _signed(tmp_path, name):
    header = open(os.path.join(CSRC, "ar_steps.h")).read()
    signed, n = re.subn(rf"using {name} = uint32_t;", f"using {name} = int32_t;", header)
    assert n == 1
    (tmp_path / "ar_steps.h").write_text(signed)
    return tmp_path


def test_every_row_size(tmp_path):
    r = subprocess.run([_build(tmp_path, CSRC), *map(str, ROWS)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("row", [2 ** 31 - 1, 2 ** 31 - 8191])
def test_a_sign_shows(tmp_path, row):
    """The walk itself: with signed offsets it does not end in the row."""
    r = subprocess.run([_build(tmp_path, _signed(tmp_path, "row_bytes_t")), str(row)], capture_output=True, text=True, timeout=120)
    assert r.returncode != 0


def test_every_number_of_choices(tmp_path):
    counts = [1, 7, 8, 9, 64, 2 ** 31 - 16, *range(2 ** 31 - 9, 2 ** 31)]
    r = subprocess.run([_build(tmp_path, CSRC, "choice_steps"), *map(str, counts)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def test_counting_up_shows_in_the_choices(tmp_path):
    exe = _build(tmp_path, CSRC, "choice_steps", "-DCOUNT_UP")
    assert subprocess.run([exe, str(2 ** 31 - 8)], capture_output=True, text=True, timeout=120).returncode == 0
    r = subprocess.run([exe, str(2 ** 31 - 1)], capture_output=True, text=True, timeout=120)
    assert r.returncode != 0


ENDS = [16, 17, 2 ** 20, 2 ** 31 - 17, *range(2 ** 31 - 16, 2 ** 31)]


def test_pads_up_to_every_end(tmp_path):
    r = subprocess.run([_build(tmp_path, CSRC, "pad_steps"), *map(str, ENDS)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def test_a_sign_shows_in_the_pads(tmp_path):
    exe = _build(tmp_path, _signed(tmp_path, "sorted_row_t"), "pad_steps")
    r = subprocess.run([exe, str(2 ** 31 - 1)], capture_output=True, text=True, timeout=120)
    assert r.returncode != 0
