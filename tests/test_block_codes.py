"""Planted mistakes in 8-bit rows on the CPU: the comparison shows a NaN code, a code one step off and a wrong scale."""
import pytest
import torch

import block_codes
import block_ref as ref

ROWS, HIDDEN = 3, 300


def _rows():
    g = torch.Generator().manual_seed(7)
    v = torch.randn(ROWS, HIDDEN, generator=g, dtype=torch.float64)
    pad = torch.nn.functional.pad(v, (0, ref.blocks(HIDDEN) * ref.BLOCK - HIDDEN)).view(ROWS, -1, ref.BLOCK)
    scales = (pad.abs().amax(2) / 448).float()
    codes = (v / ref.spread(scales.double(), HIDDEN)).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)
    return v, codes, scales, torch.zeros_like(v)


def test_good_rows_pass():
    v, codes, scales, bound = _rows()
    block_codes.close_codes(codes, scales, v, bound, "rows")


@pytest.mark.parametrize("at", [(0, 0), (1, 127), (1, 128), (2, 299)])
@pytest.mark.parametrize("code", [0x7F, 0xFF])
def test_a_nan_code_shows(at, code):
    v, codes, scales, bound = _rows()
    codes[at] = code
    ref.close_codes(codes, scales, v, bound, "rows")  # the comparison of the values alone does not see it
    with pytest.raises(AssertionError, match="NaN"):
        block_codes.close_codes(codes, scales, v, bound, "rows")


def test_all_nan_shows():
    v, codes, scales, bound = _rows()
    with pytest.raises(AssertionError, match="NaN"):
        block_codes.close_codes(torch.full_like(codes, 0x7F), scales, v, bound, "rows")


def test_a_number_for_nan_shows():
    v, codes, scales, bound = _rows()
    v[0, 0] = float("nan")
    with pytest.raises(AssertionError, match="NaN"):
        block_codes.close_codes(codes, scales, v, bound, "rows")


def test_a_wrong_code_and_a_wrong_scale_show():
    v, codes, scales, bound = _rows()
    at = (v.abs() > 1).nonzero()[0].tolist()
    codes[tuple(at)] += 2
    with pytest.raises(AssertionError, match="codes off"):
        block_codes.close_codes(codes, scales, v, bound, "rows")
    v, codes, scales, bound = _rows()
    scales[1, 1] *= 1.001
    with pytest.raises(AssertionError, match="scales"):
        block_codes.close_codes(codes, scales, v, bound, "rows")
