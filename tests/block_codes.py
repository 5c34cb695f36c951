"""8-bit rows against 64 bits, NaN codes included: block_ref's comparison alone is false for a NaN, so a code that stands for
none of the values passes it."""
import torch

import block_ref as ref


def close_codes(codes, scales, want, bound, what):
    v = ref.codes_f64(codes)
    bad = torch.isnan(v) != torch.isnan(want)
    assert not bad.any(), f"{what}: {int(bad.sum())} codes are NaN, or not NaN, in the wrong place, first at {bad.nonzero()[0].tolist()}"
    assert torch.isfinite(ref.f64(scales)).all(), f"{what}: scales"
    ref.close_codes(codes, scales, want, bound, what)
