"""8-bit results and checkpoints of the norm: NaN codes nowhere but where the value is NaN, and the bits of the block codec on
the fp32 values that the formula gives (sums in rank order, the residual last; then h * rstd * gamma with the kernel's rstd)."""
import numpy as np
import pytest
import torch

import all_reduce_reduction_ring_amd as ar
import block_ref as ref
import oracle
from block_codes import close_codes
from test_gpu_block import BF16, DEV, E4M3, F16, F32, NORM, Guarded, gen, norm_inputs, randn

pytestmark = pytest.mark.gpu


def run(ins, res, gamma, eps, offset=0):
    rows, hidden = ins[0].shape
    put, nb, n = Guarded(offset), ref.blocks(hidden), len(ins)
    outs, sc = [put.new((rows, hidden), E4M3) for _ in range(n)], [put.new((rows, nb), F32) for _ in range(n)]
    rs, sv, svs = put.new((rows,), F32), put.new((rows, hidden), torch.uint8), put.new((rows, nb), F32)
    ar.ar_allreduce_rmsnorm(ins, gamma, outs, res, None, rs, sc, sv, svs, eps=eps)
    torch.cuda.synchronize()
    put.check()
    return outs, sc, rs, sv, svs


@pytest.mark.parametrize("n,rows,hidden,dt,residual,g32,offset",
                         [(c[0], c[1], c[2], c[3], c[4], c[7], c[8]) for c in NORM if c[5] or c[6]])
def test_no_code_is_nan(n, rows, hidden, dt, residual, g32, offset):
    ins, res, gamma = norm_inputs(n, rows, hidden, dt, residual, g32, offset)
    outs, sc, rs, sv, svs = run(ins, res, gamma, 1e-4, offset)
    h, rstd, y, dh, rel, dy = ref.norm(ins, res, gamma, 1e-4)
    for r in range(n):
        close_codes(outs[r], sc[r], y, dy, f"out {r}")
    close_codes(sv, svs, h, dh, "saved")


def assert_codec(codes, scales, values):
    codes, scales = codes.cpu().view(torch.uint8).numpy(), scales.cpu().numpy()
    for r, row in enumerate(values.cpu().numpy()):
        want, sc = oracle.fp8_quant(np.ascontiguousarray(row), oracle.F32)
        np.testing.assert_array_equal(codes[r], want)
        np.testing.assert_array_equal(scales[r].view(np.uint32), np.asarray(sc).view(np.uint32))


@pytest.mark.parametrize("n,rows,hidden,dt,residual", [
    (8, 3, 4096, BF16, True), (8, 3, 4096, F32, True), (2, 40, 64, F32, True), (3, 21, 127, F16, False), (4, 9, 129, F32, True),
    (2, 33, 200, BF16, True), (5, 7, 256, F32, False), (3, 6, 257, F32, True), (6, 5, 1000, F32, True), (7, 4, 2050, BF16, True),
    (16, 3, 520, F32, True), (2, 3, 3, F32, True), (3, 2, 8192, F32, True), (2, 2, 8200, F32, True), (1, 2, 16384, BF16, True),
    (2, 2, 16388, F32, True), (2, 2, 32767, F16, True)])
def test_the_codecs_bits(n, rows, hidden, dt, residual):
    """Rows from 2^-24 to 2^40 of their usual size, a block of zeros and single large elements among them."""
    g = gen(11)
    size = torch.logspace(-24 if dt != F16 else -6, 40 if dt != F16 else 4, rows, base=2, device=DEV)[:, None]
    mk = lambda: (randn(g, rows, hidden) * size).to(dt)
    ins, res = [mk() for _ in range(n)], mk() if residual else None
    for t in [*ins, *([res] if residual else [])]:
        t[rows // 2, :hidden // 3] = 0.0
    ins[0][0, hidden - 1] *= 300
    gamma = 1 + 0.3 * randn(g, hidden)
    outs, sc, rs, sv, svs = run(ins, res, gamma.to(dt) if dt == F32 else gamma, 1e-6)
    h = ins[0].float()
    for x in ins[1:]:
        h = h + x.float()
    if residual:
        h = h + res.float()
    assert_codec(sv, svs, h)
    y = h * rs[:, None]
    y = y * gamma
    for r in (0, n - 1):
        assert_codec(outs[r], sc[r], y)
