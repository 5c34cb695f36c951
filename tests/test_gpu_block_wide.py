"""Wide rows: just below 2^31 bytes, the widest that the expert entry points take, where every byte arrives and none beside
them; and the norm and its gradient above 8192 elements, streaming and not."""
import pytest
import torch

import all_reduce_reduction_ring_amd as ar
import block_ref as ref
from test_gpu_block import BF16, E4M3, F16, F32, Guarded, norm_inputs
from test_gpu_block_paths import check_bwd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
GUARD = 1 << 16


def _guarded(nbytes):
    base = torch.full((nbytes + 2 * GUARD,), 0x5A, dtype=torch.uint8, device=DEV)
    return base, base[GUARD:GUARD + nbytes]


def _untouched(base, nbytes):
    return bool((base[:GUARD] == 0x5A).all()) and bool((base[GUARD + nbytes:] == 0x5A).all())


@pytest.mark.parametrize("short_by,es", [(1, 1), (15, 1), (17, 1), (8191, 1), (2, 2), (8190, 2), (4, 4), (16, 4)])
def test_dispatch(short_by, es):
    n = 2 ** 31 - short_by
    dt = {1: torch.uint8, 2: torch.float16, 4: torch.float32}[es]
    x = torch.randint(0, 256, (n,), dtype=torch.uint8, device=DEV)
    base, out = _guarded(n)
    pos = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    scales = {}
    if es == 1:
        sc = torch.rand(1, -(-n // 128), device=DEV)
        scales = dict(x_scales=sc, xs_scales=torch.zeros_like(sc))
    ar.ar_expert_dispatch(x.view(dt)[None], pos, None, None, out.view(dt)[None], **scales)
    torch.cuda.synchronize()
    assert _untouched(base, n) and torch.equal(out, x)
    if es == 1:
        assert torch.equal(scales["xs_scales"], scales["x_scales"])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_combine_and_its_gradient(dt):
    n = 2 ** 31 - dt.itemsize
    hidden = n // dt.itemsize
    y = torch.empty(hidden, dtype=dt, device=DEV)
    y.view(torch.uint8).view(torch.int16)[:] = 0x3F80  # 1.0 in bfloat16, 1.00194... in float32
    y[::1023] = -2.0
    base, out = _guarded(n)
    pos, w = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.full((1, 1), 0.5, device=DEV)
    ar.ar_expert_combine(y[None], pos, out.view(dt)[None], w)
    torch.cuda.synchronize()
    assert _untouched(base, n) and torch.equal(out.view(dt), y * 0.5)
    base.fill_(0x5A)
    dw = torch.empty(1, 1, device=DEV)
    ar.ar_expert_combine_bwd(y[None], y.clone()[None], pos, w, None, None, out.view(dt)[None], dw)
    torch.cuda.synchronize()
    assert _untouched(base, n) and torch.equal(out.view(dt), y * 0.5)


def test_sort_up_to_the_last_row():
    """One segment of 2^31 - 1 rows, all but one of them pads."""
    align = 2 ** 31 - 1
    rows = ar.ar_expert_rows(1, 1, 1, align)
    assert rows == align
    i32 = torch.int32
    base = torch.full((rows + 2 * GUARD,), 77, dtype=i32, device=DEV)
    src = base[GUARD:GUARD + rows]
    off, cnt, pos = torch.empty(2, dtype=i32, device=DEV), torch.empty(1, dtype=i32, device=DEV), torch.empty(1, 1, dtype=i32, device=DEV)
    ar.ar_expert_sort(torch.zeros(1, 1, dtype=i32, device=DEV), off, cnt, pos, src, align)
    torch.cuda.synchronize()
    assert off.tolist() == [0, rows] and cnt.tolist() == [1] and pos.tolist() == [[0]]
    assert src[0].item() == 0 and bool((src[1:] == -1).all())
    assert bool((base[:GUARD] == 77).all()) and bool((base[GUARD + rows:] == 77).all())


@pytest.mark.parametrize("n,rows,hidden,dt,streaming", [
    (1, 1100, 16384, BF16, True), (2, 600, 16384, F32, True), (4, 300, 32768, BF16, True), (5, 460, 12288, F16, True),
    (8, 70, 32768, F32, True), (4, 100, 32768, BF16, False), (2, 100, 8256, F32, False)])
def test_norm_and_its_gradient(n, rows, hidden, dt, streaming):
    assert (rows * hidden * dt.itemsize * (2 * n + 2) >= 128 << 20) == streaming
    ins, res, gamma = norm_inputs(n, rows, hidden, dt, True, False, 0)
    nb, put = ref.blocks(hidden), Guarded(0)
    h, rstd, y, dh, rel, dy = ref.norm(ins, res, gamma, 1e-4)
    for out8 in (False, True):
        outs = [put.new((rows, hidden), E4M3 if out8 else dt) for _ in range(n)]
        sc = [put.new((rows, nb), F32) for _ in range(n)] if out8 else None
        ro, rs = put.new((rows, hidden), dt), put.new((rows,), F32)
        ar.ar_allreduce_rmsnorm(ins, gamma, outs, res, ro, rs, sc, eps=1e-4)
        torch.cuda.synchronize()
        put.check()
        ref.close(ro, h, dh, "residual_out")
        ref.close(rs[:, None], rstd, rel * rstd, "rstd")
        for r in (0, n - 1):
            if out8:
                ref.close_codes(outs[r], sc[r], y, dy, f"out {r}")
            else:
                ref.close(outs[r], y, dy, f"out {r}")
    for in_place in (False, True):
        check_bwd(n, rows, hidden, dt, True, in_place, 0, in_place)
