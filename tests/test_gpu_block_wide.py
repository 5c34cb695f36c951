"""Rows just below 2^31 bytes, the widest that the expert entry points take: every byte arrives, none beside them."""
import pytest
import torch

import all_reduce_reduction_ring_amd as ar

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
