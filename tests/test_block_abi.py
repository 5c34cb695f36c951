"""Refusals of the block-boundary entry points: the library's own checks with addresses that no call reaches, and the
binding's checks of tensors. Nothing is launched."""
import ctypes
import math

import pytest
import torch

import all_reduce_reduction_ring_amd as ar

BASE, STEP = 0x60000000, 1 << 24


def _ptrs(n, first=0):
    return [BASE + (first + r) * STEP for r in range(n)]


def _arr(ps):
    return None if ps is None else (ctypes.c_void_p * len(ps))(*ps)


def _norm(n=2, rows=4, hidden=256, dtype=ar.AR_BF16, gdt=ar.AR_BF16, eps=1e-5, ins="", outs="", residual=None, gamma="",
          out_scales=None, residual_out=None, rstd=None, saved=None, saved_scales=None):
    m = max(n, 1)
    ins = _ptrs(m) if ins == "" else ins
    outs = _ptrs(m, 100) if outs == "" else outs
    gamma = BASE + 300 * STEP if gamma == "" else gamma
    return ar.lib().ar_allreduce_rmsnorm(_arr(ins), n, rows, hidden, dtype, residual, gamma, gdt, eps, _arr(outs),
                                         _arr(out_scales), residual_out, rstd, saved, saved_scales, None)


def test_norm_refusals():
    assert _norm(rows=0) == ar.AR_OK
    for bad in (dict(n=0), dict(n=65), dict(hidden=0), dict(dtype=9), dict(gdt=9), dict(gdt=ar.AR_F16),
                dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf), dict(gamma=None), dict(ins=None),
                dict(outs=None), dict(ins=[BASE, 0]), dict(outs=[BASE + STEP * 9, 0]), dict(ins=[BASE + 1, BASE + STEP]),
                dict(gamma=BASE + 300 * STEP + 1), dict(saved=BASE + 400 * STEP), dict(rstd=BASE + 400 * STEP + 2),
                dict(out_scales=[BASE + 400 * STEP, 0]), dict(rows=1 << 60), dict(residual=BASE + 401 * STEP + 1)):
        assert _norm(**bad) == ar.AR_ERR_INVALID, bad
    assert _norm(dtype=ar.AR_I32, gdt=ar.AR_I32) == ar.AR_ERR_UNSUPPORTED
    assert _norm(hidden=ar.AR_NORM_MAX_HIDDEN + 1) == ar.AR_ERR_UNSUPPORTED
    far = BASE + 400 * STEP
    for bad in (dict(ins=[BASE, BASE + 64]), dict(outs=[BASE + 64, BASE + 200 * STEP]), dict(residual=BASE),
                dict(outs=[BASE + STEP, BASE]), dict(residual_out=BASE), dict(rstd=BASE + 16),
                dict(residual=far, residual_out=far + 16), dict(saved=far, saved_scales=far + 16),
                dict(outs=_ptrs(2), out_scales=_ptrs(2, 500))):  # codes do not go over the inputs
        assert _norm(**bad) == ar.AR_ERR_ALIAS, bad
    rec = ar.ar_last_call()
    assert rec["entry"] == "ar_allreduce_rmsnorm" and rec["nranks"] == 2 and rec["status"] == ar.AR_ERR_ALIAS


def _bwd(n=2, rows=4, hidden=256, dtype=ar.AR_BF16, gdt=ar.AR_BF16, ins="", outs="", saved=BASE + 300 * STEP,
         saved_scales=None, gamma=BASE + 301 * STEP, rstd=BASE + 302 * STEP, rg=None, dgamma=BASE + 303 * STEP,
         ws=BASE + 304 * STEP, wsb=1 << 22):
    m = max(n, 1)
    return ar.lib().ar_allreduce_rmsnorm_bwd(_arr(_ptrs(m) if ins == "" else ins), n, rows, hidden, dtype, saved,
                                             saved_scales, gamma, gdt, rstd, rg,
                                             _arr(_ptrs(m, 100) if outs == "" else outs), dgamma, ws, wsb, None)


def test_norm_bwd_refusals():
    for bad in (dict(n=0), dict(hidden=0), dict(dtype=9), dict(gdt=ar.AR_F16), dict(saved=None), dict(gamma=None),
                dict(rstd=None), dict(dgamma=None), dict(ins=None), dict(outs=[BASE + STEP * 9, 0]),
                dict(ws=BASE + 304 * STEP + 128), dict(rg=BASE + 305 * STEP + 1), dict(dgamma=BASE + 303 * STEP + 2)):
        assert _bwd(**bad) == ar.AR_ERR_INVALID, bad
    need = ar.ar_allreduce_rmsnorm_bwd_workspace_size(4, 256)
    assert need >= 4
    assert _bwd(ws=None) == ar.AR_ERR_WORKSPACE and _bwd(wsb=need - 1) == ar.AR_ERR_WORKSPACE
    assert _bwd(dtype=ar.AR_I32, gdt=ar.AR_I32) == ar.AR_ERR_UNSUPPORTED
    assert _bwd(hidden=ar.AR_NORM_MAX_HIDDEN + 1) == ar.AR_ERR_UNSUPPORTED
    for bad in (dict(ws=BASE), dict(dgamma=BASE + 64), dict(rg=BASE), dict(saved=BASE + 100 * STEP),
                dict(outs=[BASE + 305 * STEP] * 2, rg=BASE + 305 * STEP)):  # one rank in place of it at most
        assert _bwd(**bad) == ar.AR_ERR_ALIAS, bad
    with pytest.raises(ar.ArError):
        ar.ar_allreduce_rmsnorm_bwd_workspace_size(4, 0)
    with pytest.raises(ar.ArError):
        ar.ar_allreduce_rmsnorm_bwd_workspace_size(4, ar.AR_NORM_MAX_HIDDEN + 1)


def test_expert_rows_and_workspace():
    assert ar.ar_expert_rows(10, 2, 4) == 20
    assert ar.ar_expert_rows(10, 2, 4, 16) == 20 + 4 * 15
    assert ar.ar_expert_rows(1, 2, 64, 16) == 2 + 2 * 15  # no more than two experts can have rows
    assert ar.ar_expert_rows(0, 2, 4, 16) == 0
    assert ar.ar_expert_sort_workspace_size(1, 1, 1024) == 0
    for tokens in (10_000, 1 << 20, 1 << 27):  # never more than 513 tiles
        assert 0 < ar.ar_expert_sort_workspace_size(tokens, 8, 256) <= 513 * 256 * 4
    for bad in ((10, 0, 4, 1), (10, 2, 0, 1), (10, 2, ar.AR_MAX_EXPERTS + 1, 1), (10, 2, 4, 0), (1 << 31, 1, 4, 1),
                (1 << 62, 8, 4, 1), (1 << 20, 8, 1024, 1 << 22)):
        with pytest.raises(ar.ArError):
            ar.ar_expert_rows(*bad)


def _sort(ids=BASE, tokens=100, k=2, experts=8, align=4, offsets=BASE + STEP, counts=BASE + 2 * STEP,
          pos=BASE + 3 * STEP, src=BASE + 4 * STEP, rows=None, ws=None, wsb=0):
    rows = tokens * k + 8 * 3 if rows is None else rows
    return ar.lib().ar_expert_sort(ids, tokens, k, experts, align, offsets, counts, pos, src, rows, ws, wsb, None)


def test_sort_refusals():
    for bad in (dict(ids=None), dict(offsets=None), dict(counts=None), dict(pos=None), dict(src=None), dict(k=0),
                dict(experts=0), dict(experts=1025), dict(align=0), dict(rows=200), dict(rows=1 << 31),
                dict(ids=BASE + 2), dict(tokens=1 << 31, rows=1 << 30)):
        assert _sort(**bad) == ar.AR_ERR_INVALID, bad
    assert _sort(tokens=1 << 20) == ar.AR_ERR_WORKSPACE
    need = ar.ar_expert_sort_workspace_size(1 << 20, 2, 8)
    assert _sort(tokens=1 << 20, ws=BASE + 9 * STEP, wsb=need - 1) == ar.AR_ERR_WORKSPACE
    assert _sort(tokens=1 << 20, ws=BASE + 9 * STEP + 4, wsb=need) == ar.AR_ERR_INVALID
    assert _sort(tokens=1 << 20, ws=BASE, wsb=need) == ar.AR_ERR_ALIAS
    assert _sort(pos=BASE) == ar.AR_ERR_ALIAS and _sort(counts=BASE + STEP) == ar.AR_ERR_ALIAS


def _dispatch(x=BASE, xsc=None, pos=BASE + STEP, off=BASE + 2 * STEP, cnt=BASE + 3 * STEP, tokens=10, k=2, experts=4,
              hidden=100, es=2, xs=BASE + 4 * STEP, xssc=None, rows=40):
    return ar.lib().ar_expert_dispatch(x, xsc, pos, off, cnt, tokens, k, experts, hidden, es, xs, xssc, rows, None)


def test_dispatch_refusals():
    assert _dispatch(tokens=0) == ar.AR_OK
    for bad in (dict(x=None), dict(pos=None), dict(xs=None), dict(off=None), dict(cnt=None), dict(hidden=0),
                dict(es=3), dict(es=8), dict(k=0), dict(experts=0), dict(x=BASE + 1), dict(xsc=BASE + 5 * STEP),
                dict(xsc=BASE + 5 * STEP, xssc=BASE + 6 * STEP), dict(rows=1 << 31), dict(hidden=1 << 62)):
        assert _dispatch(**bad) == ar.AR_ERR_INVALID, bad
    assert _dispatch(xs=BASE) == ar.AR_ERR_ALIAS and _dispatch(xs=BASE + STEP) == ar.AR_ERR_ALIAS


def _combine(ys=BASE, pos=BASE + STEP, w=BASE + 2 * STEP, add=None, tokens=10, k=2, hidden=100, dtype=ar.AR_BF16,
             rows=40, out=BASE + 3 * STEP):
    return ar.lib().ar_expert_combine(ys, pos, w, add, tokens, k, hidden, dtype, rows, out, None)


def _combine_bwd(dout=BASE, ys=BASE + STEP, pos=BASE + 2 * STEP, w=BASE + 3 * STEP, off=None, cnt=None, tokens=10, k=2,
                 experts=4, hidden=100, dtype=ar.AR_BF16, rows=40, dys=BASE + 4 * STEP, dw=BASE + 5 * STEP):
    return ar.lib().ar_expert_combine_bwd(dout, ys, pos, w, off, cnt, tokens, k, experts, hidden, dtype, rows, dys, dw,
                                          None)


def test_combine_refusals():
    assert _combine(tokens=0) == ar.AR_OK and _combine_bwd(tokens=0) == ar.AR_OK
    for bad in (dict(ys=None), dict(pos=None), dict(out=None), dict(hidden=0), dict(k=0), dict(dtype=9),
                dict(out=BASE + 3 * STEP + 1), dict(add=BASE + 9 * STEP + 1), dict(w=BASE + 2 * STEP + 2)):
        assert _combine(**bad) == ar.AR_ERR_INVALID, bad
    for bad in (dict(dout=None), dict(ys=None), dict(pos=None), dict(w=None), dict(dys=None), dict(dw=None),
                dict(off=BASE + 9 * STEP), dict(cnt=BASE + 9 * STEP), dict(experts=0), dict(dtype=-1)):
        assert _combine_bwd(**bad) == ar.AR_ERR_INVALID, bad
    assert _combine(dtype=ar.AR_I32) == ar.AR_ERR_UNSUPPORTED
    assert _combine_bwd(dtype=ar.AR_I32) == ar.AR_ERR_UNSUPPORTED
    assert _combine(out=BASE) == ar.AR_ERR_ALIAS and _combine(add=BASE + 3 * STEP + 200) == ar.AR_ERR_ALIAS
    assert _combine_bwd(dys=BASE) == ar.AR_ERR_ALIAS and _combine_bwd(dw=BASE + 3 * STEP) == ar.AR_ERR_ALIAS


def test_binding_refuses_tensors_that_do_not_fit():
    """Host tensors (and wrong types, shapes and orders) never become addresses."""
    z = torch.zeros
    m, g = z(4, 256), z(256)
    i = lambda *s: z(*s, dtype=torch.int32)
    calls = [
        lambda: ar.ar_allreduce_rmsnorm([m], g, [m]),
        lambda: ar.ar_allreduce_rmsnorm([], g, []),
        lambda: ar.ar_allreduce_rmsnorm([m[0]], g, [m]),
        lambda: ar.ar_allreduce_rmsnorm([m.int()], g, [m]),
        lambda: ar.ar_allreduce_rmsnorm_bwd([m], m, g, z(4), [m], g),
        lambda: ar.ar_expert_sort(i(4, 2), i(9), i(8), i(4, 2), i(8)),
        lambda: ar.ar_expert_sort(i(8), i(9), i(8), i(8), i(8)),
        lambda: ar.ar_expert_dispatch(m, i(4, 2), None, None, z(8, 256)),
        lambda: ar.ar_expert_dispatch(m.to(torch.uint8), i(4, 2), None, None, z(8, 256, dtype=torch.uint8)),
        lambda: ar.ar_expert_dispatch(m, i(4, 2), i(9), None, z(8, 256)),
        lambda: ar.ar_expert_combine(z(8, 256), i(4, 2), m),
        lambda: ar.ar_expert_combine_bwd(m, z(8, 256), i(4, 2), z(4, 2), None, None, z(8, 256), z(4, 2)),
    ]
    for k, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was not refused")
