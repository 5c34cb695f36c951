"""Refusals of the experts' products: the library's own checks with addresses that no call reaches, and the binding's checks
of tensors. Nothing is launched."""
import pytest
import torch

import all_reduce_reduction_ring_amd as ar

BASE, STEP = 0x60000000, 1 << 28


def at(i):
    return BASE + i * STEP


def _gated(xs=at(0), wg=at(1), wu=at(2), stride=64 * 128, off=at(3), cnt=at(4), experts=4, rows=32, hidden=128, inner=64,
           dtype=ar.AR_BF16, act=0, out=at(5), gate=None, up=None):
    return ar.lib().ar_expert_gated(xs, wg, wu, stride, off, cnt, experts, rows, hidden, inner, dtype, act, out, gate, up,
                                    None)


def _gated_bwd(dout=at(0), gate=at(1), up=at(2), xs=at(3), wg=at(4), wu=at(5), stride=64 * 128, off=at(6), cnt=at(7),
               experts=4, rows=32, hidden=128, inner=64, dtype=ar.AR_BF16, act=0, dgate=at(8), dup=at(9), dxs=at(10),
               dwg=at(11), dwu=at(12), dstride=64 * 128):
    return ar.lib().ar_expert_gated_bwd(dout, gate, up, xs, wg, wu, stride, off, cnt, experts, rows, hidden, inner, dtype,
                                        act, dgate, dup, dxs, dwg, dwu, dstride, None)


def _linear(xs=at(0), w=at(1), stride=64 * 128, off=at(3), cnt=at(4), experts=4, rows=32, inside=128, out=64,
            dtype=ar.AR_BF16, ys=at(5)):
    return ar.lib().ar_expert_linear(xs, w, stride, off, cnt, experts, rows, inside, out, dtype, ys, None)


def _linear_bwd(dys=at(0), xs=at(1), w=at(2), stride=64 * 128, off=at(3), cnt=at(4), experts=4, rows=32, inside=128, out=64,
                dtype=ar.AR_BF16, dxs=at(5), dw=at(6), dstride=64 * 128):
    return ar.lib().ar_expert_linear_bwd(dys, xs, w, stride, off, cnt, experts, rows, inside, out, dtype, dxs, dw, dstride,
                                         None)


COMMON = [dict(dtype=9), dict(dtype=-1), dict(experts=0), dict(experts=ar.AR_MAX_EXPERTS + 1), dict(rows=1 << 31),
          dict(off=None), dict(off=None, cnt=None), dict(stride=64 * 128 - 1), dict(off=at(3) + 2), dict(stride=1 << 62)]


def test_gated_refusals():
    assert _gated(rows=0) == ar.AR_OK
    for bad in (*COMMON, dict(hidden=0), dict(inner=0), dict(act=3), dict(act=-1), dict(xs=None), dict(wg=None),
                dict(wu=None), dict(out=None), dict(gate=at(6)), dict(up=at(6)), dict(xs=at(0) + 1), dict(out=at(5) + 1),
                dict(wu=at(2) + 1), dict(gate=at(6) + 1, up=at(7))):
        assert _gated(**bad) == ar.AR_ERR_INVALID, bad
    for bad in (dict(dtype=ar.AR_I32), dict(hidden=ar.AR_PRODUCT_MAX_WIDTH + 1, stride=1 << 40),
                dict(inner=ar.AR_PRODUCT_MAX_WIDTH + 1, stride=1 << 40)):
        assert _gated(**bad) == ar.AR_ERR_UNSUPPORTED, bad
    for bad in (dict(out=at(0)), dict(out=at(0) + 2), dict(gate=at(5), up=at(7)), dict(gate=at(6), up=at(6)),
                dict(wu=at(1)), dict(wu=at(1) + 2 * (64 * 128 - 2)), dict(out=at(1)), dict(cnt=at(3) + 4),
                # halves of one tensor that are not quite halves
                dict(wu=at(1) + 2 * 64 * 128, stride=2 * 64 * 128 - 2)):
        assert _gated(**bad) == ar.AR_ERR_ALIAS, bad
    rec = ar.ar_last_call()
    assert rec["entry"] == "ar_expert_gated" and rec["status"] == ar.AR_ERR_ALIAS


def test_gated_bwd_refusals():
    for bad in (*[b if "off" not in b or b["off"] is None else dict(off=at(6) + 2) for b in COMMON], dict(act=3),
                dict(dout=None), dict(gate=None), dict(up=None), dict(xs=None), dict(wg=None), dict(wu=None),
                dict(dgate=None), dict(dup=None), dict(dwg=None), dict(dwu=None), dict(dstride=64 * 128 - 1),
                dict(dxs=at(10) + 1)):
        assert _gated_bwd(**bad) == ar.AR_ERR_INVALID, bad
    assert _gated_bwd(dtype=ar.AR_I32) == ar.AR_ERR_UNSUPPORTED
    for bad in (dict(dgate=at(8), dup=at(8)), dict(dgate=at(0), dup=at(0)), dict(dgate=at(1) + 2), dict(dxs=at(3)),
                dict(dxs=at(8)), dict(dwg=at(4)), dict(dwu=at(11)), dict(dgate=at(3))):
        assert _gated_bwd(**bad) == ar.AR_ERR_ALIAS, bad


def test_linear_refusals():
    assert _linear(rows=0) == ar.AR_OK
    for bad in (*COMMON, dict(inside=0), dict(out=0), dict(xs=None), dict(w=None), dict(ys=None), dict(ys=at(5) + 1)):
        assert _linear(**bad) == ar.AR_ERR_INVALID, bad
    assert _linear(dtype=ar.AR_I32) == ar.AR_ERR_UNSUPPORTED
    for bad in (dict(ys=at(0)), dict(ys=at(1) + 4 * 64 * 128), dict(ys=at(3))):
        assert _linear(**bad) == ar.AR_ERR_ALIAS, bad
    for bad in (*COMMON, dict(dys=None), dict(xs=None), dict(w=None), dict(dstride=5), dict(dw=at(6) + 1)):
        assert _linear_bwd(**bad) == ar.AR_ERR_INVALID, bad
    assert _linear_bwd(dtype=ar.AR_I32) == ar.AR_ERR_UNSUPPORTED
    for bad in (dict(dxs=at(0)), dict(dxs=at(1)), dict(dw=at(2)), dict(dw=at(5))):
        assert _linear_bwd(**bad) == ar.AR_ERR_ALIAS, bad


def test_too_many_tiles():
    """More tiles than the kernels count: refused, not wrapped."""
    wide = ar.AR_PRODUCT_MAX_WIDTH
    assert _linear(rows=1 << 20, inside=1, out=wide, xs=1 << 40, w=1 << 50, ys=1 << 51, off=1 << 52, cnt=1 << 53,
                   stride=wide) == ar.AR_ERR_UNSUPPORTED


def test_binding_refusals():
    """Host tensors, other types, shapes and layouts never reach the library."""
    x, w, y = torch.zeros(4, 8), torch.zeros(2, 6, 8), torch.zeros(4, 6)
    off, cnt = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: ar.ar_expert_linear(x, w, y, off, cnt), lambda: ar.ar_expert_linear(x, w, y, None, cnt),
                 lambda: ar.ar_expert_linear(x, None, y), lambda: ar.ar_expert_linear(x[0], w, y),
                 lambda: ar.ar_expert_gated(x, w, w, y, off, cnt), lambda: ar.ar_expert_gated(x.int(), w, w, y, off, cnt),
                 lambda: ar.ar_expert_gated_bwd(y, y, y, x, w, w, y, y, dw_gate=w, offsets=off),
                 lambda: ar.ar_expert_gated_bwd(y, y, y, None, w, w, y, y, dw_gate=w, dw_up=w, offsets=off),
                 lambda: ar.ar_expert_gated_bwd(y, y, y, x, None, w, y, y, dxs=x, offsets=off),
                 lambda: ar.ar_expert_linear_bwd(y, x, w), lambda: ar.ar_expert_linear_bwd(y, None, w, dw=w, dxs=x),
                 lambda: ar.ar_expert_linear_bwd(y, x, None, dxs=x)):
        with pytest.raises(ValueError):
            call()
