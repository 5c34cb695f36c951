"""The plan of the gradients' norm: pieces cover every tensor once, in bounds, and the refusals. Host only."""
import ctypes

import numpy as np
import pytest
import torch

import all_reduce_reduction_ring_amd as ar

PIECE = np.dtype([("in", np.uint64), ("out", np.uint64), ("numel", np.int64), ("dtype", np.int32), ("reserved", np.int32)])
SIZE = {ar.AR_F32: 4, ar.AR_BF16: 2, ar.AR_F16: 2}


def plan(rows, room=None):
    table = np.array([tuple(r) + (0,) for r in rows], PIECE)
    n = ctypes.c_size_t(0)
    rc = ar.lib().ar_grad_plan(table.ctypes.data if len(rows) else None, len(rows), None, ctypes.byref(n))
    if rc != ar.AR_OK:
        return rc, None
    pieces = np.zeros(n.value + 1, PIECE)
    m = ctypes.c_size_t(n.value if room is None else room)
    rc = ar.lib().ar_grad_plan(table.ctypes.data if len(rows) else None, len(rows), pieces.ctypes.data, ctypes.byref(m))
    assert rc != ar.AR_OK or m.value == n.value
    assert pieces[-1]["in"] == 0
    return rc, pieces[:n.value]


BASE = 1 << 40


@pytest.mark.parametrize("dtype", SIZE)
@pytest.mark.parametrize("sizes", [[1], [0, 3, 0], [2047, 2048, 2049], [1 << 20, 5], [(1 << 26) + 3, 1], [1003 * 77] * 40])
@pytest.mark.parametrize("shift", [0, 1, 63])
def test_pieces_cover_every_tensor(sizes, dtype, shift):
    es, at, rows = SIZE[dtype], BASE + shift * SIZE[dtype], []
    for i, n in enumerate(sizes):
        rows.append((at, 0 if i % 2 else at + (1 << 38), n, dtype))
        at += n * es
    rc, pieces = plan(rows)
    assert rc == ar.AR_OK
    i = 0
    for start, out, n, _ in rows:
        done = 0
        while done < n:
            p = pieces[i]
            assert p["in"] == start + done * es and p["dtype"] == dtype and p["reserved"] == 0
            assert p["out"] == (out + done * es if out else 0)
            assert 0 < p["numel"] * es <= 32768
            done += int(p["numel"])
            i += 1
            assert done == n or (start + done * es) % 256 == 0
        assert done == n
    assert i == len(pieces)
    total = sum(sizes) * es
    assert len(pieces) <= max(2 * 1024, total // 32768) + 2 * len(sizes) + 1


def test_refusals():
    f32 = ar.AR_F32
    assert plan([])[0] == ar.AR_OK
    assert plan([(0, 0, 0, f32)])[0] == ar.AR_OK
    for bad in ([(0, 0, 1, f32)], [(BASE + 2, 0, 1, f32)], [(BASE, BASE + 4097, 1, ar.AR_BF16)], [(BASE, 0, -1, f32)],
                [(BASE, 0, 1, 9)], [(BASE, 0, 1 << 61, f32)], [(2 ** 64 - 8, 0, 4, f32)]):
        assert plan(bad)[0] == ar.AR_ERR_INVALID, bad
    assert plan([(BASE, 0, 1, ar.AR_I32)])[0] == ar.AR_ERR_UNSUPPORTED
    for bad in ([(BASE, 0, 8, f32)] * 2, [(BASE, 0, 8, f32), (BASE + 16, 0, 8, f32)], [(BASE, BASE + 4, 8, f32)],
                [(BASE, BASE + 64, 8, f32), (BASE + 64, 0, 8, f32)]):
        assert plan(bad)[0] == ar.AR_ERR_ALIAS, bad
    assert plan([(BASE, BASE, 8, f32)])[0] == ar.AR_OK
    assert plan([(BASE, 0, 1 << 20, f32)], room=3)[0] == ar.AR_ERR_INVALID
    n = ctypes.c_size_t(0)
    assert ar.lib().ar_grad_plan(None, 1, None, ctypes.byref(n)) == ar.AR_ERR_INVALID
    assert ar.lib().ar_grad_plan(None, -1, None, ctypes.byref(n)) == ar.AR_ERR_INVALID
    assert ar.lib().ar_grad_plan(None, 0, None, None) == ar.AR_ERR_INVALID


def test_call_refusals():
    L, ws = ar.lib(), BASE + 4096
    need = ar.ar_grad_norm_workspace_size(5)
    assert need == 40 and ar.ar_grad_norm_workspace_size(10 ** 6) == 8192 and ar.ar_grad_norm_workspace_size(0) == 0
    with pytest.raises(ar.ArError):
        ar.ar_grad_norm_workspace_size(1 << 31)
    with pytest.raises(ValueError):
        ar.ar_grad_norm_workspace_size(-1)
    ok = dict(pieces=BASE, n=5, kind=0, norm=BASE + 1024, ws=ws, wsb=need)

    def norm(**kw):
        a = {**ok, **kw}
        return L.ar_grad_norm(a["pieces"], a["n"], a["kind"], a["norm"], a["ws"], a["wsb"], None)

    def clip(max_norm=1.0, eps=1e-6, **kw):
        a = {**ok, **kw}
        return L.ar_grad_clip(a["pieces"], a["n"], a["kind"], max_norm, eps, a["norm"], a["ws"], a["wsb"], None)

    for f in (norm, clip):
        for bad in (dict(pieces=None), dict(pieces=BASE + 4), dict(kind=2), dict(kind=-1), dict(norm=None),
                    dict(norm=BASE + 1026), dict(n=1 << 31), dict(ws=ws + 8)):
            assert f(**bad) == ar.AR_ERR_INVALID, bad
        assert f(ws=None) == ar.AR_ERR_WORKSPACE and f(wsb=need - 1) == ar.AR_ERR_WORKSPACE
        for bad in (dict(norm=BASE), dict(norm=ws), dict(ws=BASE)):
            assert f(**bad) == ar.AR_ERR_ALIAS, bad
    for bad in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(eps=-1.0), dict(eps=float("inf")),
                dict(eps=float("nan"))):
        assert clip(**bad) == ar.AR_ERR_INVALID, bad
    for bad in (lambda: ar.ar_grad_plan([]), lambda: ar.ar_grad_plan([torch.ones(4)])):
        with pytest.raises(ValueError):
            bad()
