"""The norm over many gradient tensors and clipping against 64-bit references. The sum runs in 64 bits and the norm is
rounded once: half an fp32 step, and 2^-40 for the sums. A scaled element: the norm's error, one division, one product and
the rounding of its type: four half steps of fp32 and half a step of the type."""
import math

import pytest
import torch

import all_reduce_reduction_ring_amd as ar

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MIXED = (torch.float32, torch.bfloat16, torch.float16)


def tensors(sizes, dtypes, scale=0.01, seed=0, offset=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        base = torch.randn(n + offset, generator=g, device=DEV) * scale * (1 + i % 3)
        out.append(base.to(dtypes[i % len(dtypes)])[offset:])
    return out


def call(ts, outs=None, max_norm=None, kind=ar.AR_NORM_L2, eps=1e-6):
    plan = ar.ar_grad_plan(ts, outs)
    norm = torch.full((1,), -1.0, device=DEV)
    ws = torch.full((max(1, ar.ar_grad_norm_workspace_size(plan.shape[0])),), 0xFF, dtype=torch.uint8, device=DEV)
    if max_norm is None:
        ar.ar_grad_norm(plan, norm, kind=kind, workspace=ws)
    else:
        ar.ar_grad_clip(plan, max_norm, norm, kind=kind, eps=eps, workspace=ws)
    return norm.item()


def want_norm(ts, kind):
    if kind == ar.AR_NORM_MAX:
        return max((t.double().abs().max().item() for t in ts if t.numel()), default=0.0)
    return math.sqrt(math.fsum(t.double().square().sum().item() for t in ts))


SIZES = [[1], [0, 5, 0], [7, 1, 255, 257, 1003], [4096 * 3 + 1, 100003], [2049] * 300, [5_000_011, 17, 1_200_000]]


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("dtypes", [MIXED, MIXED[:1], MIXED[1:2], MIXED[2:]], ids=["mixed", "f32", "bf16", "f16"])
@pytest.mark.parametrize("which", range(len(SIZES)))
def test_norm_and_clip(which, dtypes, offset):
    for kind in (ar.AR_NORM_L2, ar.AR_NORM_MAX):
        ts = tensors(SIZES[which], dtypes, seed=which, offset=offset)
        want = want_norm(ts, kind)
        norm = call(ts, kind=kind)
        assert abs(norm - want) <= want * (2 ** -24 + 2 ** -40)
        for share in (0.37, 2.0):
            outs = [torch.full_like(t, 3.0) for t in ts]
            before = [t.clone() for t in ts]
            assert call(ts, outs, want * share, kind) == norm
            coef = min(1.0, want * share / (want + 1e-6))
            for t, b, o in zip(ts, before, outs):
                assert torch.equal(t, b)
                v = t.double() * coef
                f = torch.finfo(t.dtype)
                assert ((o.double() - v).abs() <= v.abs() * (4 * 2 ** -24 + f.eps / 2) + f.smallest_normal * f.eps).all()
            assert call(ts, None, want * share, kind) == norm  # in place
            for t, o in zip(ts, outs):
                assert torch.equal(t, o)
            if share > 1:
                assert all(torch.equal(t, b) for t, b in zip(ts, before))
            for t, b in zip(ts, before):
                t.copy_(b)


def test_neighbours_are_left_alone():
    """Elements before and behind a tensor, also where its last piece ends inside a vector."""
    for dtype in MIXED:
        for n in (1, 7, 8, 2047, 2049, 40003):
            base = torch.ones(n + 40, dtype=dtype, device=DEV)
            call([base[17:17 + n]], None, 1e-3)
            assert (base[:17] == 1).all() and (base[17 + n:] == 1).all() and (base[17:17 + n] < 1).all()


def test_far_numbers():
    """Squares that leave fp32 at either end; infinities and NaN."""
    big, small = torch.full((1000,), 1e30, device=DEV), torch.full((1000,), 1e-30, device=DEV)
    assert call([big]) == pytest.approx(1e30 * math.sqrt(1000), rel=2e-7)
    assert call([small]) == pytest.approx(1e-30 * math.sqrt(1000), rel=2e-7)
    sub = torch.full((64,), 2.0 ** -24, dtype=torch.float16, device=DEV)
    assert call([sub]) == 2.0 ** -21 and call([sub], kind=ar.AR_NORM_MAX) == 2.0 ** -24
    for kind in (ar.AR_NORM_L2, ar.AR_NORM_MAX):
        for value, check in ((math.inf, math.isinf), (-math.inf, math.isinf), (math.nan, math.isnan)):
            for dtype in MIXED:
                t = torch.ones(70000, dtype=dtype, device=DEV)
                t[69999] = value
                assert check(call([big, t], kind=kind))
    t = torch.ones(500, device=DEV)
    t[3] = math.nan
    call([t], None, 1.0)
    assert t.isnan().all()
    t = torch.ones(500, device=DEV)
    t[3] = math.inf
    call([t], None, 1.0)
    assert t[3].isnan() and (t[:3] == 0).all() and (t[4:] == 0).all()
    t = torch.ones(500, device=DEV)
    assert call([t], None, math.inf) == pytest.approx(math.sqrt(500)) and (t == 1).all()
    call([t], None, 0.0)
    assert (t == 0).all()


def test_bounds_that_the_norm_just_meets():
    """0 / 0 and inf / inf are no scale: zeros under a bound of 0 without eps stay, and no bound leaves infinities alone."""
    for kind in (ar.AR_NORM_L2, ar.AR_NORM_MAX):
        t, out = torch.zeros(300, device=DEV), torch.full((300,), 7.0, device=DEV)
        assert call([t], [out], 0.0, kind, eps=0.0) == 0.0 and (out == 0).all()
        t = torch.ones(300, device=DEV)
        t[5] = math.inf
        want = t.clone()
        assert math.isinf(call([t], None, math.inf, kind)) and torch.equal(t, want)
        t = torch.full((300,), 3.0, device=DEV)
        exact = math.sqrt(2700.0) if kind == ar.AR_NORM_L2 else 3.0
        norm = torch.tensor(exact, dtype=torch.float32).item()
        call([t], [out], norm, kind, eps=0.0)
        assert torch.equal(out, t)
        assert math.isnan(call([torch.full((3,), math.nan, device=DEV)], [out[:3]], math.inf, kind)) and out[:3].isnan().all()


def test_without_elements():
    empty = torch.empty(0, device=DEV)
    assert call([empty]) == 0.0 and call([empty], None, 1.0) == 0.0


def test_same_table_same_bits():
    """The order of the sum is the table's: repeated calls agree, on another stream and in a graph too."""
    ts = tensors([3_000_001, 70_003, 5], MIXED, seed=9)
    outs = [torch.empty_like(t) for t in ts]
    plan, norm = ar.ar_grad_plan(ts, outs), torch.empty(1, device=DEV)
    ws = torch.empty(ar.ar_grad_norm_workspace_size(plan.shape[0]), dtype=torch.uint8, device=DEV)
    ar.ar_grad_clip(plan, 0.5, norm, workspace=ws)
    first = [norm.clone()] + [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        ar.ar_grad_clip(plan, 0.5, norm, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, [norm] + outs))
    with torch.cuda.graph(graph):
        ar.ar_grad_clip(plan, 0.5, norm, workspace=ws)
    for i in range(4):
        for t in [norm] + outs:
            t.fill_(9.0)
        ws.fill_(0xFF)
        if i == 2:  # other gradients in the same place
            for t in ts:
                t.mul_(2.0)
            want = want_norm(ts, ar.AR_NORM_L2)
        graph.replay()
        torch.cuda.synchronize()
        if i < 2:
            assert all(torch.equal(a, b) for a, b in zip(first, [norm] + outs))
        else:
            assert abs(norm.item() - want) <= want * 2 ** -23


def test_device_refusals():
    t, n = torch.ones(8, device=DEV), torch.empty(1, device=DEV)
    plan = ar.ar_grad_plan([t])
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    for bad in (dict(workspace=None), dict(workspace=ws[:0])):
        with pytest.raises(ar.ArError):
            ar.ar_grad_norm(plan, n, **bad)
    for bad in (lambda: ar.ar_grad_plan([t, t]), lambda: ar.ar_grad_plan([t], [t[:7]]), lambda: ar.ar_grad_plan([t, t[2:4]]),
                lambda: ar.ar_grad_plan([t.int()]), lambda: ar.ar_grad_plan([t], [t.half()]),
                lambda: ar.ar_grad_norm(plan[:, :3], n, workspace=ws), lambda: ar.ar_grad_norm(plan.int(), n, workspace=ws),
                lambda: ar.ar_grad_norm(plan, n.double(), workspace=ws), lambda: ar.ar_grad_norm(plan, t, workspace=ws),
                lambda: ar.ar_grad_norm(plan, n.cpu(), workspace=ws), lambda: ar.ar_grad_norm(plan, n, kind=2, workspace=ws),
                lambda: ar.ar_grad_clip(plan, -1.0, n, workspace=ws), lambda: ar.ar_grad_clip(plan, math.nan, n, workspace=ws),
                lambda: ar.ar_grad_clip(plan, 1.0, n, eps=-1.0, workspace=ws)):
        with pytest.raises((ValueError, ar.ArError)):
            bad()
