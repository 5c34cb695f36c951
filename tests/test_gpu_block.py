"""The block-boundary operators on the GPU against the 64-bit references of block_ref.py."""
import numpy as np
import pytest
import torch

import all_reduce_reduction_ring_amd as ar
import block_ref as ref
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4M3 = torch.float8_e4m3fn
GUARD = 512  # spare bytes on each side of every output


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


class Guarded:
    """Output tensors inside larger allocations, `offset` elements in, whose surroundings must stay as they were."""

    def __init__(self, offset=0):
        self.offset, self.all = offset, []

    def new(self, shape, dtype, fill=None):
        n = int(np.prod(shape)) * dtype.itemsize
        base = torch.full((n + 2 * GUARD + 64,), 0x5A, dtype=torch.uint8, device=DEV)
        lo = GUARD + self.offset * dtype.itemsize
        self.all.append((base, lo, n))
        t = base[lo:lo + n].view(dtype).view(shape)
        if fill is not None:
            t.copy_(fill)
        return t

    def check(self):
        for base, lo, n in self.all:
            assert bool((base[:lo] == 0x5A).all()) and bool((base[lo + n:] == 0x5A).all()), "written outside an output"


def workspace(nbytes):
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=DEV)


# ------------------------------------------------------------------------------------------------ norm
NORM = [  # ranks, rows, hidden, dtype, residual, 8-bit out, 8-bit saved, gamma in fp32, offset in elements
    (1, 1, 1, BF16, False, False, False, False, 0),
    (1, 1, 1, F32, True, True, True, False, 0),
    (8, 1, 4096, BF16, True, False, False, False, 0),
    (8, 5, 4096, BF16, True, True, True, False, 0),
    (2, 3, 8192, F16, True, True, False, True, 0),
    (3, 33, 1003, F16, False, False, True, False, 1),
    (3, 17, 2050, F32, True, True, True, False, 1),
    (4, 9, 127, BF16, True, True, True, True, 3),
    (4, 9, 129, F32, False, True, True, False, 0),
    (5, 64, 64, BF16, True, False, True, False, 0),
    (16, 7, 520, F16, True, True, False, False, 5),
    (64, 3, 300, BF16, True, False, False, True, 0),
    (6, 700, 640, F32, True, False, False, False, 0),
    (7, 2, 16384, BF16, True, True, True, False, 0),
    (1, 2, 32768, F32, True, True, True, False, 0),
    (2, 2, 32767, BF16, True, True, True, False, 1),
    (1, 3000, 1000, BF16, True, True, True, False, 0),
]


def norm_inputs(n, rows, hidden, dt, residual, g32, offset, seed=1):
    g, put = gen(seed), Guarded(offset)
    ins = [put.new((rows, hidden), dt, randn(g, rows, hidden)) for _ in range(n)]
    res = put.new((rows, hidden), dt, 3 * randn(g, rows, hidden)) if residual else None
    gamma = put.new((hidden,), F32 if g32 else dt, 1 + 0.3 * randn(g, hidden))
    return ins, res, gamma


@pytest.mark.parametrize("n,rows,hidden,dt,residual,out8,save8,g32,offset", NORM)
def test_norm(n, rows, hidden, dt, residual, out8, save8, g32, offset):
    ins, res, gamma = norm_inputs(n, rows, hidden, dt, residual, g32, offset)
    put, nb = Guarded(offset), ref.blocks(hidden)
    outs = [put.new((rows, hidden), E4M3 if out8 else dt) for _ in range(n)]
    sc = [put.new((rows, nb), F32) for _ in range(n)] if out8 else None
    ro, rs = put.new((rows, hidden), dt), put.new((rows,), F32)
    sv, svs = (put.new((rows, hidden), torch.uint8), put.new((rows, nb), F32)) if save8 else (None, None)
    ar.ar_allreduce_rmsnorm(ins, gamma, outs, res, ro, rs, sc, sv, svs, eps=1e-4)
    torch.cuda.synchronize()
    put.check()
    h, rstd, y, dh, rel, dy = ref.norm(ins, res, gamma, 1e-4)
    ref.close(ro, h, dh, "residual_out")
    ref.close(rs[:, None], rstd, rel * rstd, "rstd")
    for r in range(n):
        if out8:
            ref.close_codes(outs[r], sc[r], y, dy, f"out {r}")
        else:
            ref.close(outs[r], y, dy, f"out {r}")
        assert torch.equal(outs[r].view(torch.uint8), outs[0].view(torch.uint8))
    if save8:
        ref.close_codes(sv, svs, h, dh, "saved")


@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_norm_with_only_its_outputs(dt):
    """Every optional output left out gives the same y."""
    ins, res, gamma = norm_inputs(3, 6, 700, dt, True, False, 0)
    full, alone = [torch.empty_like(x) for x in ins], [torch.empty_like(x) for x in ins]
    ar.ar_allreduce_rmsnorm(ins, gamma, full, res, torch.empty_like(res), torch.empty(6, device=DEV))
    ar.ar_allreduce_rmsnorm(ins, gamma, alone, res)
    assert all(torch.equal(a, b) for a, b in zip(full, alone))


@pytest.mark.parametrize("dt", [BF16, F32])
def test_norm_in_place(dt):
    ins, res, gamma = norm_inputs(4, 50, 1111, dt, True, False, 0)
    outs, ro = [torch.empty_like(x) for x in ins], torch.empty_like(res)
    ar.ar_allreduce_rmsnorm(ins, gamma, outs, res, ro)
    ar.ar_allreduce_rmsnorm(ins, gamma, ins, res, res)
    assert all(torch.equal(a, b) for a, b in zip(ins, outs)) and torch.equal(res, ro)


def test_norm_sum_is_the_rank_order_all_reduce():
    """Without a residual, residual_out has the bits of AR_ALGO_FUSED."""
    for dt in (BF16, F16, F32):
        ins, _, gamma = norm_inputs(6, 20, 776, dt, False, False, 0)
        ro, want = torch.empty_like(ins[0]), [torch.empty_like(x) for x in ins]
        ar.ar_allreduce(ins, want, ar.AR_SUM, ar.AR_ALGO_FUSED)
        ar.ar_allreduce_rmsnorm(ins, gamma, [torch.empty_like(x) for x in ins], None, ro)
        assert torch.equal(ro, want[0])


@pytest.mark.parametrize("dt,code", [(F32, oracle.F32), (BF16, oracle.BF16)])
def test_norm_checkpoint_is_the_block_codec(dt, code):
    """One rank, no residual: h is the input, so the checkpoint has the codec's bits (zero blocks, huge and tiny
    values and NaN among them), a row's last block short."""
    rows, hidden = 12, 1000
    x = randn(gen(5), rows, hidden) * torch.logspace(-30, 30, rows, device=DEV)[:, None]
    x[3, 128:256] = 0.0
    x[4, 5] = float("nan")
    x[5, :] = 1e-44
    x = x.to(dt)
    sv, svs = torch.empty(rows, hidden, dtype=torch.uint8, device=DEV), torch.empty(rows, 8, device=DEV)
    ar.ar_allreduce_rmsnorm([x], torch.ones(hidden, dtype=dt, device=DEV), [torch.empty_like(x)], saved=sv,
                            saved_scales=svs)
    host = x.cpu().view(torch.int32 if dt == F32 else torch.int16).numpy().view(np.uint32 if dt == F32 else np.uint16)
    for r in range(rows):
        row = host[r].view(np.float32) if dt == F32 else host[r]
        codes, scales = oracle.fp8_quant(row, code)
        np.testing.assert_array_equal(sv[r].cpu().numpy(), codes)
        np.testing.assert_array_equal(svs[r].cpu().numpy().view(np.uint32), np.asarray(scales).view(np.uint32))


def test_norm_rows_of_zeros_infinities_and_nan():
    rows, hidden = 6, 384
    x = randn(gen(6), rows, hidden).to(BF16)
    x[0] = 0.0
    x[1, 7] = float("inf")
    x[2, 300] = float("nan")
    x[3] *= 1e-20
    gamma, out = torch.ones(hidden, dtype=BF16, device=DEV), torch.empty_like(x)
    rs = torch.empty(rows, device=DEV)
    codes, sc = torch.empty(rows, hidden, dtype=torch.uint8, device=DEV), torch.empty(rows, 3, device=DEV)
    ar.ar_allreduce_rmsnorm([x], gamma, [out], rstd=rs, eps=1e-5)
    assert bool((out[0] == 0).all()) and rs[0].item() == pytest.approx(1e-5 ** -0.5, rel=1e-6)
    # an infinity makes the row's rstd zero: 0 at finite elements, NaN at itself; NaN spreads over its row alone
    assert rs[1].item() == 0 and bool(torch.isnan(out[1, 7])) and int(torch.isnan(out[1]).sum()) == 1
    assert bool(torch.isnan(out[2]).all()) and not bool(torch.isnan(out[3:]).any())
    ar.ar_allreduce_rmsnorm([x], gamma, [codes], out_scales=[sc], eps=1e-5)
    assert bool((codes[0] == 0).all()) and bool((sc[0] == 1).all())
    assert codes[1, 7].item() == 0x7F and bool((codes[2] == 0x7F).all())
    ar.ar_allreduce_rmsnorm([x[:1]], gamma, [out[:1]], eps=0.0)  # 0 * inf
    assert bool(torch.isnan(out[0]).all())


BWD = [  # ranks, rows, hidden, dtype, residual grad, 8-bit saved, gamma fp32, offset
    (1, 1, 1, F32, False, False, False, 0),
    (1, 1, 1, BF16, True, True, False, 0),
    (8, 1, 4096, BF16, True, True, False, 0),
    (8, 40, 4096, BF16, True, False, False, 0),
    (2, 129, 1003, F16, True, False, True, 1),
    (3, 65, 2050, F32, False, True, False, 1),
    (4, 9, 127, BF16, True, True, True, 3),
    (16, 33, 520, F16, True, True, False, 5),
    (64, 3, 300, BF16, False, False, True, 0),
    (1, 2500, 640, BF16, True, True, False, 0),
    (1, 5000, 96, F32, True, False, False, 0),
    (2, 3, 16384, F16, True, True, False, 0),
    (1, 3, 32768, F32, True, True, False, 0),
    (2, 3, 32767, BF16, True, True, False, 1),
]


def bwd_inputs(n, rows, hidden, dt, rgrad, save8, g32, offset, seed=2):
    g, put = gen(seed), Guarded(offset)
    h = 3 * randn(g, rows, hidden)
    rstd = put.new((rows,), F32, (h.square().mean(1) + 1e-5).rsqrt())
    ins = [put.new((rows, hidden), dt, 0.1 * randn(g, rows, hidden)) for _ in range(n)]
    gamma = put.new((hidden,), F32 if g32 else dt, 1 + 0.3 * randn(g, hidden))
    rg = put.new((rows, hidden), dt, 0.2 * randn(g, rows, hidden)) if rgrad else None
    saved, scales = put.new((rows, hidden), dt, h), None
    if save8:
        saved, scales = put.new((rows, hidden), torch.uint8), put.new((rows, ref.blocks(hidden)), F32)
        ar.ar_allreduce_rmsnorm([h], torch.ones(hidden, device=DEV), [torch.empty_like(h)], saved=saved,
                                saved_scales=scales)
    return ins, saved, scales, gamma, rstd, rg


def saved_f64(saved, scales):
    if scales is None:
        return ref.f64(saved)
    return ref.codes_f64(saved) * ref.spread(ref.f64(scales), saved.shape[1])


@pytest.mark.parametrize("n,rows,hidden,dt,rgrad,save8,g32,offset", BWD)
def test_norm_bwd(n, rows, hidden, dt, rgrad, save8, g32, offset):
    ins, saved, scales, gamma, rstd, rg = bwd_inputs(n, rows, hidden, dt, rgrad, save8, g32, offset)
    put = Guarded(offset)
    outs, dgamma = [put.new((rows, hidden), dt) for _ in range(n)], put.new((hidden,), F32)
    ws = workspace(ar.ar_allreduce_rmsnorm_bwd_workspace_size(rows, hidden))
    ar.ar_allreduce_rmsnorm_bwd(ins, saved, gamma, rstd, outs, dgamma, scales, rg, ws)
    torch.cuda.synchronize()
    put.check()
    # a column's sum: at most as many additions behind one another as there are rows, and the joining of the parts
    dx, dg, ddx, ddg = ref.norm_bwd(ins, saved_f64(saved, scales), gamma, rstd, rg, min(rows, 64) + 128)
    for r in range(n):
        ref.close(outs[r], dx, ddx, f"dx {r}")
        assert torch.equal(outs[r], outs[0])
    ref.close(dgamma, dg, ddg, "dgamma")
    again, dg2 = [torch.empty_like(x) for x in ins], torch.empty(hidden, device=DEV)
    ar.ar_allreduce_rmsnorm_bwd(ins, saved, gamma, rstd, again, dg2, scales, rg, ws)
    assert torch.equal(dg2, dgamma) and torch.equal(again[0], outs[0]), "not the same twice"


def test_norm_bwd_in_place_and_empty():
    ins, saved, scales, gamma, rstd, rg = bwd_inputs(3, 40, 1111, BF16, True, False, False, 0)
    ws = workspace(ar.ar_allreduce_rmsnorm_bwd_workspace_size(40, 1111))
    outs, dg, dg2 = [torch.empty_like(x) for x in ins], torch.empty(1111, device=DEV), torch.empty(1111, device=DEV)
    ar.ar_allreduce_rmsnorm_bwd(ins, saved, gamma, rstd, outs, dg, scales, rg, ws)
    ar.ar_allreduce_rmsnorm_bwd(ins, saved, gamma, rstd, [ins[0], rg, ins[2]], dg2, scales, rg, ws)
    for t in (ins[0], rg, ins[2]):
        assert torch.equal(t, outs[0])
    assert torch.equal(dg, dg2)
    none = torch.empty(0, 1111, dtype=BF16, device=DEV)
    ar.ar_allreduce_rmsnorm_bwd([none], none, gamma, torch.empty(0, device=DEV), [none], dg, workspace=ws)
    assert bool((dg == 0).all())
    ar.ar_allreduce_rmsnorm([none], gamma, [none])


def test_norm_gradient_against_differences():
    """A directional difference of the fp32 forward kernel. With steps of 2^-6 of unit directions the quotient's
    truncation is of the order of 2^-12, and its rounding of 2^-24 * 2^6 = 2^-18, of the loss's terms."""
    rows, hidden = 16, 512
    g = gen(8)
    x, dy, v = randn(g, rows, hidden), randn(g, rows, hidden), randn(g, rows, hidden)
    gamma, w = 1 + 0.3 * randn(g, hidden), randn(g, hidden)

    def loss(x_, gamma_):
        y = torch.empty_like(x_)
        ar.ar_allreduce_rmsnorm([x_], gamma_, [y])
        return float((y.double() * dy.double()).sum())

    h, rs, dx, dg = torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty_like(x), torch.empty_like(gamma)
    ar.ar_allreduce_rmsnorm([x], gamma, [torch.empty_like(x)], None, h, rs)
    ar.ar_allreduce_rmsnorm_bwd([dy], h, gamma, rs, [dx], dg,
                                workspace=workspace(ar.ar_allreduce_rmsnorm_bwd_workspace_size(rows, hidden)))
    s = 2.0 ** -6
    size = float(dy.double().norm() * v.double().norm())
    assert abs((loss(x + s * v, gamma) - loss(x - s * v, gamma)) / (2 * s) - float((dx.double() * v.double()).sum())) \
        < 2.0 ** -10 * size
    size = float(dy.double().norm() * w.double().norm() * rows ** 0.5)
    assert abs((loss(x, gamma + s * w) - loss(x, gamma - s * w)) / (2 * s) - float((dg.double() * w.double()).sum())) \
        < 2.0 ** -10 * size


@pytest.mark.parametrize("dt,hidden", [(BF16, 8192), (BF16, 8191)])
def test_norm_past_32_bit_offsets(dt, hidden):
    """More than 2^31 elements in a buffer: the first and last rows against the reference."""
    rows = (1 << 31) // hidden + 40
    x = torch.empty(rows, hidden, dtype=dt, device=DEV)
    g = gen(9)
    pick = [0, 1, rows // 2, rows - 2, rows - 1]
    x.fill_(1.0)
    for r in pick:
        x[r] = randn(g, hidden)
    gamma = (1 + 0.3 * randn(g, hidden)).to(dt)
    out, rs = torch.empty_like(x), torch.empty(rows, device=DEV)
    ar.ar_allreduce_rmsnorm([x], gamma, [out], rstd=rs)
    _, _, y, _, _, dy = ref.norm([x[pick]], None, gamma, 1e-5)
    ref.close(out[pick], y, dy, "out")
    dg, ws = torch.empty(hidden, device=DEV), workspace(ar.ar_allreduce_rmsnorm_bwd_workspace_size(rows, hidden))
    ar.ar_allreduce_rmsnorm_bwd([out], x, gamma, rs, [out], dg, workspace=ws)
    ins = (y + 0).to(dt)
    dx, _, ddx, _ = ref.norm_bwd([ins], ref.f64(x[pick]), gamma, rs[pick], None, 1)
    # its input is the kernel's y, which may be one step of bf16 from the rounded reference
    ref.close(out[pick], dx, ddx + 2.0 ** -7 * (y.abs() * rs[pick].cpu().double()[:, None] * 4 + dx.abs()), "dx")


# ------------------------------------------------------------------------------------------------ experts
SORT = [  # tokens, k, experts, align, kind
    (0, 2, 4, 4, "even"), (1, 1, 1, 1, "even"), (1, 8, 1024, 16, "even"), (63, 3, 7, 1, "even"),
    (64, 1, 64, 8, "one"), (1000, 2, 5, 128, "none"), (1000, 8, 60, 16, "some"), (4096, 2, 8, 1, "even"),
    (4097, 2, 8, 1, "even"), (10_007, 3, 1000, 16, "some"), (30_000, 8, 256, 128, "skew"), (70_001, 1, 3, 7, "skew"),
    (200_000, 8, 64, 1, "skew"),
]


def make_ids(tokens, k, experts, kind, seed=3):
    g = gen(seed)
    ids = torch.randint(0, experts, (tokens, k), generator=g, device=DEV, dtype=torch.int32)
    if kind == "one":
        ids[:] = experts // 2
    elif kind == "none":
        ids = torch.where(ids % 2 == 0, ids - 100, ids + experts)
    elif kind == "some":  # experts elsewhere, and numbers that are no expert
        ids = torch.where(torch.rand(tokens, k, generator=g, device=DEV) < 0.3, -1, ids)
        ids = torch.where(torch.rand(tokens, k, generator=g, device=DEV) < 0.1, experts + ids, ids)
        ids[0, 0] = 2 ** 31 - 1
        ids[-1, -1] = -2 ** 31
    elif kind == "skew":
        ids = torch.where(torch.rand(tokens, k, generator=g, device=DEV) < 0.7, ids % 2, ids)
    return ids.to(torch.int32)


def run_sort(ids, experts, align, extra=0, put=None):
    put = put or Guarded()
    tokens, k = ids.shape
    i32 = torch.int32
    rows = ar.ar_expert_rows(tokens, k, experts, align) + extra
    off, cnt = put.new((experts + 1,), i32), put.new((experts,), i32)
    pos, src = put.new((tokens, k), i32), put.new((rows,), i32)
    ws = workspace(ar.ar_expert_sort_workspace_size(tokens, k, experts))
    ar.ar_expert_sort(ids, off, cnt, pos, src, align, ws)
    torch.cuda.synchronize()
    put.check()
    return off, cnt, pos, src


@pytest.mark.parametrize("tokens,k,experts,align,kind", SORT)
def test_expert_sort(tokens, k, experts, align, kind):
    ids = make_ids(tokens, k, experts, kind)
    off, cnt, pos, src = run_sort(ids, experts, align, extra=5)
    offsets, counts, p, s = ref.sort(ids.cpu(), experts, align)
    assert off.tolist() == offsets and cnt.tolist() == counts and pos.reshape(-1).tolist() == p
    want = np.full(src.numel(), -1, np.int32)
    if s:
        want[np.fromiter(s.keys(), int)] = np.fromiter(s.values(), np.int32)
    np.testing.assert_array_equal(src.cpu().numpy(), want)


MOVE = [  # tokens, k, experts, align, kind, hidden, dtype, offset
    (1, 1, 1, 1, "even", 1, BF16, 0), (1, 8, 128, 16, "even", 4096, BF16, 0), (37, 3, 6, 16, "some", 1003, F16, 1),
    (50, 2, 4, 1, "even", 64, F32, 0), (21, 9, 30, 8, "some", 130, BF16, 3), (19, 20, 40, 4, "some", 520, F32, 0),
    (200, 4, 16, 128, "skew", 1190, BF16, 0), (65, 2, 4, 4, "none", 256, F16, 0), (300, 2, 8, 1, "skew", 8, F16, 1),
    (70, 4, 8, 16, "some", 5000, F32, 1),
]


@pytest.mark.parametrize("rows8", [False, True])
@pytest.mark.parametrize("tokens,k,experts,align,kind,hidden,dt,offset", MOVE)
def test_dispatch(tokens, k, experts, align, kind, hidden, dt, offset, rows8):
    off, cnt, pos, src = run_sort(make_ids(tokens, k, experts, kind), experts, align)
    g, put = gen(4), Guarded(offset)
    rows, nb = src.numel(), ref.blocks(hidden)
    if rows8:
        dt = torch.uint8
        x = put.new((tokens, hidden), dt, torch.randint(0, 256, (tokens, hidden), generator=g, device=DEV))
        xsc, xssc = put.new((tokens, nb), F32, randn(g, tokens, nb)), put.new((rows, nb), F32)
    else:
        x, xsc, xssc = put.new((tokens, hidden), dt, randn(g, tokens, hidden)), None, None
    xs = put.new((rows, hidden), dt)
    xs.view(torch.uint8).fill_(0x33)
    ar.ar_expert_dispatch(x, pos, off, cnt, xs, xsc, xssc)
    torch.cuda.synchronize()
    put.check()
    end = off[-1].item()
    there = (src[:end] >= 0)[:, None]
    token = src[:end].clamp(min=0).long() // k
    assert torch.equal(xs[:end], torch.where(there, x[token], 0).to(dt))
    assert bool((xs[end:].contiguous().view(torch.uint8) == 0x33).all()), "rows behind the segments were written"
    if rows8:
        assert torch.equal(xssc[:end], torch.where(there, xsc[token], 0.0))


@pytest.mark.parametrize("weighted,added", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("tokens,k,experts,align,kind,hidden,dt,offset", MOVE)
def test_combine(tokens, k, experts, align, kind, hidden, dt, offset, weighted, added):
    off, cnt, pos, src = run_sort(make_ids(tokens, k, experts, kind), experts, align)
    g, put = gen(5), Guarded(offset)
    ys = put.new((src.numel(), hidden), dt, randn(g, src.numel(), hidden))
    ys[src < 0] = float("nan")  # rows that no slot has are not read
    w = put.new((tokens, k), F32, randn(g, tokens, k)) if weighted else None
    add = put.new((tokens, hidden), dt, randn(g, tokens, hidden)) if added else None
    out = put.new((tokens, hidden), dt)
    ar.ar_expert_combine(ys, pos, out, w, add)
    torch.cuda.synchronize()
    put.check()
    want, bound = ref.combine(ys, pos.cpu(), w, add)
    ref.close(out, want, bound, "out")
    if added:  # in place of the addend
        ar.ar_expert_combine(ys, pos, add, w, add)
        assert torch.equal(add, out)


@pytest.mark.parametrize("tokens,k,experts,align,kind,hidden,dt,offset", MOVE)
def test_combine_bwd(tokens, k, experts, align, kind, hidden, dt, offset):
    off, cnt, pos, src = run_sort(make_ids(tokens, k, experts, kind), experts, align)
    g, put, rows = gen(6), Guarded(offset), src.numel()
    ys = put.new((rows, hidden), dt, randn(g, rows, hidden))
    ys[src < 0] = float("nan")
    w = put.new((tokens, k), F32, randn(g, tokens, k))
    w[pos < 0] = float("nan")
    dout = put.new((tokens, hidden), dt, randn(g, tokens, hidden))
    dys, dw = put.new((rows, hidden), dt), put.new((tokens, k), F32)
    dys.view(torch.uint8).fill_(0x33)
    ar.ar_expert_combine_bwd(dout, ys, pos, w, off, cnt, dys, dw)
    torch.cuda.synchronize()
    put.check()
    want, dweights, bound = ref.combine_bwd(dout, ys, pos.cpu(), w, rows)
    end = off[-1].item()
    ref.close(dys[:end], want[:end], ref.U * want[:end].abs(), "dys")
    assert bool((dys[end:].contiguous().view(torch.uint8) == 0x33).all()), "rows behind the segments were written"
    ref.close(dw, dweights, bound, "dweights")
    dw2 = torch.empty_like(dw)
    ar.ar_expert_combine_bwd(dout, ys, pos, w, off, cnt, ys, dw2)  # in place of the experts' rows
    assert torch.equal(ys[:end], dys[:end]) and torch.equal(dw2, dw)


def test_positions_out_of_range_are_absent():
    """Positions that no sort makes are slots without a row, never addresses."""
    tokens, hidden, rows = 5, 200, 7
    pos = torch.tensor([[0, 7], [2 ** 31 - 1, 1], [-5, 2], [-2 ** 31, 3], [4, 1 << 20]], dtype=torch.int32, device=DEV)
    bad = (pos < 0) | (pos >= rows)
    g = gen(7)
    x, ys, w = randn(g, tokens, hidden), randn(g, rows, hidden), randn(g, tokens, 2)
    xs = torch.zeros(rows, hidden, device=DEV)
    ar.ar_expert_dispatch(x, pos, None, None, xs)
    assert torch.equal(xs[:5], x) and bool((xs[5:] == 0).all())
    out = torch.empty(tokens, hidden, device=DEV)
    ar.ar_expert_combine(ys, pos, out, w)
    fixed = torch.where(bad, -1, pos).cpu()
    want, bound = ref.combine(ys, fixed, w, None)
    ref.close(out, want, bound, "out")
    dys, dw = torch.zeros_like(ys), torch.empty_like(w)
    # segment tables that no sort makes only ever zero rows inside the buffer
    off = torch.tensor([6, 2 ** 31 - 1, -3], dtype=torch.int32, device=DEV)
    cnt = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    ar.ar_expert_combine_bwd(x, ys, pos, w, off, cnt, dys, dw)
    want, dwant, bound = ref.combine_bwd(x, ys, fixed, w, rows)
    ref.close(dys[:5], want[:5], ref.U * want[:5].abs(), "dys")
    ref.close(dw, dwant, bound, "dweights")


def test_rows_past_32_bit_offsets():
    """Sorted rows of more than 2^31 elements in all: tokens whose rows lie at the far end."""
    hidden, tokens, k = 8192, 150_000, 2
    ids = make_ids(tokens, k, 16, "even")
    off, cnt, pos, src = run_sort(ids, 16, 1)
    x = torch.randn(tokens, hidden, device=DEV, dtype=BF16)
    xs = torch.empty(src.numel(), hidden, device=DEV, dtype=BF16)
    ar.ar_expert_dispatch(x, pos, off, cnt, xs)
    for r in (0, 1, src.numel() // 2, src.numel() - 2, src.numel() - 1):
        assert torch.equal(xs[r], x[src[r].item() // k])
    out, dw = torch.empty_like(x), torch.empty(tokens, k, device=DEV)
    ar.ar_expert_combine(xs, pos, out)
    assert torch.equal(out, x + x)  # exact: twice the same value
    ar.ar_expert_combine_bwd(x, xs, pos, torch.ones(tokens, k, device=DEV), off, cnt, xs, dw)
    for r in (0, src.numel() - 1):
        assert torch.equal(xs[r], x[src[r].item() // k])


# ------------------------------------------------------------------------------------------------ streams, graphs
def test_side_stream_and_graph_replays():
    """All operators in one captured graph on a side stream, replayed on new inputs with eager work between."""
    n, rows, hidden, k, experts, align = 4, 96, 1536, 2, 8, 16
    ins, res, gamma = norm_inputs(n, rows, hidden, BF16, True, False, 0)
    i32, nb = torch.int32, ref.blocks(hidden)
    new = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device=DEV)
    outs, ro, rs = [new(rows, hidden) for _ in range(n)], new(rows, hidden), new(rows, dtype=F32)
    sv, svs = new(rows, hidden, dtype=torch.uint8), new(rows, nb, dtype=F32)
    dxs, dg = [new(rows, hidden) for _ in range(n)], new(hidden, dtype=F32)
    ws = workspace(ar.ar_allreduce_rmsnorm_bwd_workspace_size(rows, hidden))
    cap = ar.ar_expert_rows(rows, k, experts, align)
    ids = make_ids(rows, k, experts, "some")
    off, cnt, pos, src = (new(s, dtype=i32) for s in (experts + 1, experts, (rows, k), cap))
    w = torch.rand(rows, k, device=DEV)
    xs, out, dys, dw = torch.zeros(cap, hidden, dtype=BF16, device=DEV), new(rows, hidden), \
        torch.zeros(cap, hidden, dtype=BF16, device=DEV), new(rows, k, dtype=F32)

    def step():
        ar.ar_allreduce_rmsnorm(ins, gamma, outs, res, ro, rs, saved=sv, saved_scales=svs)
        ar.ar_expert_sort(ids, off, cnt, pos, src, align)
        ar.ar_expert_dispatch(outs[0], pos, off, cnt, xs)
        ar.ar_expert_combine(xs, pos, out, w, ro)
        ar.ar_expert_combine_bwd(out, xs, pos, w, off, cnt, dys, dw)
        ar.ar_allreduce_rmsnorm_bwd(dxs_in, sv, gamma, rs, dxs, dg, svs, out, ws)

    dxs_in = [torch.randn_like(x) for x in ins]
    results = lambda: [t.clone() for t in (*outs, ro, rs, sv, svs, off, cnt, pos, src, xs, out, dys, dw, *dxs, dg)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for k_ in range(3):
        g = gen(20 + k_)
        for x in (*ins, *dxs_in, res):
            x.copy_(randn(g, rows, hidden))
        ids.copy_(make_ids(rows, k, experts, "some", seed=30 + k_))
        xs.zero_()
        dys.zero_()
        step()
        torch.cuda.synchronize()
        want = results()
        xs.zero_()
        dys.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(results(), want):
            assert torch.equal(a.view(torch.uint8) if a.dtype == E4M3 else a, b), k_
