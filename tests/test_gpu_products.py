"""The experts' products and their gradients against 64-bit references: every type, sizes that nothing divides, segments
that are empty, of one row, cut inside a tile, padded, with what must not be read set to NaN."""
import pytest
import torch

import all_reduce_reduction_ring_amd as ar
import product_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
KEEP = 7.0  # what rows that are not written hold

# hidden, inner, counts of the experts, align
SHAPES = [
    (64, 64, [1], 1),
    (1, 1, [3, 0, 1], 1),
    (17, 5, [2, 7, 0, 33], 1),
    (128, 256, [128, 0, 256, 1], 128),
    (130, 70, [129, 1, 0, 0, 64], 16),
    (264, 136, [5, 300, 2], 8),
    (1003, 77, [40], 1),
    (96, 384, [0, 0, 0], 4),
    (520, 200, [3] * 70 + [0, 9], 2),
]


def make(hidden, inner, counts, align, dtype, dense=False, spare=3, seed=0):
    g = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g)
    starts, rows = ref.segments(counts, align, 0 if dense else spare)
    inside = torch.zeros(rows, 1, dtype=torch.bool)
    for lo, c in zip(starts, counts):
        inside[lo:lo + c] = True
    row = lambda w, s=1.0: torch.where(inside, randn(rows, w) * s, torch.nan).to(DT[dtype]).to(DEV)
    n = len(counts)
    mat = lambda o, i: (randn(n, o, i) / i ** 0.5).to(DT[dtype]).to(DEV)
    seg = {} if dense else {"offsets": torch.tensor(starts, dtype=torch.int32, device=DEV),
                            "counts": torch.tensor(counts, dtype=torch.int32, device=DEV)}
    spans = [(e, slice(lo, lo + c)) for e, (lo, c) in enumerate(zip(starts, counts)) if c]
    new = lambda w: torch.full((rows, w), KEEP, dtype=DT[dtype], device=DEV)
    return {"rows": rows, "row": row, "mat": mat, "seg": seg, "spans": spans, "new": new, "inside": inside[:, 0].to(DEV)}


def untouched(c, *outs):
    for t in outs:
        assert (t[~c["inside"]] == KEEP).all(), "rows outside the segments were written"


def one(w, e):
    return w[e]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_gated(shape, dtype):
    hidden, inner, counts, align = SHAPES[shape]
    c = make(hidden, inner, counts, align, dtype, seed=shape)
    x, wg, wu = c["row"](hidden), c["mat"](inner, hidden), c["mat"](inner, hidden)
    for act in ref.ACTS:
        out, gate, up = (c["new"](inner) for _ in range(3))
        ar.ar_expert_gated(x, wg, wu, out, gate=gate, up=up, act=act, **c["seg"])
        alone = c["new"](inner)
        ar.ar_expert_gated(x, wg, wu, alone, act=act, **c["seg"])
        untouched(c, out, gate, up, alone)
        assert torch.equal(out, alone)
        for e, rows in c["spans"]:
            want = ref.gated(x[rows], wg[e], wu[e], act, DT[dtype])
            for t, (v, tol), what in zip((out, gate, up), want, ("out", "gate", "up")):
                ref.close(t[rows], v, tol, f"{what} of expert {e}, act {act}")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_gated_bwd(shape, dtype):
    hidden, inner, counts, align = SHAPES[shape]
    c, dt = make(hidden, inner, counts, align, dtype, seed=100 + shape), DT[dtype]
    x, wg, wu = c["row"](hidden), c["mat"](inner, hidden), c["mat"](inner, hidden)
    dout, gate, up = c["row"](inner), c["row"](inner, 2.0), c["row"](inner)
    for act in ref.ACTS:
        dgate, dup, dxs = c["new"](inner), c["new"](inner), c["new"](hidden)
        dwg, dwu = torch.full_like(wg, torch.nan), torch.full_like(wu, torch.nan)
        ar.ar_expert_gated_bwd(dout, gate, up, x, wg, wu, dgate, dup, dxs=dxs, dw_gate=dwg, dw_up=dwu, act=act, **c["seg"])
        untouched(c, dgate, dup, dxs)
        empty = set(range(len(counts)))
        for e, rows in c["spans"]:
            empty.discard(e)
            for t, (v, tol), what in zip((dgate, dup), ref.slopes(dout[rows], gate[rows], up[rows], act, dt), ("dgate", "dup")):
                ref.close(t[rows], v, tol, f"{what} of expert {e}, act {act}")
            both = torch.cat([dgate[rows], dup[rows]], 1), torch.cat([wg[e], wu[e]], 0)
            ref.close(dxs[rows], *ref.rounded(ref.mm(*both), dt), f"dxs of expert {e}")
            for t, d, what in ((dwg, dgate, "dw_gate"), (dwu, dup, "dw_up")):
                ref.close(t[e], *ref.rounded(ref.mm(d[rows].t(), x[rows]), dt), f"{what} of expert {e}")
        for e in empty:
            assert (dwg[e] == 0).all() and (dwu[e] == 0).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_linear_and_its_gradient(shape, dtype):
    inside, out, counts, align = SHAPES[shape]
    c, dt = make(inside, out, counts, align, dtype, seed=200 + shape), DT[dtype]
    x, w, dy = c["row"](inside), c["mat"](out, inside), c["row"](out)
    y, dxs, dw = c["new"](out), c["new"](inside), torch.full_like(w, torch.nan)
    ar.ar_expert_linear(x, w, y, **c["seg"])
    ar.ar_expert_linear_bwd(dy, x, w, dxs=dxs, dw=dw, **c["seg"])
    untouched(c, y, dxs)
    for e, rows in c["spans"]:
        ref.close(y[rows], *ref.rounded(ref.mm(x[rows], w[e].t()), dt), f"ys of expert {e}")
        ref.close(dxs[rows], *ref.rounded(ref.mm(dy[rows], w[e]), dt), f"dxs of expert {e}")
        ref.close(dw[e], *ref.rounded(ref.mm(dy[rows].t(), x[rows]), dt), f"dw of expert {e}")
    for e, n in enumerate(counts):
        assert n or (dw[e] == 0).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,hidden,inner", [(1, 128, 128), (5, 77, 300), (257, 256, 192)])
def test_dense(rows, hidden, inner, dtype):
    """One matrix for all rows, without tables."""
    c, dt = make(hidden, inner, [rows], 1, dtype, dense=True, seed=3), DT[dtype]
    x, wg, wu, dy = c["row"](hidden), c["mat"](inner, hidden)[0], c["mat"](inner, hidden)[0], c["row"](inner)
    out, y, gate, up = (c["new"](inner) for _ in range(4))
    ar.ar_expert_gated(x, wg, wu, out, gate=gate, up=up)
    ar.ar_expert_linear(x, wg, y)
    ref.close(out, *ref.gated(x, wg, wu, ar.AR_ACT_SILU, dt)[0], "out")
    ref.close(y, *ref.rounded(ref.mm(x, wg.t()), dt), "ys")
    dgate, dup, dxs, dw, dw_up = c["new"](inner), c["new"](inner), c["new"](hidden), torch.empty_like(wg), torch.empty_like(wu)
    ar.ar_expert_gated_bwd(dy, gate, up, x, wg, wu, dgate, dup, dxs=dxs, dw_gate=dw, dw_up=dw_up)
    ref.close(dw_up, *ref.rounded(ref.mm(dup.t(), x), dt), "dw_up")
    ref.close(dxs, *ref.rounded(ref.mm(torch.cat([dgate, dup], 1), torch.cat([wg, wu], 0)), dt), "dxs")
    ar.ar_expert_linear_bwd(dy, x, wg, dxs=dxs, dw=dw)
    ref.close(dw, *ref.rounded(ref.mm(dy.t(), x), dt), "dw")


@pytest.mark.parametrize("dtype", DT)
def test_halves_of_one_weight(dtype):
    """w_gate and w_up as the halves of one tensor, their gradients too; counts left out; gradients in place."""
    hidden, inner, counts = 192, 96, [5, 0, 130, 64]
    c, dt = make(hidden, inner, counts, 1, dtype, seed=4), DT[dtype]
    x, w, dout = c["row"](hidden), c["mat"](2 * inner, hidden), c["row"](inner)
    wg, wu = w[:, :inner], w[:, inner:]
    out, gate, up, dxs = c["new"](inner), c["new"](inner), c["new"](inner), c["new"](hidden)
    seg = {"offsets": c["seg"]["offsets"]}
    ar.ar_expert_gated(x, wg, wu, out, gate=gate, up=up, **seg)
    dw = torch.full_like(w, torch.nan)
    first = c["new"](inner), c["new"](inner)
    args = dict(dxs=dxs, dw_gate=dw[:, :inner], dw_up=dw[:, inner:], **seg)
    ar.ar_expert_gated_bwd(dout, gate, up, x, wg, wu, *first, **args)
    kept, dw_kept = dxs.clone(), dw.clone()
    again = gate.clone(), up.clone()
    ar.ar_expert_gated_bwd(dout, *again, x, wg, wu, *again, **args)
    for a, b in zip((*again, dxs, dw), (*first, kept, dw_kept)):
        assert torch.equal(a[c["inside"]] if a.dim() == 2 else a, b[c["inside"]] if b.dim() == 2 else b)
    for e, rows in c["spans"]:
        ref.close(out[rows], *ref.gated(x[rows], wg[e], wu[e], ar.AR_ACT_SILU, dt)[0], "out")
        ref.close(dw[e], *ref.rounded(ref.mm(torch.cat([first[0][rows], first[1][rows]], 1).t(), x[rows]), dt), "dw")


def test_tables_that_leave_the_rows():
    """Segments that run past the buffers are cut, ones that start outside have no rows; nothing else is written."""
    x, w = torch.randn(40, 64, device=DEV).bfloat16(), torch.randn(4, 32, 64, device=DEV).bfloat16()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    out = torch.full((40, 32), KEEP, dtype=torch.bfloat16, device=DEV)
    ar.ar_expert_linear(x, w, out, offsets=i32(-5, 10, 30, 90, 100), counts=i32(9, 4, 2 ** 31 - 1, 8))
    for e, rows in ((1, slice(10, 14)), (2, slice(30, 40))):
        ref.close(out[rows], *ref.rounded(ref.mm(x[rows], w[e].t()), torch.bfloat16), f"expert {e}")
    assert (out[:10] == KEEP).all() and (out[14:30] == KEEP).all()
    ar.ar_expert_linear(x, w, out, offsets=i32(0, 2 ** 31 - 1, -2 ** 31, 7, 3), counts=i32(0, 1, 1, -4))
    assert (out[:10] == KEEP).all()


@pytest.mark.parametrize("dtype", DT)
def test_gradient_against_differences(dtype):
    """The block's gradient along a direction against central differences of its 64-bit definition."""
    hidden, inner, counts = 96, 40, [7, 0, 30]
    c, dt = make(hidden, inner, counts, 1, dtype, seed=5, spare=0), DT[dtype]
    x, wg, wu, dout = c["row"](hidden), c["mat"](inner, hidden), c["mat"](inner, hidden), c["row"](inner)
    gen = torch.Generator(device=DEV).manual_seed(6)
    vx, vg, vu = (torch.randn(t.shape, generator=gen, device=DEV, dtype=ref.F64) for t in (x, wg, wu))
    for act in ref.ACTS:
        out, gate, up = (c["new"](inner) for _ in range(3))
        ar.ar_expert_gated(x, wg, wu, out, gate=gate, up=up, act=act, **c["seg"])
        dgate, dup, dxs, dwg, dwu = c["new"](inner), c["new"](inner), c["new"](hidden), torch.empty_like(wg), torch.empty_like(wu)
        ar.ar_expert_gated_bwd(dout, gate, up, x, wg, wu, dgate, dup, dxs=dxs, dw_gate=dwg, dw_up=dwu, act=act, **c["seg"])
        got = sum((g.to(ref.F64) * v).sum() for g, v in ((dxs, vx), (dwg, vg), (dwu, vu)))

        def loss(h):
            total = 0.0
            for e, rows in c["spans"]:
                xs, a, b = x[rows].to(ref.F64) + h * vx[rows], wg[e].to(ref.F64) + h * vg[e], wu[e].to(ref.F64) + h * vu[e]
                total = total + (dout[rows].to(ref.F64) * ref.act(xs @ a.t(), act) * (xs @ b.t())).sum()
            return total
        want = (loss(1e-5) - loss(-1e-5)) / 2e-5
        # gate and up are rounded (half a step each) before they enter dgate and dup, these once, the gradients once: four
        # half steps of every product's magnitude, with |act''| and |act'| below 1.13, and a step for the sums
        size = 0.0
        for e, rows in c["spans"]:
            d, g, u, xr = (t[rows].to(ref.F64).abs() for t in (dout, gate, up, x))
            mg = d * u * (1.13 + 1.13 * g) + d * 1.13 * u
            mu = d * (1.13 * g + 1.13 * g)
            size = size + ((mg @ wg[e].to(ref.F64).abs() + mu @ wu[e].to(ref.F64).abs()) * vx[rows].abs()).sum()
            size = size + ((mg.t() @ xr) * vg[e].abs()).sum() + ((mu.t() @ xr) * vu[e].abs()).sum()
        assert abs(got - want) <= size * 4 * torch.finfo(dt).eps / 2 + abs(want) * 1e-6, (act, got, want)


@pytest.mark.parametrize("dtype", DT)
def test_extremes_stay_in_their_rows(dtype):
    """A row of infinities or NaN changes its own row only; a NaN weight its own column; far-out gates keep to the limits."""
    c = make(128, 64, [3, 4], 1, dtype, seed=7)
    x, w = c["row"](128), c["mat"](64, 128)
    y = c["new"](64)
    ar.ar_expert_linear(x, w, y, **c["seg"])
    x2, w2, y2 = x.clone(), w.clone(), c["new"](64)
    x2[1], x2[5, 3], w2[1, 9, 100] = torch.inf, torch.nan, torch.nan
    ar.ar_expert_linear(x2, w2, y2, **c["seg"])
    assert y2[5].isnan().all() and not y2[1].isfinite().any() and y2[3:7, 9].isnan().all()
    same = torch.ones_like(y, dtype=torch.bool)
    same[[1, 5]] = False
    same[3:7, 9] = False
    assert torch.equal(y[same & c["inside"][:, None]], y2[same & c["inside"][:, None]])
    big = torch.tensor([1e4, -1e4, 300.0, -300.0, 0.0, -0.0, 60.0, -60.0], dtype=DT[dtype], device=DEV)
    gate, one_ = big[None].repeat(2, 1).contiguous(), torch.ones(2, 8, dtype=DT[dtype], device=DEV)
    for act in ref.ACTS:
        dgate, dup = torch.empty_like(one_), torch.empty_like(one_)
        ar.ar_expert_gated_bwd(one_, gate, one_.clone(), None, None, None, dgate, dup, act=act)
        # next to the limits, x or 0 and 1 or 0: silu, the slowest, is off by 60 exp(-60) = 5.3e-25 at -60
        assert ((dup[0] - torch.relu(big)).abs() <= 1e-24).all()
        assert ((dgate[0, [0, 1, 2, 3, 6, 7]].float().cpu() - torch.tensor([1.0, 0, 1, 0, 1, 0])).abs() <= 1e-24).all()
        assert (dgate[0, 4:6] == 0.5).all()


def test_small_numbers_are_kept():
    """f16 subnormals are operands like any other."""
    tiny = torch.full((2, 64), 2.0 ** -20, dtype=torch.float16, device=DEV)
    w, y = torch.full((16, 64), 16.0, dtype=torch.float16, device=DEV), torch.empty(2, 16, dtype=torch.float16, device=DEV)
    ar.ar_expert_linear(tiny, w, y)
    assert (y == 2.0 ** -10).all()


# widths at which an operand's rows are multiples of 16 bytes, of 4, and of neither, on either side of a step's and a tile's
# end; lengths of the sum over one, two and several steps
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("hidden,inner", [(64, 66), (66, 64), (126, 130), (62, 58), (190, 258), (258, 190), (129, 127), (322, 34),
                                          (2, 200), (200, 2), (4, 6)])
def test_widths_around_a_step(hidden, inner, dtype):
    counts = [130, 0, 1, 17, 65]
    c, dt = make(hidden, inner, counts, 1, dtype, seed=11), DT[dtype]
    x, wg, wu, dy = c["row"](hidden), c["mat"](inner, hidden), c["mat"](inner, hidden), c["row"](inner)
    out, gate, up, dgate, dup = (c["new"](inner) for _ in range(5))
    dxs, dwg, dwu, dx1 = c["new"](hidden), torch.empty_like(wg), torch.empty_like(wu), c["new"](hidden)
    ar.ar_expert_gated(x, wg, wu, out, gate=gate, up=up, **c["seg"])
    ar.ar_expert_gated_bwd(dy, gate, up, x, wg, wu, dgate, dup, dxs=dxs, dw_gate=dwg, dw_up=dwu, **c["seg"])
    ar.ar_expert_linear_bwd(dy, x, wg, dxs=dx1, **c["seg"])
    untouched(c, out, gate, up, dgate, dup, dxs, dx1)
    for e, rows in c["spans"]:
        ref.close(out[rows], *ref.gated(x[rows], wg[e], wu[e], ar.AR_ACT_SILU, dt)[0], "out")
        both = torch.cat([dgate[rows], dup[rows]], 1), torch.cat([wg[e], wu[e]], 0)
        ref.close(dxs[rows], *ref.rounded(ref.mm(*both), dt), "dxs")
        ref.close(dx1[rows], *ref.rounded(ref.mm(dy[rows], wg[e]), dt), "dxs of one projection")
        ref.close(dwu[e], *ref.rounded(ref.mm(dup[rows].t(), x[rows]), dt), "dw_up")


@pytest.mark.parametrize("rows,hidden,inner", [(128, 2046, 2050), (300, 2050, 2046), (20, 1022, 6)])
def test_matrices_at_the_end_of_their_memory(rows, hidden, inner):
    """Weights that end a few bytes before a 2 MiB boundary, rows that are no multiples of 16 bytes, narrow matrices: no load
    runs past them."""
    c, dt = make(hidden, inner, [rows], 1, "bf16", dense=True, seed=12), torch.bfloat16
    x, wg, wu, dy = c["row"](hidden), c["mat"](inner, hidden)[0], c["mat"](inner, hidden)[0], c["row"](inner)
    out, gate, up, dgate, dup = (c["new"](inner) for _ in range(5))
    dxs, dwg, dwu = c["new"](hidden), torch.empty_like(wg), torch.empty_like(wu)
    ar.ar_expert_gated(x, wg, wu, out, gate=gate, up=up)
    ar.ar_expert_gated_bwd(dy, gate, up, x, wg, wu, dgate, dup, dxs=dxs, dw_gate=dwg, dw_up=dwu)
    ref.close(out, *ref.gated(x, wg, wu, ar.AR_ACT_SILU, dt)[0], "out")
    ref.close(dxs, *ref.rounded(ref.mm(torch.cat([dgate, dup], 1), torch.cat([wg, wu], 0)), dt), "dxs")
    ref.close(dwg, *ref.rounded(ref.mm(dgate.t(), x), dt), "dw_gate")


@pytest.mark.parametrize("dtype", DT)
def test_few_rows_that_meet_at_few_experts(dtype):
    """Few rows on average, nearly all of them at a few of the experts: 16 rows at a time, the last ones not full."""
    hidden, inner, counts = 200, 72, [0] * 90
    counts[3], counts[40], counts[89] = 117, 16, 17
    c = make(hidden, inner, counts, 1, dtype, seed=11)
    x, wg, wu = c["row"](hidden), c["mat"](inner, hidden), c["mat"](inner, hidden)
    out, gate, up, y = (c["new"](inner) for _ in range(4))
    ar.ar_expert_gated(x, wg, wu, out, gate=gate, up=up, **c["seg"])
    ar.ar_expert_linear(x, wg, y, **c["seg"])
    untouched(c, out, gate, up, y)
    for e, rows in c["spans"]:
        want = ref.gated(x[rows], wg[e], wu[e], ar.AR_ACT_SILU, DT[dtype])
        for t, (v, tol), what in zip((out, gate, up), want, ("out", "gate", "up")):
            ref.close(t[rows], v, tol, f"{what} of expert {e}")
        ref.close(y[rows], *ref.rounded(ref.mm(x[rows], wg[e].t()), DT[dtype]), f"linear of expert {e}")
