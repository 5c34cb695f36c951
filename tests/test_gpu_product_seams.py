"""The rows' gradient in its large tiles, where the second product's loads follow the first one's within the same pipelined
loop: sums of one step, of an odd and an even number, that end with a step or inside one, in every size of tile and way of
loading that 16-bit types have. Every call is made twice, into buffers that hold NaN and other numbers before, and has to
give the same bits.

Which tile a call takes on 256 compute units, of `rows` rows and `hidden` columns: 64 x 64 below 256 tiles of 128 x 128;
256 x 256 with 16-byte rows, 192 rows an expert and 192 tiles of that size."""
import pytest
import torch

import all_reduce_reduction_ring_amd as ar
import product_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
# a step is 64 elements of the sum: one; one cut; two; three; four, the last cut; five, the last cut; six
STEPS = [64, 40, 128, 136, 200, 264, 384]

CASES = [("256", hidden, inner) for hidden, inner in [(4096, i) for i in STEPS] + [(4104, 200)]]  # 16 x 16 and 17 large tiles
CASES += [("128", 2048, i) for i in STEPS]                                 # 17 x 16 tiles, 8 x 8 large ones
CASES += [("128 cut", 2050, i) for i in (34, 66, 130, 190, 258, 322)]      # rows of 4 bytes' multiples
CASES += [("128 registers", h, i) for h, i in ((2049, 64), (2049, 321), (2048, 65), (2048, 127), (2049, 130))]
COUNTS = {"256": [1999, 1, 0, 1100, 1095], "128": [1003, 0, 130, 1, 960]}


def make(kind, hidden, inner, dtype, seed):
    counts, dt = COUNTS["256" if kind == "256" else "128"], DT[dtype]
    g = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)
    starts, rows = ref.segments(counts, 1, 5)
    inside = torch.zeros(rows, 1, dtype=torch.bool, device=DEV)
    for lo, c in zip(starts, counts):
        inside[lo:lo + c] = True
    row = lambda w: torch.where(inside, randn(rows, w), torch.nan).to(dt)
    seg = dict(offsets=torch.tensor(starts, dtype=torch.int32, device=DEV), counts=torch.tensor(counts, dtype=torch.int32, device=DEV))
    spans = [(e, slice(lo, lo + c)) for e, (lo, c) in enumerate(zip(starts, counts)) if c]
    mat = lambda o, i: (randn(len(counts), o, i) / i ** 0.5).to(dt)
    new = lambda w, value: torch.full((rows, w), value, dtype=dt, device=DEV)
    return row, mat, new, seg, spans, ~inside[:, 0]


def same(a, b, spans=None):
    for x, y in zip(a, b):
        for r in [slice(None)] if spans is None else [s for _, s in spans]:
            assert torch.equal(x[r], y[r])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("kind,hidden,inner", CASES)
def test_two_products_in_one_sum(kind, hidden, inner, dtype):
    row, mat, new, seg, spans, outside = make(kind, hidden, inner, dtype, inner)
    dt, x, wg, wu = DT[dtype], row(hidden), mat(inner, hidden), mat(inner, hidden)
    dout, gate, up = row(inner), row(inner), row(inner)
    runs = []
    for before in (torch.nan, 3.0):
        rows_ = [new(inner, before), new(inner, before), new(hidden, before)]
        mats = [torch.full_like(wg, before), torch.full_like(wu, before)]
        ar.ar_expert_gated_bwd(dout, gate, up, x, wg, wu, rows_[0], rows_[1], dxs=rows_[2], dw_gate=mats[0], dw_up=mats[1], **seg)
        runs.append((rows_, mats))
    same(runs[0][0], runs[1][0], spans)
    same(runs[0][1], runs[1][1])
    (dgate, dup, dxs), (dwg, dwu) = runs[1]
    for t in runs[1][0]:
        assert bool((t[outside] == 3.0).all()), "rows outside the segments were written"
    for e, r in spans:
        both = torch.cat([dgate[r], dup[r]], 1), torch.cat([wg[e], wu[e]], 0)
        ref.close(dxs[r], *ref.rounded(ref.mm(*both), dt), f"dxs of expert {e}")
        for t, d, what in ((dwg, dgate, "dw_gate"), (dwu, dup, "dw_up")):
            ref.close(t[e], *ref.rounded(ref.mm(d[r].t(), x[r]), dt), f"{what} of expert {e}")
    assert not dwg[2 if kind == "256" else 1].any()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("kind,hidden,inner", CASES)
def test_one_product(kind, hidden, inner, dtype):
    """The single projection's gradient through the same tiles, on either side of what picks them."""
    row, mat, new, seg, spans, outside = make(kind, hidden, inner, dtype, 1000 + inner)
    dt, x, w, dy = DT[dtype], row(hidden), mat(inner, hidden), row(inner)
    runs = []
    for before in (torch.nan, 3.0):
        dxs, dw = new(hidden, before), torch.full_like(w, before)
        ar.ar_expert_linear_bwd(dy, x, w, dxs=dxs, dw=dw, **seg)
        runs.append((dxs, dw))
    same(runs[0][:1], runs[1][:1], spans)
    same(runs[0][1:], runs[1][1:])
    dxs, dw = runs[1]
    assert bool((dxs[outside] == 3.0).all()), "rows outside the segments were written"
    for e, r in spans:
        ref.close(dxs[r], *ref.rounded(ref.mm(dy[r], w[e]), dt), f"dxs of expert {e}")
        ref.close(dw[e], *ref.rounded(ref.mm(dy[r].t(), x[r]), dt), f"dw of expert {e}")
