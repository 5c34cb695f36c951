"""The experts' products as a program uses them: on other streams, in graphs, behind the sort and before the combine, far
into large buffers, with many experts, and one after the other in place."""
import pytest
import torch

import all_reduce_reduction_ring_amd as ar
import product_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def _layer(tokens, k, experts, hidden, inner, align, dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)
    new = lambda *s, dt=dtype: torch.zeros(*s, dtype=dt, device=DEV)
    i32, rows = torch.int32, ar.ar_expert_rows(tokens, k, experts, align)
    d = dict(x=randn(tokens, hidden).to(dtype), wg=(randn(experts, inner, hidden) / hidden ** 0.5).to(dtype),
             wu=(randn(experts, inner, hidden) / hidden ** 0.5).to(dtype), wd=(randn(experts, hidden, inner) / inner ** 0.5).to(dtype),
             dout=randn(tokens, hidden).to(dtype), weights=torch.rand(tokens, k, generator=g, device=DEV),
             ids=torch.randint(-1, experts, (tokens, k), generator=g, device=DEV, dtype=i32),
             offsets=new(experts + 1, dt=i32), counts=new(experts, dt=i32), pos=new(tokens, k, dt=i32), src=new(rows, dt=i32),
             ws=new(max(1, ar.ar_expert_sort_workspace_size(tokens, k, experts)), dt=torch.uint8), align=align)
    for name, w in dict(xs=hidden, gate=inner, up=inner, h=inner, ys=hidden, dys=hidden, dh=inner, dgate=inner, dup=inner, dxs=hidden).items():
        d[name] = new(rows, w)
    for name in ("wg", "wu", "wd"):
        d["d" + name] = torch.full_like(d[name], torch.nan)
    d["out"], d["dx"], d["dweights"] = new(tokens, hidden), new(tokens, hidden), new(tokens, k, dt=torch.float32)
    grads = [d["dwg"], d["dwu"], d["dwd"]]
    d["plan"], d["norm"] = ar.ar_grad_plan(grads), new(1, dt=torch.float32)
    d["norm_ws"] = new(ar.ar_grad_norm_workspace_size(d["plan"].shape[0]), dt=torch.uint8)
    return d


def _run(d, max_norm=None):
    """Forward and backward of an expert layer, and its gradients clipped."""
    seg = dict(offsets=d["offsets"], counts=d["counts"])
    ar.ar_expert_sort(d["ids"], d["offsets"], d["counts"], d["pos"], d["src"], align=d["align"], workspace=d["ws"])
    ar.ar_expert_dispatch(d["x"], d["pos"], d["offsets"], d["counts"], d["xs"])
    ar.ar_expert_gated(d["xs"], d["wg"], d["wu"], d["h"], gate=d["gate"], up=d["up"], **seg)
    ar.ar_expert_linear(d["h"], d["wd"], d["ys"], **seg)
    ar.ar_expert_combine(d["ys"], d["pos"], d["out"], weights=d["weights"])
    ar.ar_expert_combine_bwd(d["dout"], d["ys"], d["pos"], d["weights"], d["offsets"], d["counts"], d["dys"], d["dweights"])
    ar.ar_expert_linear_bwd(d["dys"], d["h"], d["wd"], dxs=d["dh"], dw=d["dwd"], **seg)
    ar.ar_expert_gated_bwd(d["dh"], d["gate"], d["up"], d["xs"], d["wg"], d["wu"], d["dgate"], d["dup"], dxs=d["dxs"], dw_gate=d["dwg"],
                           dw_up=d["dwu"], **seg)
    ar.ar_expert_combine(d["dxs"], d["pos"], d["dx"])
    if max_norm is not None:
        ar.ar_grad_clip(d["plan"], max_norm, d["norm"], workspace=d["norm_ws"])


RESULTS = ("out", "dx", "dweights", "dwg", "dwu", "dwd", "norm")


@pytest.mark.parametrize("tokens,k,experts,hidden,inner,align", [(50, 3, 7, 96, 64, 1), (33, 2, 5, 70, 51, 16), (1, 4, 16, 256, 128, 8)])
def test_layer_against_autograd(tokens, k, experts, hidden, inner, align):
    """fp32, so the roundings are fp32's: sums of at most `terms` products, passed through five operators."""
    d = _layer(tokens, k, experts, hidden, inner, align, torch.float32)
    _run(d)
    req = lambda t: t.double().clone().requires_grad_(True)
    x, wg, wu, wd, weights = (req(d[n]) for n in ("x", "wg", "wu", "wd", "weights"))
    want = torch.zeros(tokens, hidden, dtype=torch.float64, device=DEV)
    rows = []
    for t in range(tokens):
        for j in range(k):
            e = int(d["ids"][t, j])
            if e >= 0:
                y = (ref.act(wg[e] @ x[t], ar.AR_ACT_SILU) * (wu[e] @ x[t])) @ wd[e].t()
                rows.append((t, weights[t, j] * y))
    want = want.index_add(0, torch.tensor([t for t, _ in rows], device=DEV), torch.stack([r for _, r in rows]))
    want.backward(d["dout"].double())
    terms = max(hidden, inner, tokens * k)
    for name, w in (("out", want.detach()), ("dx", x.grad), ("dweights", weights.grad), ("dwg", wg.grad), ("dwu", wu.grad), ("dwd", wd.grad)):
        # 2 K 2^-24 for the sums of each of five operators, of results that are sums of independent terms
        assert (d[name].double() - w).norm() <= 5 * 2 * terms * 2.0 ** -24 * w.norm() + 1e-12, name


def test_streams_and_graphs():
    """On a side stream and replayed from a graph, with other inputs in the same place, as eagerly."""
    d = _layer(120, 4, 16, 256, 192, 16, BF, seed=1)
    _run(d, 0.5)
    first = {n: d[n].clone() for n in RESULTS}
    side = torch.cuda.Stream()
    for n in RESULTS:
        d[n].fill_(3.0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _run(d, 0.5)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(d[n], first[n]) for n in RESULTS)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(d, 0.5)
    other = _layer(120, 4, 16, 256, 192, 16, BF, seed=2)
    keep = {n: d[n].clone() for n in ("x", "ids", "dout")}
    for i in range(5):
        if i in (2, 3):
            for n in keep:
                d[n].copy_(other[n] if i == 2 else keep[n])
        _run(d, 0.5)
        torch.cuda.synchronize()
        want = {n: d[n].clone() for n in RESULTS}
        for n in RESULTS:
            d[n].fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        for n in RESULTS:
            assert torch.equal(d[n], want[n]), (n, i)
        assert i != 4 or all(torch.equal(d[n], first[n]) for n in RESULTS)


def test_two_streams_at_once():
    """Calls that share their inputs run at the same time on two streams: they have nothing else in common."""
    x, w = torch.randn(700, 512, device=DEV).to(BF), torch.randn(4, 384, 512, device=DEV).to(BF)
    off = torch.tensor([0, 100, 300, 301, 700], dtype=torch.int32, device=DEV)
    want = torch.empty(700, 384, dtype=BF, device=DEV)
    ar.ar_expert_linear(x, w, want, offsets=off)
    outs, streams = [torch.empty_like(want) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(8):
        for o, s in zip(outs, streams):
            ar.ar_expert_linear(x, w, o, offsets=off, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("width,dt", [(2048, BF), (2050, BF), (2049, BF), (1024, torch.float32)])
def test_rows_past_32_bits(width, dt):
    """Segments that lie more than 2^32 bytes, and 2^31 elements, into the rows."""
    rows = (2 ** 31 // width + 300) if dt is BF else (2 ** 30 // width + 300)
    x, y = torch.empty(rows, width, dtype=dt, device=DEV), torch.empty(rows, width, dtype=dt, device=DEV)
    at = [rows - 250, rows - 100, rows]
    off, cnt = torch.tensor(at, dtype=torch.int32, device=DEV), torch.tensor([150, 9], dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(0)
    x[at[0]:] = torch.randn(250, width, generator=g, device=DEV).to(dt)
    y[at[0]:] = 5.0
    wg, wu = ((torch.randn(2, width, width, generator=g, device=DEV) / width ** 0.5).to(dt) for _ in range(2))
    ar.ar_expert_gated(x, wg, wu, y, offsets=off, counts=cnt)
    spans = [(0, slice(at[0], at[0] + 150)), (1, slice(at[1], at[1] + 9))]
    for e, r in spans:
        ref.close(y[r], *ref.gated(x[r], wg[e], wu[e], ar.AR_ACT_SILU, dt)[0], "out")
    assert (y[at[1] + 9:] == 5).all()
    dw = torch.empty_like(wg)
    ar.ar_expert_linear_bwd(y, x, None, dw=dw, offsets=off, counts=cnt)
    for e, r in spans:
        ref.close(dw[e], *ref.rounded(ref.mm(y[r].t(), x[r]), dt), "dw")
    keep = y[at[0]:].clone()
    ar.ar_expert_linear_bwd(x, None, wg, dxs=y, offsets=off, counts=cnt)
    for e, r in spans:
        ref.close(y[r], *ref.rounded(ref.mm(x[r], wg[e]), dt), "dxs")
    assert torch.equal(y[at[1] + 9:], keep[at[1] + 9 - at[0]:])


def test_weights_past_32_bits():
    """The last of many experts' matrices lies more than 2^32 bytes behind the first one."""
    experts, n = 520, 2048
    w = torch.empty(experts, n, n, dtype=BF, device=DEV)
    w[-1] = torch.randn(n, n, device=DEV) / n ** 0.5
    x = torch.randn(40, n, device=DEV).to(BF)
    off = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
    off[-1] = 40
    y = torch.empty(40, n, dtype=BF, device=DEV)
    ar.ar_expert_linear(x, w, y, offsets=off)
    ref.close(y, *ref.rounded(ref.mm(x, w[-1].t()), BF), "ys")
    dxs, dw = torch.empty_like(x), torch.empty_like(w)
    ar.ar_expert_linear_bwd(y, x, w, dxs=dxs, dw=dw, offsets=off)
    ref.close(dxs, *ref.rounded(ref.mm(y, w[-1]), BF), "dxs")
    ref.close(dw[-1], *ref.rounded(ref.mm(y.t(), x), BF), "dw")
    assert not dw[:-1].any()


@pytest.mark.parametrize("experts", [63, 64, 65, 1000, ar.AR_MAX_EXPERTS])
def test_many_experts(experts):
    """Tables longer than a wave, with rows for the first, the last and some between."""
    g = torch.Generator().manual_seed(experts)
    counts = torch.where(torch.rand(experts, generator=g) < 0.2, torch.randint(1, 40, (experts,), generator=g), 0)
    counts[0], counts[-1] = 3, 200
    off = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32)
    x, w = torch.randn(int(off[-1]), 64, device=DEV).to(BF), torch.randn(experts, 48, 64, device=DEV).to(BF)
    y, dw, dxs = torch.empty(x.shape[0], 48, dtype=BF, device=DEV), torch.empty_like(w), torch.empty_like(x)
    gated, act = torch.empty_like(y), ar.AR_ACT_GELU
    seg = dict(offsets=off.to(DEV), counts=counts.to(torch.int32).to(DEV))
    ar.ar_expert_linear(x, w, y, **seg)
    ar.ar_expert_gated(x, w, w.clone(), gated, act=act, **seg)
    ar.ar_expert_linear_bwd(y, x, w, dxs=dxs, dw=dw, **seg)
    for e in counts.nonzero()[:, 0].tolist():
        r = slice(int(off[e]), int(off[e + 1]))
        ref.close(y[r], *ref.rounded(ref.mm(x[r], w[e].t()), BF), "ys")
        ref.close(gated[r], *ref.gated(x[r], w[e], w[e], act, BF)[0], "out")
        ref.close(dxs[r], *ref.rounded(ref.mm(y[r], w[e]), BF), "dxs")
        ref.close(dw[e], *ref.rounded(ref.mm(y[r].t(), x[r]), BF), "dw")
    assert not dw[(counts == 0).to(DEV)].any()


# both sides of every rule that picks a kernel: few rows or tiles, tiles of 64, 128 and 256, whole and cut chunks
@pytest.mark.parametrize("dt", [BF, torch.float32])
@pytest.mark.parametrize("experts,per,inside,out", [(4, 8, 512, 512), (4, 9, 512, 512), (0, 16, 1024, 640), (0, 17, 1024, 640),
                                                    (16, 40, 264, 2048), (16, 200, 264, 4224), (3, 700, 512, 8448), (2, 500, 510, 8448),
                                                    (8, 256, 320, 2048), (40, 3, 256, 1408)])
def test_both_sides_of_the_kernels_rules(experts, per, inside, out, dt):
    rows, n = per * max(experts, 1), max(experts, 1)
    g = torch.Generator(device=DEV).manual_seed(rows)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x, y = randn(rows, inside).to(dt), torch.empty(rows, out, dtype=dt, device=DEV)
    w, wu = ((randn(n, out, inside) / inside ** 0.5).to(dt) for _ in range(2))
    seg = dict(offsets=torch.arange(n + 1, dtype=torch.int32, device=DEV) * per) if experts else {}
    dy, h, dxs, dw = randn(rows, out).to(dt), torch.empty_like(y), torch.empty_like(x), torch.empty_like(w)
    ar.ar_expert_linear(x, w, y, **seg)
    ar.ar_expert_gated(x, w, wu, h, **seg)
    ar.ar_expert_linear_bwd(dy, x, w, dxs=dxs, dw=dw, **seg)
    for e in {0, n // 2, n - 1}:
        r = slice(e * per, (e + 1) * per)
        ref.close(y[r], *ref.rounded(ref.mm(x[r], w[e].t()), dt), "ys")
        ref.close(h[r], *ref.gated(x[r], w[e], wu[e], ar.AR_ACT_SILU, dt)[0], "out")
        ref.close(dxs[r], *ref.rounded(ref.mm(dy[r], w[e]), dt), "dxs")
        ref.close(dw[e], *ref.rounded(ref.mm(dy[r].t(), x[r]), dt), "dw")


@pytest.mark.parametrize("rows", [1, 16, 128, 513])
def test_same_rows_same_bits(rows):
    """A row's result does not depend on the other experts' rows."""
    x, w = torch.randn(rows, 320, device=DEV).to(BF), torch.randn(3, 256, 320, device=DEV).to(BF)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    y, z = torch.empty(2 * rows + 900, 256, dtype=BF, device=DEV), torch.empty(2 * rows + 900, 256, dtype=BF, device=DEV)
    big = torch.randn(2 * rows + 900, 320, device=DEV).to(BF)
    big[:rows], cut = x, big.clone()
    ar.ar_expert_linear(big, w, y, offsets=i32(0, rows, rows, rows), counts=i32(rows, 0, 0))
    ar.ar_expert_linear(big, w, z, offsets=i32(0, rows, rows + 77, 2 * rows + 900), counts=i32(rows, 70, rows + 800))
    assert torch.equal(y[:rows], z[:rows])


def test_empty_calls():
    """No rows at all: forward calls do nothing, weights' gradients are set to zero."""
    x, w = torch.empty(0, 32, dtype=BF, device=DEV), torch.randn(2, 16, 32, device=DEV).to(BF)
    y, off = torch.empty(0, 16, dtype=BF, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    ar.ar_expert_linear(x, w, y, offsets=off)
    ar.ar_expert_gated(x, w, w.clone(), y, offsets=off)
    dw, dg = torch.full_like(w, 9.0), torch.full_like(w, 9.0)
    ar.ar_expert_linear_bwd(y, x, w, dxs=x.clone(), dw=dw, offsets=off)
    assert not dw.any()
    ar.ar_expert_gated_bwd(y, y.clone(), y.clone(), x, w, w.clone(), y.clone(), y.clone(), dxs=x.clone(), dw_gate=dg, dw_up=dw.fill_(9.0), offsets=off)
    assert not dw.any() and not dg.any()
