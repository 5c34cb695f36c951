"""A captured graph of all block-boundary operators replayed on new inputs, every output overwritten before each replay, so
that an operator which a replay left out would show. Sizes below and above those at which the norm's gradient and the sort
take a second launch and a workspace."""
import pytest
import torch

import all_reduce_reduction_ring_amd as ar
import block_ref as ref
from test_gpu_block import BF16, DEV, F32, gen, make_ids, norm_inputs, randn, workspace

pytestmark = pytest.mark.gpu
I32 = torch.int32
UNWRITTEN = 0x5A


def spoil(tensors):
    for t in tensors:
        t.view(torch.uint8).fill_(UNWRITTEN)


def spoiled(t):
    return t.contiguous().view(torch.uint8) == UNWRITTEN


@pytest.mark.parametrize("rows8", [False, True])
@pytest.mark.parametrize("n,rows,hidden,dt,k,experts", [(4, 96, 1536, BF16, 2, 8), (8, 700, 2048, BF16, 8, 64), (3, 1500, 1001, F32, 3, 300)])
def test_replays(n, rows, hidden, dt, k, experts, rows8):
    align, nb = 16, ref.blocks(hidden)
    two_launches = rows > 256
    assert two_launches == (ar.ar_expert_sort_workspace_size(rows, k, experts) > 0)
    new = lambda *s, dtype=dt: torch.empty(*s, dtype=dtype, device=DEV)
    ins, res, gamma = norm_inputs(n, rows, hidden, dt, True, False, 0)
    ids, w = make_ids(rows, k, experts, "some"), torch.rand(rows, k, device=DEV)
    dy = [torch.randn_like(x) for x in ins]
    cap = ar.ar_expert_rows(rows, k, experts, align)
    ro, rs, out, dw = new(rows, hidden), new(rows, dtype=F32), new(rows, hidden), new(rows, k, dtype=F32)
    outs = [new(rows, hidden, dtype=torch.uint8 if rows8 else dt) for _ in range(n)]
    sc = [new(rows, nb, dtype=F32) for _ in range(n)] if rows8 else None
    sv, svs = new(rows, hidden, dtype=torch.uint8), new(rows, nb, dtype=F32)
    off, cnt, pos, src = (new(s, dtype=I32) for s in (experts + 1, experts, (rows, k), cap))
    xs, xss = new(cap, hidden, dtype=torch.uint8 if rows8 else dt), new(cap, nb, dtype=F32) if rows8 else None
    ys, dys = randn(gen(3), cap, hidden).to(dt), new(cap, hidden)
    dxs, dg = [new(rows, hidden) for _ in range(n)], new(hidden, dtype=F32)
    sort_ws = workspace(ar.ar_expert_sort_workspace_size(rows, k, experts))
    norm_ws = workspace(ar.ar_allreduce_rmsnorm_bwd_workspace_size(rows, hidden))
    named = {"residual_out": ro, "rstd": rs, "saved": sv, "saved_scales": svs, "offsets": off, "counts": cnt, "pos": pos,
             "src": src, "xs": xs, "out": out, "dys": dys, "dweights": dw, "dgamma": dg}
    named.update({f"out {r}": o for r, o in enumerate(outs)}, **{f"dx {r}": d for r, d in enumerate(dxs)})
    if rows8:
        named.update({f"scales {r}": s for r, s in enumerate(sc)}, xs_scales=xss)

    def step():
        ar.ar_allreduce_rmsnorm(ins, gamma, outs, res, ro, rs, out_scales=sc, saved=sv, saved_scales=svs)
        ar.ar_expert_sort(ids, off, cnt, pos, src, align, sort_ws if two_launches else None)
        ar.ar_expert_dispatch(outs[0], pos, off, cnt, xs, sc[0] if rows8 else None, xss)
        ar.ar_expert_combine(ys, pos, out, w, ro)
        ar.ar_expert_combine_bwd(out, ys, pos, w, off, cnt, dys, dw)
        ar.ar_allreduce_rmsnorm_bwd(dy, sv, gamma, rs, dxs, dg, svs, out, norm_ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for i in range(3):
        g = gen(20 + i)
        for x in (*ins, *dy, res, ys):
            x.copy_(randn(g, *x.shape))
        w.copy_(torch.rand(rows, k, generator=g, device=DEV))
        ids.copy_(make_ids(rows, k, experts, "some", seed=30 + i))
        spoil(named.values())
        step()
        torch.cuda.synchronize()
        want = {what: t.clone() for what, t in named.items()}
        end = off[-1].item()  # rows from here on are not written
        for what, t in want.items():
            there = spoiled(t[:end] if what in ("xs", "dys", "xs_scales") else t)
            assert float(there.float().mean()) < 0.05, f"{what} was not written"
        spoil([*named.values(), sort_ws, norm_ws])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for what, t in named.items():
            assert torch.equal(t.view(torch.uint8), want[what].view(torch.uint8)), (i, what)
