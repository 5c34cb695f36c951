"""The block-boundary operators at sizes on both sides of every choice their host code makes: workgroups of one and of
several rows, one launch and two, rank counts with and without a kernel of their own, streaming and cached access, lanes
per token, sort tiles. Against the 64-bit references of block_ref.py."""
import pytest
import torch

import all_reduce_reduction_ring_amd as ar
import block_ref as ref
from test_gpu_block import (BF16, E4M3, F16, F32, Guarded, bwd_inputs, gen, make_ids, norm_inputs, randn, run_sort,
                            saved_f64, workspace)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def check_bwd(n, rows, hidden, dt, rgrad, save8, offset, in_place):
    ins, saved, scales, gamma, rstd, rg = bwd_inputs(n, rows, hidden, dt, rgrad, save8, False, offset)
    dx, dg, ddx, ddg = ref.norm_bwd(ins, saved_f64(saved, scales), gamma, rstd, rg, min(rows, 64) + 128)
    put = Guarded(offset)
    outs = ins if in_place else [put.new((rows, hidden), dt) for _ in range(n)]
    dgamma = put.new((hidden,), F32)
    ws = workspace(ar.ar_allreduce_rmsnorm_bwd_workspace_size(rows, hidden))
    ar.ar_allreduce_rmsnorm_bwd(ins, saved, gamma, rstd, outs, dgamma, scales, rg, ws)
    torch.cuda.synchronize()
    put.check()
    for r in range(n):
        ref.close(outs[r], dx, ddx, f"dx {r}")
    ref.close(dgamma, dg, ddg, "dgamma")


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,rows,hidden,dt,rgrad,save8,offset", [
    (1, 256, 512, BF16, True, False, 0), (1, 257, 512, BF16, True, True, 0), (2, 511, 200, F16, True, True, 1),
    (3, 513, 1000, BF16, False, False, 0), (4, 2049, 64, F32, True, True, 0), (5, 700, 1601, BF16, True, False, 1),
    (8, 300, 4096, F32, True, True, 0), (8, 256, 1536, BF16, True, True, 0), (6, 2500, 130, F32, True, False, 1),
    (7, 1300, 2050, F16, True, True, 0), (1, 9000, 37, BF16, True, False, 0), (2, 256, 8192, F32, True, False, 0),
    (3, 300, 9000, BF16, True, True, 0), (9, 40, 20000, F16, True, True, 0), (1, 255, 4, F32, False, False, 0),
    (2, 300, 3, BF16, True, True, 0),
])
def test_norm_bwd(n, rows, hidden, dt, rgrad, save8, offset, in_place):
    check_bwd(n, rows, hidden, dt, rgrad, save8, offset, in_place)


@pytest.mark.parametrize("n,rows,hidden,dt", [(8, 1100, 4096, BF16), (1, 9000, 4096, F16), (3, 2200, 2048, F32),
                                              (5, 1100, 8192, BF16), (4, 2600, 4160, BF16)])
def test_streaming_norm_and_its_gradient(n, rows, hidden, dt):
    """128 MiB and more in whole lines."""
    assert rows * hidden * dt.itemsize * (2 * n + 2) >= 128 << 20
    ins, res, gamma = norm_inputs(n, rows, hidden, dt, True, False, 0)
    nb, put = ref.blocks(hidden), Guarded(0)
    for out8 in (False, True):
        outs = [put.new((rows, hidden), E4M3 if out8 else dt) for _ in range(n)]
        sc = [put.new((rows, nb), F32) for _ in range(n)] if out8 else None
        ro, rs = put.new((rows, hidden), dt), put.new((rows,), F32)
        sv, svs = put.new((rows, hidden), torch.uint8), put.new((rows, nb), F32)
        ar.ar_allreduce_rmsnorm(ins, gamma, outs, res, ro, rs, sc, sv, svs, eps=1e-4)
        torch.cuda.synchronize()
        put.check()
        h, rstd, y, dh, rel, dy = ref.norm(ins, res, gamma, 1e-4)
        ref.close(ro, h, dh, "residual_out")
        ref.close(rs[:, None], rstd, rel * rstd, "rstd")
        ref.close_codes(sv, svs, h, dh, "saved")
        for r in (0, n - 1):
            if out8:
                ref.close_codes(outs[r], sc[r], y, dy, f"out {r}")
            else:
                ref.close(outs[r], y, dy, f"out {r}")
            assert torch.equal(outs[r].view(torch.uint8), outs[0].view(torch.uint8))
        del outs, sc
    check_bwd(n, rows, hidden, dt, True, True, 0, False)


@pytest.mark.parametrize("tokens,k,hidden,dt", [
    (2047, 3, 1000, BF16), (2048, 3, 1000, BF16), (2100, 2, 2000, F16), (2100, 1, 2600, F32), (3000, 2, 60, BF16),
    (2050, 10, 520, F32), (2200, 8, 4096, BF16), (700, 12, 8192, F32)])
def test_rows_by_lanes_and_streaming(tokens, k, hidden, dt):
    off, cnt, pos, src = run_sort(make_ids(tokens, k, 24, "some"), 24, 16)
    g, put, rows = gen(6), Guarded(0), src.numel()
    x = put.new((tokens, hidden), dt, randn(g, tokens, hidden))
    xs = put.new((rows, hidden), dt)
    ar.ar_expert_dispatch(x, pos, off, cnt, xs)
    torch.cuda.synchronize()
    put.check()
    end = off[-1].item()
    there = src[:end] >= 0
    assert torch.equal(xs[:end][there], x[src[:end][there].long() // k]) and bool((xs[:end][~there] == 0).all())
    ys, w = put.new((rows, hidden), dt, randn(g, rows, hidden)), put.new((tokens, k), F32, randn(g, tokens, k))
    ys[src < 0] = float("nan")
    out = put.new((tokens, hidden), dt)
    ar.ar_expert_combine(ys, pos, out, w, x)
    torch.cuda.synchronize()
    put.check()
    want, bound = ref.combine(ys, pos.cpu(), w, x)
    ref.close(out, want, bound, "out")
    dys, dw = put.new((rows, hidden), dt), put.new((tokens, k), F32)
    ar.ar_expert_combine_bwd(x, ys, pos, w, off, cnt, dys, dw)
    torch.cuda.synchronize()
    put.check()
    want, dweights, bound = ref.combine_bwd(x, ys, pos.cpu(), w, rows)
    ref.close(dys[:end], want[:end], ref.U * want[:end].abs(), "dys")
    ref.close(dw, dweights, bound, "dweights")


@pytest.mark.parametrize("tokens,k,experts,align", [(4095, 1, 1024, 128), (4096, 1, 1024, 3), (4097, 1, 1, 64),
                                                    (1025, 4, 256, 128), (65_537, 8, 96, 16), (337_501, 8, 7, 5)])
def test_sort_tiles(tokens, k, experts, align):
    """One workgroup and many, and tiles of more slots than a thread holds."""
    ids = make_ids(tokens, k, experts, "some" if experts > 1 else "even")
    off, cnt, pos, src = run_sort(ids, experts, align, extra=70)
    offsets, counts, p, s = ref.sort(ids.cpu(), experts, align)
    assert off.tolist() == offsets and cnt.tolist() == counts
    assert torch.equal(pos.cpu().reshape(-1), torch.tensor(p, dtype=torch.int32))
    want = torch.full((src.numel(),), -1, dtype=torch.int32)
    want[torch.tensor(list(s.keys()))] = torch.tensor(list(s.values()), dtype=torch.int32)
    assert torch.equal(src.cpu(), want)
