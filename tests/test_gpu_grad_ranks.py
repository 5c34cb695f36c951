"""Clipping by a norm over several ranks' gradients: every rank passes max_norm * (own + eps) / (all + eps), so that its own
factor is the common one. Here the ranks are tables on one GPU."""
import math

import pytest
import torch

import all_reduce_reduction_ring_amd as ar

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("kind", [ar.AR_NORM_L2, ar.AR_NORM_MAX])
@pytest.mark.parametrize("share", [0.05, 0.9, 1.5, 40.0])  # of the norm over all ranks; the last two leave all as it is
def test_a_norm_over_ranks(kind, share):
    g, eps = torch.Generator(device=DEV).manual_seed(1), 1e-6
    # one rank's gradients are a hundred times another's, one rank's are zero
    ranks = [[(torch.randn(n, generator=g, device=DEV) * s).to(dt) for n, dt in ((5003, torch.float32), (70_001, torch.bfloat16))]
             for s in (1.0, 0.01, 0.3, 0.0)]
    plans = [ar.ar_grad_plan(r) for r in ranks]
    ws = torch.empty(max(ar.ar_grad_norm_workspace_size(p.shape[0]) for p in plans), dtype=torch.uint8, device=DEV)
    norms = []
    for p in plans:
        norm = torch.empty(1, device=DEV)
        ar.ar_grad_norm(p, norm, kind=kind, workspace=ws)
        norms.append(norm.item())
    total = max(norms) if kind == ar.AR_NORM_MAX else math.sqrt(math.fsum(n * n for n in norms))
    bound = share * total
    want = [[t.double() * min(1.0, bound / (total + eps)) for t in r] for r in ranks]
    for p, r, own, ws_ in zip(plans, ranks, norms, want):
        again = torch.empty(1, device=DEV)
        ar.ar_grad_clip(p, bound * (own + eps) / (total + eps), again, kind=kind, eps=eps, workspace=ws)
        assert again.item() == own
        for t, w in zip(r, ws_):
            # half steps of fp32: the norms (each part's enters the total), the bound passed on, own + eps, the quotient, the
            # product; half a step of the type
            f = torch.finfo(t.dtype)
            assert ((t.double() - w).abs() <= w.abs() * (7 * 2.0 ** -24 + f.eps / 2) + f.smallest_normal * f.eps).all()
