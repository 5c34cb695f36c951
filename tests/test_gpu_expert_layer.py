"""The example of examples/expert_layer.py: its gradients against autograd in 64 bits, and a few steps of it."""
import importlib.util
import os

import pytest
import torch

import all_reduce_reduction_ring_amd as ar
import block_ref as ref

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("expert_layer", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_loss_goes_down(example):
    losses = example.main()
    assert all(b < a for a, b in zip(losses, losses[1:]))


def test_layer_against_autograd(example):
    """fp32 storage, so the only roundings are fp32's and the checkpoint's: half a step of E4M3 (relative 2^-4) of every
    element of the saved residual, which reaches dx through xhat and dgamma through xhat."""
    ranks, tokens, hidden, experts, k = 3, 40, 256, 5, 2
    g = torch.Generator().manual_seed(2)
    randn = lambda *s: torch.randn(*s, generator=g)
    parts, residual, gamma = [randn(tokens, hidden) for _ in range(ranks)], randn(tokens, hidden), 1 + 0.2 * randn(hidden)
    w, dout = randn(experts, hidden, hidden) / 16, randn(tokens, hidden)
    ids, weights = example.route(residual, randn(hidden, experts), k)
    block = example.ExpertBlock(ranks, tokens, hidden, experts, k, dtype=torch.float32)
    dev = lambda t: t.cuda()
    dp, rg, gg, ww = [dev(p) for p in parts], dev(residual), dev(gamma), dev(w)
    out = block.forward(dp, rg, gg, ww, dev(ids), dev(weights)).cpu().double()
    dx, dgamma, dw, dweights = (t.cpu().double() for t in block.backward(dev(dout), gg, ww, dev(weights)))
    # 64 bits
    req = lambda t: t.double().requires_grad_(True)
    h, g64, w64, r64 = req(sum(p.double() for p in parts) + residual.double()), req(gamma), req(w), req(weights)
    y = h * (h.square().mean(1, keepdim=True) + example.EPS).rsqrt() * g64
    rows = torch.stack([torch.stack([y[t] @ w64[ids[t, j]] for j in range(k)]) for t in range(tokens)])
    want = (rows * r64[:, :, None]).sum(1) + h
    want.backward(dout.double())
    # forward, dw, dweights: products of 256 fp32 terms (and of the library's own order), 2^-24 each, with room for the
    # norm's statistics; sizes by the terms' magnitudes
    tol = 1024 * ref.U
    assert ((out - want.detach()).abs() <= tol * (want.detach().abs() + rows.detach().abs().sum(1) + 16)).all()
    assert ((dw - w64.grad).norm() <= tol * w64.grad.norm())
    assert ((dweights - r64.grad).norm() <= tol * r64.grad.norm() + tol)
    # dx = rstd (gd - xhat mean(gd xhat)) + dout: xhat off by 2^-4 of itself changes the second term by at most
    # 2 * 2^-4 + 2^-8 of its size |xhat| mean |gd xhat|
    rstd = (h.detach().square().mean(1, keepdim=True) + example.EPS).rsqrt()
    xh = (h.detach() * rstd).abs()
    dn = torch.zeros(tokens, hidden, dtype=torch.float64)
    for t in range(tokens):
        for j in range(k):
            dn[t] += (weights[t, j].double() * dout[t].double()) @ w[ids[t, j]].double().t()
    gd = (dn * gamma.double()).abs()
    bound = rstd * xh * (gd * xh).mean(1, keepdim=True) * (2.0 ** -3 + 2.0 ** -8) + tol * (gd * rstd + dout.double().abs() + 1)
    assert ((dx - h.grad).abs() <= bound).all()
    bound = (dn.abs() * xh).sum(0) * 2.0 ** -4 + tol * (dn.abs() * xh).sum(0)
    assert ((dgamma - g64.grad).abs() <= bound).all()
    assert ar.ar_last_call()["status"] == ar.AR_OK
