"""The gated layer of examples/expert_layer.py: it runs, its gradients against autograd in 64 bits, and its clipping."""
import importlib.util
import math
import os

import pytest
import torch

import all_reduce_reduction_ring_amd as ar
import product_ref as ref

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("expert_layer", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_it_runs(example):
    losses = example.main_gated(steps=2, tokens=64, hidden=256, inner=128, experts=8)
    assert all(math.isfinite(x) for x in losses)


@pytest.mark.parametrize("act", ref.ACTS)
def test_gradients_against_autograd(example, act):
    """fp32 storage: the roundings are fp32's, sums of at most 256 terms through six operators, and the checkpoint's of the
    residual (half a step of E4M3, relative 2^-4), which reaches dgamma and the residual's gradient only."""
    ranks, tokens, hidden, inner, experts, k = 2, 40, 256, 72, 5, 2
    g = torch.Generator().manual_seed(3)
    randn = lambda *s: torch.randn(*s, generator=g)
    parts, residual, gamma = [randn(tokens, hidden) for _ in range(ranks)], randn(tokens, hidden), 1 + 0.2 * randn(hidden)
    w_in, w_out, dout = randn(experts, 2 * inner, hidden) / 16, randn(experts, hidden, inner) / 8, randn(tokens, hidden)
    ids, weights = example.route(residual, randn(hidden, experts), k)
    block = example.GatedExpertBlock(ranks, tokens, hidden, inner, experts, k, dtype=torch.float32, act=act)
    dev = lambda t: t.cuda()
    win, wout, gg, rw = dev(w_in), dev(w_out), dev(gamma), dev(weights)
    out = block.forward([dev(p) for p in parts], dev(residual), gg, win, wout, dev(ids), rw).cpu().double()
    grads = [t.clone() for t in block.backward(dev(dout), gg, win, wout, rw)]
    _, dgamma, dwi, dwo, dweights = (t.cpu().double() for t in grads)
    req = lambda t: t.double().requires_grad_(True)
    h, g64, i64, o64, r64 = sum(p.double() for p in parts) + residual.double(), req(gamma), req(w_in), req(w_out), req(weights)
    y = h * (h.square().mean(1, keepdim=True) + example.EPS).rsqrt() * g64
    rows = torch.stack([torch.stack([(ref.act(i64[e, :inner] @ y[t], act) * (i64[e, inner:] @ y[t])) @ o64[e].t()
                                     for e in ids[t].tolist()]) for t in range(tokens)])
    want = (rows * r64[:, :, None]).sum(1) + h
    want.backward(dout.double())
    tol = 6 * 2 * 256 * 2.0 ** -24
    assert (out - want.detach()).norm() <= tol * want.detach().norm()
    for got, w in ((dwi, i64.grad), (dwo, o64.grad), (dweights, r64.grad)):
        assert (got - w).norm() <= tol * w.norm() + tol
    assert (dgamma - g64.grad).norm() <= (2.0 ** -4 + tol) * g64.grad.norm() * 2
    # clipping: the norm of the three, and all of them times the same number
    norm = math.sqrt(sum(t.cpu().double().square().sum().item() for t in grads[1:4]))
    assert abs(block.clip(norm / 3).item() - norm) <= norm * 2 ** -23
    coef = (norm / 3) / (norm + 1e-6)
    for now, before in zip((block.dgamma, block.dw_in, block.dw_out), (grads[1], grads[2], grads[3])):
        b = before.double() * coef
        assert ((now.double() - b).abs() <= b.abs() * 5 * 2 ** -24 + 1e-37).all()
    assert ar.ar_last_call()["entry"] == "ar_grad_clip"
