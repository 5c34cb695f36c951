"""The bound and eps of ar_grad_clip are numbers on the host. A GPU tensor is refused by both ways into the library: reading
it would wait for the GPU, and break a capture."""
import ctypes

import numpy as np
import pytest
import torch

import all_reduce_reduction_ring_amd as ar


def test_numbers():
    for v, want in ((1, 1.0), (0.25, 0.25), (True, 1.0), (np.float32(0.5), 0.5), (np.float64(2), 2.0), (np.int64(3), 3.0),
                    (torch.tensor(0.5), 0.5), (torch.tensor([2]), 2.0), (float("inf"), float("inf"))):
        assert ar._reals(max_norm=v, eps=0) == (want, 0.0) and type(ar._reals(x=v)[0]) is float
    for v in (None, "x", object(), 1 << 2000, torch.ones(2), torch.ones((), device="meta"), torch.ones(1, device="meta"), 1j):
        with pytest.raises(ValueError, match="max_norm"):
            ar._reals(eps=1.0, max_norm=v)


@pytest.mark.gpu
@pytest.mark.parametrize("compiled", [True, False])
def test_gpu_tensors_are_refused(monkeypatch, compiled):
    if ar._native is None:
        ar._load_native()
    assert ar._native
    if not compiled:
        monkeypatch.setattr(ar, "_native", False)
    g = torch.full((100,), 3.0, device="cuda:0")
    plan, norm = ar.ar_grad_plan([g]), torch.full((1,), -1.0, device="cuda:0")
    ws = torch.empty(ar.ar_grad_norm_workspace_size(plan.shape[0]), dtype=torch.uint8, device="cuda:0")
    one = torch.ones(1, device="cuda:0")
    for bad in (dict(max_norm=one), dict(max_norm=one[0]), dict(max_norm=1.0, eps=one)):
        with pytest.raises(ValueError, match="number"):
            ar.ar_grad_clip(plan, norm=norm, workspace=ws, **bad)
    torch.cuda.synchronize()
    assert norm.item() == -1.0 and bool((g == 3.0).all())
    # in a capture too, which goes on
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="number"):
            ar.ar_grad_clip(plan, one, norm, workspace=ws)
        ar.ar_grad_clip(plan, np.float32(15.0), norm, workspace=ws)
    for _ in range(3):
        g.fill_(3.0)
        norm.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        # 30 + eps is off 30 by a step of it at most (2^-23.9 of 30); one division, one product: 2^-24 each
        assert norm.item() == 30.0 and bool(((g - 1.5).abs() <= 1.5 * 2.0 ** -22).all())


@pytest.mark.gpu
def test_host_numbers_of_any_kind_are_the_same_call():
    out = []
    for v in (0.5, np.float32(0.5), np.float64(0.5), torch.tensor(0.5), ctypes.c_float(0.5).value):
        g = torch.linspace(-1, 1, 301, device="cuda:0")
        plan, norm = ar.ar_grad_plan([g]), torch.empty(1, device="cuda:0")
        ws = torch.empty(ar.ar_grad_norm_workspace_size(plan.shape[0]), dtype=torch.uint8, device="cuda:0")
        ar.ar_grad_clip(plan, v, norm, eps=type(v)(0.0) if not torch.is_tensor(v) else torch.tensor(0.0), workspace=ws)
        out.append(g)
    assert all(torch.equal(out[0], o) for o in out)
