"""The compiled argument checks of the experts' products and the gradients' norm: what does not plainly fit goes back to the
checks in Python, and both lead to the same calls."""
import pytest
import torch

import all_reduce_reduction_ring_amd as ar

I32 = torch.int32


def _calls(dev, dt=torch.bfloat16):
    """(name, arguments of the compiled function, the outputs among them, the public call) of fitting calls."""
    g = torch.Generator().manual_seed(1)
    mk = lambda *s: (torch.randn(*s, generator=g) * 0.3).to(dt).to(dev)
    experts, inner, hidden, rows = 3, 40, 72, 20
    off, cnt = torch.tensor([0, 8, 8, 20], dtype=I32, device=dev), torch.tensor([7, 0, 12], dtype=I32, device=dev)
    both, dboth = mk(experts, 2 * inner, hidden), torch.zeros(experts, 2 * inner, hidden, dtype=dt, device=dev)
    wg, wu, dwg, dwu = both[:, :inner], both[:, inner:], dboth[:, :inner], dboth[:, inner:]
    x, y, gate, up, dout = mk(rows, hidden), mk(rows, inner), mk(rows, inner), mk(rows, inner), mk(rows, inner)
    new = lambda w: torch.zeros(rows, w, dtype=dt, device=dev)
    out, og, ou, dg, du, dx, w, dw = new(inner), new(inner), new(inner), new(inner), new(inner), new(hidden), mk(experts, inner, hidden), torch.zeros(experts, inner, hidden, dtype=dt, device=dev)
    calls = [
        ("expert_gated", (x, wg, wu, out, off, cnt, og, ou, 1, None), [out, og, ou],
         lambda a: ar.ar_expert_gated(*a[:4], offsets=a[4], counts=a[5], gate=a[6], up=a[7], act=a[8], stream=a[9])),
        ("expert_gated_bwd", (dout, gate, up, x, wg, wu, dg, du, dx, dwg, dwu, off, cnt, 2, None), [dg, du, dx, dboth],
         lambda a: ar.ar_expert_gated_bwd(*a[:8], dxs=a[8], dw_gate=a[9], dw_up=a[10], offsets=a[11], counts=a[12], act=a[13],
                                          stream=a[14])),
        ("expert_linear", (x, w, new(inner), off, None, None), [],
         lambda a: ar.ar_expert_linear(*a[:3], offsets=a[3], counts=a[4], stream=a[5])),
        ("expert_linear_bwd", (dout, x, w, new(hidden), dw, off, cnt, None), [dw],
         lambda a: ar.ar_expert_linear_bwd(*a[:3], dxs=a[3], dw=a[4], offsets=a[5], counts=a[6], stream=a[7])),
    ]
    for name, args, outs, _ in calls[2:]:
        outs.append(args[2] if name == "expert_linear" else args[3])
    if dev != "cpu":
        ts, outs = [mk(1000), mk(33, 7)], [torch.zeros(1000, dtype=dt, device=dev), torch.zeros(33, 7, dtype=dt, device=dev)]
        plan, n1, n2 = ar.ar_grad_plan(ts, outs), torch.zeros(1, device=dev), torch.zeros((), device=dev)
        ws = torch.zeros(1 << 14, dtype=torch.uint8, device=dev)
        keep = [plan, n1, n2, ws, ts]
        calls += [("grad_norm", (plan, n1, 1, ws, None), [n1], lambda a, keep=keep: ar.ar_grad_norm(a[0], a[1], kind=a[2], workspace=a[3], stream=a[4])),
                  ("grad_clip", (plan, 0.5, n2, 0, 1e-6, ws, None), [n2, *outs],
                   lambda a, keep=keep: ar.ar_grad_clip(a[0], a[1], a[2], kind=a[3], eps=a[4], workspace=a[5], stream=a[6]))]
    return calls


@pytest.fixture
def native():
    if ar._native is None:
        ar._load_native()
    assert ar._native, "the compiled checks were not built"
    return ar._native


def test_host_tensors_and_wrong_arguments_come_back(native):
    for name, args, _, public in _calls("cpu"):
        f = getattr(native, name)
        assert f(*args) is None and f() is None and f(*args, None) is None, name
        with pytest.raises(ValueError):
            public(args)
        for i in range(len(args)):
            assert f(*args[:i], object(), *args[i + 1:]) is None and f(*args[:i], 1 << 80, *args[i + 1:]) is None, (name, i)
    for name, n in (("grad_norm", 5), ("grad_clip", 7)):
        assert getattr(native, name)(*[torch.zeros(1)] * n) is None
    with pytest.raises(TypeError):
        native.bind_products(1)
    with pytest.raises(ValueError):
        native.bind_products(0, 0, 0, 0, 0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
def test_both_ways_lead_to_the_same_call(native, monkeypatch, dt):
    for (name, args, outs, _), (_, args2, outs2, public) in zip(_calls("cuda:0", dt), _calls("cuda:0", dt)):
        assert getattr(native, name)(*args) == ar.AR_OK, name
        record = ar.ar_last_call()
        monkeypatch.setattr(ar, "_native", False)
        public(args2)
        monkeypatch.setattr(ar, "_native", native)
        again = ar.ar_last_call()
        assert record["entry"] == again["entry"] and record["count"] == again["count"] and again["status"] == ar.AR_OK
        torch.cuda.synchronize()
        for a, b in zip(outs, outs2):
            assert torch.equal(a, b) and a.any(), name


@pytest.mark.gpu
def test_what_does_not_fit_is_named(native):
    """Wrong types, shapes, layouts and numbers on the GPU, through the public call; nothing is written."""
    for name, args, outs, public in _calls("cuda:0"):
        before = [o.clone() for o in outs]
        for i, a in enumerate(args):
            if torch.is_tensor(a) and a.dim() >= 1 and a.dtype != torch.uint8:
                wrong = [a[:-1] if a.dim() > 1 or a.numel() > 1 else a.double(), a.cpu(), a.to(torch.float64) if a.is_floating_point() else a.long().float()]
                if a.dim() >= 2:
                    wrong.append(a.transpose(-1, -2).contiguous().transpose(-1, -2))
            elif isinstance(a, (int, float)) and not isinstance(a, bool):
                wrong = [-1, 1 << 40]
            else:
                continue
            for w in wrong:
                if name == "grad_clip" and i == 1 and w == 1 << 40 or name.startswith("grad") and torch.is_tensor(w) and w.dim() == 2 and w.dtype == torch.int64 and w.is_cuda and w.is_contiguous():
                    continue  # a large norm and a part of a table are fitting arguments
                if name == "grad_clip" and i == 4 and w == 1 << 40:
                    continue
                with pytest.raises((ValueError, ar.ArError)):
                    public(args[:i] + (w,) + args[i + 1:])
        for handle in (1 << 80, -1):
            with pytest.raises(ValueError, match="stream"):
                public(args[:-1] + (handle,))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, before)), name
