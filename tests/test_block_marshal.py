"""The compiled argument checks of the block-boundary entry points: what does not plainly fit goes back to the checks in
Python, which name it, and both lead to the same calls."""
import sys
import warnings

import pytest
import torch

import all_reduce_reduction_ring_amd as ar

I32 = torch.int32


def _calls(dev, dt=torch.bfloat16):
    """(name, arguments of the compiled function, the outputs among them) of one fitting call each."""
    g = torch.Generator().manual_seed(1)
    mk = lambda *s: torch.randn(*s, generator=g).to(dev)
    rows, hidden, k, experts = 6, 200, 2, 4
    ins, outs = [mk(rows, hidden).to(dt) for _ in range(3)], [mk(rows, hidden).to(dt) for _ in range(3)]
    gamma, rstd, sc = mk(hidden).to(dt), mk(rows).abs() + 0.5, mk(rows, 2)
    new = lambda *s, t=dt: torch.zeros(*s, dtype=t, device=dev)
    ro, dg, ws = new(rows, hidden), new(hidden, t=torch.float32), new(1 << 20, t=torch.uint8)
    codes, scales = new(rows, hidden, t=torch.uint8), new(rows, 2, t=torch.float32)
    ids = torch.randint(0, experts, (rows, k), generator=g, dtype=I32).to(dev)
    off, cnt, pos, src = (new(s, t=I32) for s in (experts + 1, experts, (rows, k), rows * k))
    pos2 = torch.randperm(rows * k, generator=g).to(I32).view(rows, k).to(dev)
    w, xs, dys, dw = mk(rows, k), new(rows * k, hidden), new(rows * k, hidden), new(rows, k, t=torch.float32)
    ys, out = mk(rows * k, hidden).to(dt), new(rows, hidden)
    return [
        ("rmsnorm", (ins, gamma, outs, ins[0].clone(), ro, rstd.clone(), None, codes, scales, 1e-5, None), [*outs, ro, codes, scales]),
        ("rmsnorm_bwd", (ins, outs[0].clone(), gamma, rstd, outs, dg, None, ins[1].clone(), ws, None), [*outs, dg]),
        ("expert_sort", (ids, off, cnt, pos, src, 1, None, None), [off, cnt, pos, src]),
        ("expert_dispatch", (ins[0], pos2, None, None, xs, None, None, None), [xs]),
        ("expert_combine", (ys, pos2, out, w, None, None), [out]),
        ("expert_combine_bwd", (ins[0], ys, pos2, w, None, None, dys, dw, None), [dys, dw]),
    ]


PUBLIC = {"rmsnorm": "ar_allreduce_rmsnorm", "rmsnorm_bwd": "ar_allreduce_rmsnorm_bwd", "expert_sort": "ar_expert_sort",
          "expert_dispatch": "ar_expert_dispatch", "expert_combine": "ar_expert_combine",
          "expert_combine_bwd": "ar_expert_combine_bwd"}


@pytest.fixture
def native():
    if ar._native is None:
        ar._load_native()
    assert ar._native, "the compiled checks were not built"
    return ar._native


def test_host_tensors_come_back(native):
    for name, args, _ in _calls("cpu"):
        assert getattr(native, name)(*args) is None, name
        with pytest.raises(ValueError):
            _public(name, args)


def test_wrong_numbers_and_kinds_of_arguments_come_back(native):
    for name, args, _ in _calls("cpu"):
        f = getattr(native, name)
        assert f() is None and f(*args, None) is None
        for i in range(len(args)):
            assert f(*args[:i], object(), *args[i + 1:]) is None, (name, i)
            assert f(*args[:i], "x", *args[i + 1:]) is None, (name, i)
    assert native.rmsnorm([], None, [], None, None, None, None, None, None, 0.0, None) is None
    with pytest.raises(TypeError):
        native.bind(1)
    with pytest.raises(ValueError):
        native.bind(0, 0, 0, 0, 0, 0, len, len)


def _public(name, a):
    """The public entry point with the compiled function's arguments."""
    f = getattr(ar, PUBLIC[name])
    if name == "rmsnorm":
        return f(*a[:9], eps=a[9], stream=a[10])
    if name == "rmsnorm_bwd":
        return f(*a[:6], saved_scales=a[6], residual_grad=a[7], workspace=a[8], stream=a[9])
    if name == "expert_sort":
        return f(*a[:5], align=a[5], workspace=a[6], stream=a[7])
    return f(*a)


def test_without_the_compiled_checks(monkeypatch):
    """A missing module is said once; the calls go through the checks in Python."""
    monkeypatch.setattr(ar, "_native", None)
    monkeypatch.setitem(sys.modules, ar.__name__ + "._marshal", None)
    monkeypatch.delattr(ar, "_marshal", raising=False)
    with pytest.warns(UserWarning, match="_marshal.so"):
        assert ar._load_native() is False
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError):
            ar.ar_allreduce_rmsnorm([torch.zeros(2, 8)], torch.zeros(8), [torch.zeros(2, 8)])


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
def test_both_ways_lead_to_the_same_call(native, monkeypatch, dt):
    for (name, args, outs), (_, args2, outs2) in zip(_calls("cuda:0", dt), _calls("cuda:0", dt)):
        assert getattr(native, name)(*args) == ar.AR_OK, name
        record = ar.ar_last_call()
        monkeypatch.setattr(ar, "_native", False)
        _public(name, args2)
        monkeypatch.setattr(ar, "_native", native)
        again = ar.ar_last_call()
        assert record["entry"] == again["entry"] and record["count"] == again["count"] and again["status"] == ar.AR_OK
        torch.cuda.synchronize()
        for a, b in zip(outs, outs2):
            assert torch.equal(a, b), name


@pytest.mark.gpu
def test_misfits_on_the_gpu_come_back_and_are_named(native):
    """Wrong types, shapes, orders and overlaps: the compiled checks return None or the library's status, and the public
    call raises."""
    for name, args, _ in _calls("cuda:0"):
        for i, a in enumerate(args):
            t = a[0] if isinstance(a, list) else a
            if not isinstance(t, torch.Tensor) or t.dtype == torch.uint8:
                continue
            for bad in (t.to(torch.float64), t.reshape(-1)[:-1], t.cpu(),
                        torch.empty(*t.shape, 2, dtype=t.dtype, device="cuda:0")[..., 0]):
                if name == "expert_sort" and i == 4 and bad.dtype == I32 and bad.is_cuda and bad.is_contiguous():
                    continue  # src may have any length of its own; one too short is the library's to refuse
                new = list(args)
                new[i] = [bad] + a[1:] if isinstance(a, list) else bad
                assert getattr(native, name)(*new) is None, (name, i)
                with pytest.raises(ValueError):
                    _public(name, new)
    name, args, _ = _calls("cuda:0")[0]
    assert native.rmsnorm(args[0], args[1], [args[0][1], args[0][0], args[0][2]], *args[3:]) == ar.AR_ERR_ALIAS
    with pytest.raises(ar.ArError):
        ar.ar_allreduce_rmsnorm(args[0], args[1], [args[0][1], args[0][0], args[0][2]])


@pytest.mark.gpu
def test_streams_and_both_kinds_of_codes():
    """A stream object, a raw handle and the current stream; code buffers of both 8-bit types in one list."""
    x, gamma = torch.randn(40, 256, device="cuda:0"), torch.ones(256, device="cuda:0")
    want, got = torch.empty_like(x), torch.zeros_like(x)
    ar.ar_allreduce_rmsnorm([x], gamma, [want])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    ar.ar_allreduce_rmsnorm([x], gamma, [got], stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    got.zero_()
    torch.cuda.synchronize()
    ar.ar_allreduce_rmsnorm([x], gamma, [got], stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want)
    with torch.cuda.stream(s):
        got.zero_()
        ar.ar_allreduce_rmsnorm([x], gamma, [got])
    s.synchronize()
    assert torch.equal(got, want)
    codes = [torch.empty(40, 256, dtype=torch.uint8, device="cuda:0"),
             torch.empty(40, 256, dtype=torch.float8_e4m3fn, device="cuda:0")]
    sc = [torch.empty(40, 2, device="cuda:0") for _ in codes]
    ar.ar_allreduce_rmsnorm([x, x.clone()], gamma, codes, out_scales=sc)
    assert torch.equal(codes[0], codes[1].view(torch.uint8))
