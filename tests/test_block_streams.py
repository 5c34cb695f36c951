"""Stream handles that are no addresses: refused, never another stream."""
import pytest
import torch

import all_reduce_reduction_ring_amd as ar
from test_block_marshal import _calls, _public

BAD = [1 << 80, 1 << 64, (1 << 64) - 1, -1, -(1 << 70)]


@pytest.mark.parametrize("handle", BAD)
def test_the_binding_refuses_them(handle):
    with pytest.raises(ValueError, match="stream"):
        ar._stream(handle)
    assert ar._stream(1 << 40).value == 1 << 40 and not ar._stream(0).value


@pytest.mark.gpu
@pytest.mark.parametrize("handle", BAD)
def test_nothing_is_called(handle):
    if ar._native is None:
        ar._load_native()
    for name, args, outs in _calls("cuda:0"):
        args, before = args[:-1] + (handle,), [o.clone() for o in outs]
        ar.ar_allreduce_rmsnorm([torch.ones(1, 8, device="cuda:0")], torch.ones(8, device="cuda:0"), [torch.ones(1, 8, device="cuda:0")])
        record = ar.ar_last_call()
        assert getattr(ar._native, name)(*args) is None, name
        with pytest.raises(ValueError, match="stream"):
            _public(name, args)
        torch.cuda.synchronize()
        assert ar.ar_last_call() == record and all(torch.equal(a, b) for a, b in zip(outs, before)), name
