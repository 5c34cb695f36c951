"""Calls on nothing: no tokens for buffers that hold rows, as on a rank that the router passed by, and no rows for tokens.
An empty tensor has no address, which is not the same as an argument left out."""
import pytest
import torch

import all_reduce_reduction_ring_amd as ar

A, STEP = 0x60000000, 1 << 24  # addresses that no call here reads


def _dispatch(tokens, rows, x_scales, xs_scales, xs=A + STEP, es=1):
    return ar.lib().ar_expert_dispatch(A, x_scales, A + 4 * STEP, None, None, tokens, 2, 1, 256, es, xs, xs_scales, rows, None)


def test_no_tokens_of_codes():
    assert _dispatch(0, 16, None, A + 2 * STEP) == ar.AR_OK
    assert _dispatch(0, 0, None, None) == ar.AR_OK and _dispatch(0, 16, A + 3 * STEP, A + 2 * STEP) == ar.AR_OK
    assert _dispatch(0, 16, None, A + 2 * STEP, es=2) == ar.AR_ERR_INVALID  # scales of rows that have none


def test_no_rows_for_codes():
    """Gets past the check of the scales: refused for positions that overlap the tokens."""
    args = (A, A + 2 * STEP, A, None, None, 3, 2, 1, 256, 1, None, None, 0, None)
    assert ar.lib().ar_expert_dispatch(*args) == ar.AR_ERR_ALIAS
    for scales in ((A + 2 * STEP, None), (None, A + 2 * STEP)):
        assert _dispatch(3, 16, *scales) == ar.AR_ERR_INVALID


@pytest.mark.gpu
def test_tensors():
    new = lambda *s, dt=torch.uint8: torch.full(s, 3, dtype=dt, device="cuda:0")
    i32, f32 = torch.int32, torch.float32
    xs, xsc = new(16, 256), new(16, 2, dt=f32)
    ar.ar_expert_dispatch(new(0, 256), new(0, 2, dt=i32), None, None, xs, x_scales=new(0, 2, dt=f32), xs_scales=xsc)
    off, cnt = torch.zeros(5, dtype=i32, device="cuda:0"), torch.zeros(4, dtype=i32, device="cuda:0")
    ar.ar_expert_dispatch(new(0, 256), new(0, 2, dt=i32), off, cnt, xs, x_scales=new(0, 2, dt=f32), xs_scales=xsc)
    # tokens whose slots all went elsewhere, and no row for any of them
    ar.ar_expert_dispatch(new(3, 256), torch.full((3, 2), -1, dtype=i32, device="cuda:0"), None, None, new(0, 256),
                          x_scales=new(3, 2, dt=f32), xs_scales=new(0, 2, dt=f32))
    torch.cuda.synchronize()
    assert bool((xs == 3).all()) and bool((xsc == 3).all())


def test_workspace_of_the_most_rows():
    """The gradient's workspace stops growing: no more for the most rows that a call can name than for many."""
    for hidden in (1, 100, 256, 4096, 16384, 32768):
        many = ar.ar_allreduce_rmsnorm_bwd_workspace_size(1 << 40, hidden)
        for rows in (2 ** 63 - 1, 2 ** 63 - 2, 2 ** 63 - 40, 2 ** 62):
            assert ar.ar_allreduce_rmsnorm_bwd_workspace_size(rows, hidden) == many
        with pytest.raises(ar.ArError):
            ar.ar_allreduce_rmsnorm_bwd_workspace_size(2 ** 63, hidden)
