"""Numbers past the C types of the block-boundary entry points are refused; ctypes would cut them to their low bits."""
import pytest
import torch

import all_reduce_reduction_ring_amd as ar

BIG = 1 << 32


def test_sizes():
    calls = [lambda: ar.ar_expert_rows(10, 2, 4, BIG + 1), lambda: ar.ar_expert_rows(10, BIG + 2, 4),
             lambda: ar.ar_expert_rows(10, 2, BIG + 4), lambda: ar.ar_expert_rows((1 << 64) + 10, 2, 4),
             lambda: ar.ar_expert_rows(-1, 2, 4), lambda: ar.ar_expert_sort_workspace_size(10_000, BIG + 2, 4),
             lambda: ar.ar_expert_sort_workspace_size(10_000, 2, BIG + 4),
             lambda: ar.ar_expert_sort_workspace_size((1 << 64) + 10_000, 2, 4),
             lambda: ar.ar_allreduce_rmsnorm_bwd_workspace_size((1 << 64) + 4, 256),
             lambda: ar.ar_allreduce_rmsnorm_bwd_workspace_size(4, (1 << 64) + 256)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(ar.ArError):  # in range, refused by the library
        ar.ar_expert_rows(10, 2, 4, -1)
    assert ar.ar_expert_rows(1, 1, 1, 2 ** 31 - 1) == 2 ** 31 - 1


@pytest.mark.gpu
def test_align():
    new = lambda *s: torch.full(s, 5, dtype=torch.int32, device="cuda:0")
    ids, off, cnt, pos, src = new(3, 2), new(9), new(8), new(3, 2), new(6)
    for align in (BIG + 1, BIG * BIG + 1, 1 - BIG):
        with pytest.raises(ValueError, match="align"):
            ar.ar_expert_sort(ids, off, cnt, pos, src, align=align)
    torch.cuda.synchronize()
    assert all(bool((t == 5).all()) for t in (off, cnt, pos, src))
