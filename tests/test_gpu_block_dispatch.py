"""Dispatch on both sides of the row size from which positions are read before the row, with up to eight choices and more,
with and without scales."""
import pytest
import torch

import all_reduce_reduction_ring_amd as ar
import block_ref as ref
from test_gpu_block import DEV, F32, Guarded, gen, make_ids, randn, run_sort

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [1, 8, 9, 17])
@pytest.mark.parametrize("row", [513, 1024, 4095, 4096, 4097, 8191, 8192, 8193, 8208, 16385, 20000])
def test_rows(row, k):
    tokens, experts = 70, 32
    off, cnt, pos, src = run_sort(make_ids(tokens, k, experts, "some"), experts, 16)
    g, put, rows, nb = gen(4), Guarded(3), src.numel(), ref.blocks(row)
    x = put.new((tokens, row), torch.uint8, torch.randint(0, 256, (tokens, row), generator=g, device=DEV))
    sc, xs, xss = put.new((tokens, nb), F32, randn(g, tokens, nb)), put.new((rows, row), torch.uint8), put.new((rows, nb), F32)
    xs.fill_(0x33)
    ar.ar_expert_dispatch(x, pos, off, cnt, xs, sc, xss)
    torch.cuda.synchronize()
    put.check()
    end = off[-1].item()
    there, token = (src[:end] >= 0)[:, None], src[:end].clamp(min=0).long() // k
    assert torch.equal(xs[:end], torch.where(there, x[token], 0).to(torch.uint8)) and bool((xs[end:] == 0x33).all())
    assert torch.equal(xss[:end], torch.where(there, sc[token], 0.0))
