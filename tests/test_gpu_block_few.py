"""Sorts of few slots on both sides of the sizes up to which a small workgroup does them."""
import numpy as np
import pytest

import block_ref as ref
from test_gpu_block import make_ids, run_sort

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("align", [1, 16])
@pytest.mark.parametrize("experts", [1, 2, 100, 128, 129, 255, 256, 257, 1000])
@pytest.mark.parametrize("tokens,k", [(1, 1), (64, 1), (255, 1), (256, 2), (511, 1), (512, 1), (513, 1), (171, 3)])
def test_expert_sort(tokens, k, experts, align):
    ids = make_ids(tokens, k, experts, "some" if tokens > 1 else "even")
    off, cnt, pos, src = run_sort(ids, experts, align, extra=3)
    offsets, counts, p, s = ref.sort(ids.cpu(), experts, align)
    assert off.tolist() == offsets and cnt.tolist() == counts and pos.reshape(-1).tolist() == p
    want = np.full(src.numel(), -1, np.int32)
    want[np.fromiter(s.keys(), int, len(s))] = np.fromiter(s.values(), np.int32, len(s))
    np.testing.assert_array_equal(src.cpu().numpy(), want)
