"""The 64-bit references of the block-boundary operators: gradients against central differences, and a planted mistake
that the differences show."""
import pytest
import torch

import block_ref as ref


def _diff(f, x, v, h=1e-5):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


@pytest.mark.parametrize("residual", [False, True])
def test_norm_gradient_matches_differences(residual):
    g = torch.Generator().manual_seed(3)
    mk = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x, res, gamma, dy, dres = mk(5, 37), mk(5, 37), mk(37), mk(5, 37), mk(5, 37)
    use = res if residual else None

    def loss(x_, gamma_):
        h, _, y, *_ = ref.norm([x_], use, gamma_, 1e-3)
        return float((y * dy).sum() + ((h * dres).sum() if residual else 0.0))

    h, rstd, *_ = ref.norm([x], use, gamma, 1e-3)
    dx, dgamma, _, _ = ref.norm_bwd([dy], h, gamma, rstd[:, 0], dres if residual else None, 5)
    for _ in range(4):
        v, w = mk(5, 37), mk(37)
        assert _diff(lambda a: loss(a, gamma), x, v) == pytest.approx(float((dx * v).sum()), rel=1e-7, abs=1e-8)
        assert _diff(lambda a: loss(x, a), gamma, w) == pytest.approx(float((dgamma * w).sum()), rel=1e-7, abs=1e-8)
        # without the term through the statistics the differences disagree
        wrong = rstd * dy * gamma + (dres if residual else 0.0)
        assert abs(_diff(lambda a: loss(a, gamma), x, v) - float((wrong * v).sum())) > 1e-3


def test_combine_gradient_matches_differences():
    g = torch.Generator().manual_seed(4)
    mk = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    ids = torch.tensor([[0, 2], [2, -1], [1, 0], [-1, -1]], dtype=torch.int32)
    _, _, pos, _ = ref.sort(ids, 3, 2)
    pos = torch.tensor(pos).view(4, 2)
    ys, w, dout = mk(8, 11), mk(4, 2), mk(4, 11)
    loss = lambda a, b: float((ref.combine(a, pos, b, None)[0] * dout).sum())
    dys, dw, _ = ref.combine_bwd(dout, ys, pos, w, 8)
    for _ in range(4):
        v, x = mk(8, 11), mk(4, 2)
        assert _diff(lambda a: loss(a, w), ys, v) == pytest.approx(float((dys * v).sum()), rel=1e-7, abs=1e-8)
        assert _diff(lambda a: loss(ys, a), w, x) == pytest.approx(float((dw * x).sum()), rel=1e-7, abs=1e-8)
    # dispatch's gradient: the rows of ones-weighted combine
    x = mk(4, 11)
    there = pos >= 0
    xs = torch.zeros(8, 11, dtype=torch.float64)
    xs[pos[there]] = x[torch.arange(4)[:, None].expand(4, 2)[there]]
    dxs = mk(8, 11)
    assert float((xs * dxs).sum()) == pytest.approx(float((ref.combine(dxs, pos, None, None)[0] * x).sum()), rel=1e-12)


def test_sort_by_hand():
    ids = torch.tensor([[2, 0], [0, 7], [2, 2], [-1, 0]], dtype=torch.int32)
    offsets, counts, pos, src = ref.sort(ids, 3, 2)
    assert offsets == [0, 4, 4, 8] and counts == [3, 0, 3]
    assert pos == [4, 0, 1, -1, 5, 6, -1, 2] and src == {0: 1, 1: 2, 2: 7, 4: 0, 5: 4, 6: 5}
