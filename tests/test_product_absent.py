"""Weights and gradients of weights that a call leaves out need no distance between their matrices: what is NULL is neither
read nor checked. Every call has an alias planted in it, so that it gets as far as the last check and nothing is launched."""
import pytest

import all_reduce_reduction_ring_amd as ar
import test_product_abi as abi

at = abi.at
ONLY_ROWS = dict(xs=None, dw=None, dxs=at(0))
ONLY_WEIGHTS = dict(w=None, dxs=None, dw=at(1))


@pytest.mark.parametrize("stride", [0, 1, 1 << 63, (1 << 64) - 1])
def test_distances_of_absent_weights(stride):
    assert abi._linear_bwd(**ONLY_ROWS, dstride=stride) == ar.AR_ERR_ALIAS
    assert abi._linear_bwd(**ONLY_WEIGHTS, stride=stride) == ar.AR_ERR_ALIAS
    assert abi._gated_bwd(dwg=None, dwu=None, dstride=stride, dxs=at(8)) == ar.AR_ERR_ALIAS
    assert abi._gated_bwd(dwg=None, dwu=None, xs=None, dstride=stride, dxs=at(8)) == ar.AR_ERR_ALIAS
    assert abi._gated_bwd(dxs=None, wg=None, wu=None, stride=stride, dwg=at(3)) == ar.AR_ERR_ALIAS
    # the gradients of the two products alone
    assert abi._gated_bwd(dxs=None, wg=None, wu=None, stride=stride, xs=None, dwg=None, dwu=None, dstride=stride,
                          dgate=at(9)) == ar.AR_ERR_ALIAS


@pytest.mark.parametrize("stride", [0, 64 * 128 - 1, 1 << 62])
def test_distances_of_given_weights_are_checked(stride):
    assert abi._linear_bwd(dxs=at(0), stride=stride) == ar.AR_ERR_INVALID
    assert abi._linear_bwd(dxs=at(0), dstride=stride) == ar.AR_ERR_INVALID
    assert abi._linear_bwd(dxs=None, dw=at(1), stride=stride) == ar.AR_ERR_INVALID  # given, though not read
    assert abi._gated_bwd(dxs=at(8), stride=stride) == ar.AR_ERR_INVALID
    assert abi._gated_bwd(dxs=at(8), dstride=stride) == ar.AR_ERR_INVALID
    assert abi._gated_bwd(dxs=None, dwg=at(3), wg=None, stride=stride) == ar.AR_ERR_INVALID
