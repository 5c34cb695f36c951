"""Limits of the expert entry points that no small tensor reaches, by the library's own checks with addresses that no call
reads: rows of 2^31 bytes are refused, the widest below are not (they fail later, on overlapping buffers)."""
import pytest

import all_reduce_reduction_ring_amd as ar

BASE, FAR = 1 << 40, 1 << 44


def _dispatch(hidden, es, xs=FAR):
    return ar.lib().ar_expert_dispatch(BASE, None, FAR * 2, None, None, 1, 1, 1, hidden, es, xs, None, 1, None)


def _combine(hidden, dtype, out=FAR):
    return ar.lib().ar_expert_combine(BASE, FAR * 2, None, None, 1, 1, hidden, dtype, 1, out, None)


def _combine_bwd(hidden, dtype, dys=FAR):
    return ar.lib().ar_expert_combine_bwd(BASE, FAR * 3, FAR * 2, FAR * 2 + 4096, None, None, 1, 1, 1, hidden, dtype, 1, dys,
                                          FAR * 4, None)


@pytest.mark.parametrize("es,dtype", [(4, ar.AR_F32), (2, ar.AR_BF16), (2, ar.AR_F16)])
def test_rows_of_two_gibibytes(es, dtype):
    most = (2 ** 31 - 1) // es
    assert _dispatch(most + 1, es) == ar.AR_ERR_UNSUPPORTED and _dispatch(most, es, xs=BASE) == ar.AR_ERR_ALIAS
    assert _combine(most + 1, dtype) == ar.AR_ERR_UNSUPPORTED and _combine(most, dtype, out=BASE) == ar.AR_ERR_ALIAS
    assert _combine_bwd(most + 1, dtype) == ar.AR_ERR_UNSUPPORTED
    assert _combine_bwd(most, dtype, dys=BASE) == ar.AR_ERR_ALIAS


def test_rows_of_two_gibibytes_of_codes():
    assert _dispatch(2 ** 31, 1) == ar.AR_ERR_UNSUPPORTED and _dispatch(2 ** 31 - 1, 1, xs=BASE) == ar.AR_ERR_ALIAS
