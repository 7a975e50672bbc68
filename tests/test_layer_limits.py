"""Sizes next to 2^31 and past it in the calls around the experts.  Nothing here runs a kernel: the calls
are refused."""
import pytest

from test_layer_abi import PA, PB, UNSUP, back, combine, dispatch

MOST = 2 ** 31 - 64          # the last count that a 32-bit number walks 64 at a time


@pytest.mark.parametrize("count", [MOST + 1, 2 ** 31 - 1])
def test_counts_that_a_32_bit_walk_would_pass_are_unsupported(count):
    assert combine(tokens=1, top=count, ldw=count) == UNSUP
    assert combine(tokens=1, top=count, w=0, ldw=0) == UNSUP
    assert back(tokens=1, top=count, ldw=count, lddw=count) == UNSUP
    assert back(tokens=1, top=count, ldw=count, dw=0, lddw=0) == UNSUP
    assert dispatch(tokens=1, top=count) == UNSUP
    assert dispatch(tokens=1, top=1, cols=count, s=PA, lds=count, t=PB, ldt=count) == UNSUP
    assert dispatch(tokens=0, top=1, cols=count, s=PA, lds=count, t=PB, ldt=count) == UNSUP
