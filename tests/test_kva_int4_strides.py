"""The calls on a cache held in 4 bits agree on the strides they take: positive
ones of pages, planes and heads, any of layers (no device needed)."""
import pytest

from test_kva_int4_abi import (CALLS, CODES, INVAL, OK, SCALES, cache, group_scales,
                               swapped)

# places of pages, planes and heads among the strides of codes and of scales
PLACES = [("num_pages", 0, 0), (None, 1, 1), ("num_heads", 4, 3)]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("name,codes,scales", PLACES)
@pytest.mark.parametrize("sign", [0, -1])
def test_strides_that_are_not_positive(call, name, codes, scales, sign):
    """A place in a page of a negative stride would pass for no page."""
    assert call(cache(strides=swapped(CODES, codes, sign * CODES[codes])), group_scales()) == INVAL
    assert call(cache(), group_scales(
        strides=swapped(SCALES, scales, sign * SCALES[scales]))) == INVAL
    if name:  # of one index no stride is used
        assert call(cache(**{name: 1, "strides": swapped(CODES, codes, sign * CODES[codes])}),
                    group_scales(strides=swapped(SCALES, scales, sign * SCALES[scales]))) == OK


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("sign", [0, -1])
def test_layers_may_lie_in_any_order(call, sign):
    assert call(cache(strides=swapped(CODES, 2, sign * CODES[2])),
                group_scales(strides=swapped(SCALES, 2, sign * SCALES[2]))) == OK
