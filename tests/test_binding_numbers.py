"""Numbers past 32 bits are refused by the binding: as C ints they would become
other numbers (a window of 2^32 + 100 one of 100)."""
import ctypes

import pytest

import trellis_coded_quantized_amd as tq

PAST = [2 ** 31, 2 ** 32, 2 ** 32 + 100, 2 ** 63 - 1, 2 ** 64 + 16, -2 ** 31 - 1, -2 ** 32 + 100]


def test_what_ctypes_does_with_them():
    assert [ctypes.c_int(v).value for v in (2 ** 32 + 100, -2 ** 32 + 100, 2 ** 64 + 16)] == [100, 100, 16]


@pytest.mark.parametrize("value", PAST)
@pytest.mark.parametrize("name", ["max_q", "window", "sinks"])
def test_window_attention(name, value):
    with pytest.raises(ValueError, match=name):
        tq.window_attention(*[None] * 6, **{"max_q": 1, name: value})


@pytest.mark.parametrize("value", PAST)
def test_tree_attention(value):
    with pytest.raises(ValueError, match="max_q"):
        tq.tree_attention(*[None] * 7, value)


@pytest.mark.parametrize("value", PAST)
def test_cache_reserve(value):
    with pytest.raises(ValueError, match="page_size"):
        tq.cache_reserve(None, None, None, value, None, None, 1)


def test_numbers_of_32_bits_reach_the_library():
    for v in (-2 ** 31, -1, 0, 2 ** 31 - 1):
        assert tq._c_int(v, "v") == v
