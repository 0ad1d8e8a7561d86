"""Sizes whose products pass 64 bits are refused like other large ones (no GPU,
no launches)."""
import ctypes

import pytest

import trellis_coded_quantized_amd as tq
from tests.test_abi_attention import FAKE, cache, rope, said, state, tree, window


# 2^56 pages of 256, 2^60 of 16: products of 2^64, which is 0 in 64 bits; 2^55 of 256: the sign bit
@pytest.mark.parametrize("pages,page_size", [
    (1 << 56, 256), (1 << 60, 16), (1 << 55, 256), (1 << 62, 64), ((1 << 63) - 1, 16), ((1 << 56) + 1, 256)])
def test_pools_whose_slots_pass_64_bits(pages, page_size):
    c = cache(pages=pages, page_size=page_size)
    for call in (window, tree, rope):
        assert call(c=c) == tq.EINVAL
        said("pages=")
    lib, s = tq.load_library(), state()
    assert lib.trellis_cache_reserve_workspace_bytes(ctypes.byref(c), ctypes.byref(s), 1) == 0
    assert lib.trellis_cache_free(ctypes.byref(c), ctypes.byref(s), FAKE, 1, None) == tq.EINVAL
    said("pages=")


@pytest.mark.parametrize("seqs,width", [(8, 1 << 60), (8, (1 << 63) - 1), (1 << 62, 4), (1 << 31, 4), (8, 1 << 31)])
def test_tables_that_pass_32_bits(seqs, width):
    s = state(seqs=seqs, width=width)
    for call in (window, tree):
        assert call(s=s) == tq.EINVAL
        said("table of")
