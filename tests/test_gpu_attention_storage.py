"""Attention and the storage behind a table: tables that end inside a tile,
keys whose page is not there."""
import pytest
import torch

import trellis_coded_quantized_amd as tq
from tests.test_gpu_attention import BF16, DEV, FP16, Case, random_tree, signed, tree_sees, window_sees

pytestmark = pytest.mark.gpu


def full_table(n, width, P, D, dtype, seed):
    """One sequence that fills its table, which is the end of an array with page numbers of nothing behind it.
    Infinities and NaN in the last tile, seen by the last token only."""
    c = Case([width * P - n], [n], 8, 2, D, P, dtype, seed=seed, pad=0)
    c.vals[0][-1, 0, 3], c.vals[0][-1, 1, D - 1] = float("inf"), float("nan")
    q = c.to_device()
    assert c.args[2].shape == (1, width)
    longer = torch.full((width + 64,), 2 ** 31 - 1, dtype=torch.int32, device=DEV)
    longer[:width] = c.args[2][0]
    table = longer[:width].view(1, width)
    return c, q, c.args[:2] + (table,) + c.args[3:]


@pytest.mark.parametrize("n,width,P", [(2, 3, 16), (1, 1, 16), (3, 5, 32), (40, 5, 16), (40, 6, 16), (40, 7, 16), (33, 3, 32)])
@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, FP16), (256, BF16)])
def test_tables_that_end_inside_a_tile(n, width, P, D, dtype):
    c, q, args = full_table(n, width, P, D, dtype, seed=n + width)
    for window, sinks in ((0, 0), (20, 3)):
        got = tq.window_attention(q, *args, n, window=window, sinks=sinks)
        c.check(got, window_sees(c, window, sinks), D ** -0.5, f"window {window}")
    masks = random_tree(n, c.g)
    c.check(tq.tree_attention(q, *args, signed(masks), n), tree_sees(c, masks), D ** -0.5, "tree")
