"""NaN among the scores that a row sees: it reaches the row's outputs however
the keys are cut, and nobody else's."""
import pytest
import torch

import trellis_coded_quantized_amd as tq
from tests.test_gpu_attention import BF16, FP16, Case, random_tree, signed, tree_sees, window_sees

pytestmark = pytest.mark.gpu

NAN = float("nan")


def both(c, scale, windows=((0, 0), (300, 5))):
    q = c.to_device()
    n = max(c.ns)
    for window, sinks in windows:
        got = tq.window_attention(q, *c.args, n, window=window, sinks=sinks)
        c.check(got, window_sees(c, window, sinks), scale, f"window {window}")
    if n <= 64:
        masks = [m for x in c.ns for m in random_tree(x, c.g)]
        c.check(tq.tree_attention(q, *c.args, signed(masks), n), tree_sees(c, masks), scale, "tree")


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, FP16), (256, BF16)])
@pytest.mark.parametrize("ctx", [0, 5, 100, 1000, 9001])
@pytest.mark.parametrize("n", [1, 4, 50])
def test_a_query_of_nan(n, ctx, D, dtype):
    c = Case([ctx, 70], [n, n], 8, 2, D, 16, dtype, seed=ctx)
    c.q[n // 2, 3, 7] = NAN
    both(c, D ** -0.5)


@pytest.mark.parametrize("D,dtype", [(64, FP16), (128, BF16), (256, BF16)])
@pytest.mark.parametrize("first,last", [
    (0, 9001), (0, 512), (1024, 1152), (0, 600), (2000, 2100), (8000, 9002), (9001, 9002)])
@pytest.mark.parametrize("n", [1, 40])
def test_runs_of_keys_of_nan(n, first, last, D, dtype):
    """From one key to whole parts (128 keys) and nothing else, and all of them."""
    c = Case([9001, 70], [n, n], 8, 2, D, 16, dtype, seed=first)
    c.keys[0][first:last, 0, 5] = NAN                              # of one key head
    both(c, D ** -0.5)


@pytest.mark.parametrize("n", [1, 40])
def test_a_row_of_nan_scores_beside_rows_that_see_nothing(n):
    c = Case([0, 3000], [n, n], 4, 1, 64, 16, BF16)
    c.q[n:] = NAN
    q = c.to_device()
    got = tq.tree_attention(q, *c.args, signed([0] * n + [1] * n), n)
    assert not got[:n].any()
    assert got[n:].isnan().all()
