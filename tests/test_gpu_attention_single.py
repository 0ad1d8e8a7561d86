"""One entry by itself: its keys are cut without a search for the chunk, by a
condition that has to be the same for all lanes of a wave."""
import pytest
import torch

import trellis_coded_quantized_amd as tq
from tests.test_gpu_attention import BF16, FP16, Case, random_tree, signed, tree_sees, window_sees

pytestmark = pytest.mark.gpu


# contexts around one chunk of 128 keys, around as many chunks as there are workgroups a head, and past it;
# rows of one tile (few and many) and of several
@pytest.mark.parametrize("ctx", [0, 127, 128, 129, 4095, 4097, 16383, 16500, 33000])
@pytest.mark.parametrize("n,hq,hkv,D,dtype", [(1, 8, 8, 64, BF16), (3, 8, 2, 128, FP16), (20, 8, 2, 64, BF16),
                                              (64, 12, 2, 256, BF16)])
def test_single_entries(ctx, n, hq, hkv, D, dtype):
    c = Case([ctx], [n], hq, hkv, D, 64, dtype, seed=ctx)
    masks = random_tree(n, c.g)
    q = c.to_device()
    c.check(tq.tree_attention(q, *c.args, signed(masks), n), tree_sees(c, masks), D ** -0.5, "tree")
    c.check(tq.window_attention(q, *c.args, n), window_sees(c, 0, 0), D ** -0.5, "window")


def test_a_single_entry_without_tokens_or_sequence():
    c = Case([40], [2], 4, 2, 64, 16, BF16)
    q = c.to_device()
    out = torch.full_like(q, 3.0)
    gone = torch.tensor([5], dtype=torch.int32, device=q.device)
    tq.tree_attention(q, *c.args, signed([1, 3]), 2, seq_ids=gone, out=out)
    none = torch.zeros(2, dtype=torch.int32, device=q.device)
    tq.tree_attention(q, *c.args[:4], none, signed([1, 3]), 2, out=out)
    assert (out == 3.0).all()
