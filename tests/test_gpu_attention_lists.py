"""Attention over lists of many unlike entries: how the work is cut between
workgroups, and what a captured call reads again at each replay."""
import pytest
import torch

import trellis_coded_quantized_amd as tq
from tests.test_gpu_attention import (BF16, FP16, Case, random_tree, run_tree, run_window, signed, tree_sees,
                                      window_sees)

pytestmark = pytest.mark.gpu


def unlike(entries, most, longest, seed):
    """Counts and contexts with empty, single and full entries in any order."""
    g = torch.Generator().manual_seed(seed)
    ns = torch.randint(0, most + 1, (entries,), generator=g).tolist()
    ctxs = torch.randint(0, longest + 1, (entries,), generator=g).tolist()
    ns[0], ns[-1], ns[entries // 2] = 0, most, 1
    ctxs[0], ctxs[-1], ctxs[entries // 3] = longest, 0, longest
    return ctxs, ns


# The last four have many entries for the workgroups of a key head
@pytest.mark.parametrize("entries,most,longest,hq,hkv,D,P,dtype", [
    (3, 64, 1500, 16, 1, 64, 16, BF16), (3, 64, 1500, 12, 2, 128, 32, FP16), (3, 64, 1500, 12, 2, 256, 16, BF16),
    (40, 9, 700, 16, 16, 128, 16, BF16), (40, 64, 300, 32, 16, 64, 16, FP16), (30, 40, 300, 32, 16, 256, 16, BF16),
    (130, 5, 600, 32, 4, 128, 64, BF16)])
def test_trees_of_unlike_entries(entries, most, longest, hq, hkv, D, P, dtype):
    ctxs, ns = unlike(entries, most, longest, D + entries)
    c = Case(ctxs, ns, hq, hkv, D, P, dtype, seed=D)
    masks = [m for n in ns for m in random_tree(n, c.g)]
    c.check(run_tree(c, masks), tree_sees(c, masks), D ** -0.5)


@pytest.mark.parametrize("entries,most,longest,hq,hkv,D,P,dtype", [
    (3, 400, 900, 8, 1, 64, 16, FP16), (3, 400, 900, 12, 2, 128, 64, BF16), (3, 300, 900, 12, 2, 256, 16, FP16),
    (40, 6, 700, 16, 16, 64, 32, BF16), (70, 80, 200, 8, 2, 128, 16, BF16), (70, 60, 200, 12, 2, 256, 16, BF16),
    (130, 50, 150, 4, 2, 64, 16, FP16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
def test_windows_of_unlike_entries(entries, most, longest, hq, hkv, D, P, dtype, window, sinks):
    ctxs, ns = unlike(entries, most, longest, D + entries)
    c = Case(ctxs, ns, hq, hkv, D, P, dtype, seed=D)
    c.check(run_window(c, window, sinks), window_sees(c, window, sinks), D ** -0.5)


def test_no_entry_has_a_token():
    c = Case([5, 6], [0, 0], 4, 2, 64, 16, BF16, extra_pages=4)
    q = c.to_device()
    assert tq.window_attention(q, *c.args, 3).shape == (0, 4, 64)
    assert tq.tree_attention(q, *c.args, signed([]), 3).shape == (0, 4, 64)


@pytest.mark.parametrize("n,D", [(3, 128), (50, 128), (40, 256)])
def test_tree_in_a_graph_reads_lengths_and_masks_again(n, D):
    c = Case([600, 90, 0], [n, n, n], 8, 2, D, 16, BF16)
    masks = [m for _ in range(3) for m in random_tree(n, c.g)]
    q = c.to_device()
    bits, out = signed(masks), torch.empty_like(q)
    tq.tree_attention(q, *c.args, bits, n, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.tree_attention(q, *c.args, bits, n, out=out)
    for rep in range(4):
        out.zero_()
        c.args[3][0] = 600 - 133 * rep
        bits[rep::4] &= ~1
        eager = tq.tree_attention(q, *c.args, bits, n)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16)), rep
