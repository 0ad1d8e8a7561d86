"""What a workspace holds before a call does not matter: every note and part
that the fold reads is written by the call itself."""
import pytest
import torch

import trellis_coded_quantized_amd as tq
from tests.test_gpu_attention import BF16, FP16, Case, random_tree, signed, tree_sees, window_sees
from tests.test_gpu_attention_lists import unlike

pytestmark = pytest.mark.gpu


# runs that end with the list, runs past its end, runs that begin in the middle of a unit
@pytest.mark.parametrize("entries,most,longest,hq,hkv,D,P,dtype", [
    (1, 1, 0, 8, 2, 64, 16, BF16), (1, 300, 40, 8, 1, 64, 16, FP16), (3, 400, 900, 12, 2, 128, 64, BF16),
    (2, 64, 3000, 12, 2, 256, 16, BF16), (70, 60, 200, 12, 2, 256, 16, FP16), (130, 50, 150, 4, 2, 64, 16, BF16),
    (90, 2, 2000, 8, 8, 128, 16, FP16)])
@pytest.mark.parametrize("filled", [0x00, 0x01, 0x5A, 0xFF])
def test_workspaces_of_any_content(entries, most, longest, hq, hkv, D, P, dtype, filled):
    ctxs, ns = unlike(entries, most, longest, D) if entries > 1 else ([longest], [most])
    c = Case(ctxs, ns, hq, hkv, D, P, dtype, seed=entries)
    q = c.to_device()
    workspace = torch.full((1 << 28,), filled, dtype=torch.uint8, device=q.device)
    got = tq.window_attention(q, *c.args, max(ns), window=300, sinks=3, workspace=workspace)
    c.check(got, window_sees(c, 300, 3), D ** -0.5, "window")
    if max(ns) <= 64:
        masks = [m for n in ns for m in random_tree(n, c.g)]
        workspace.fill_(filled)
        c.check(tq.tree_attention(q, *c.args, signed(masks), max(ns), workspace=workspace), tree_sees(c, masks),
                D ** -0.5, "tree")
