"""max_q is a bound, not a size: it chooses kernels and workspaces, never
results beyond rounding; and a call stays inside the workspace it asked for."""
import ctypes

import pytest
import torch

import trellis_coded_quantized_amd as tq
from tests.test_gpu_attention import (BF16, FP16, Case, random_tree, run_tree, run_window, signed, tree_sees,
                                      window_sees)

pytestmark = pytest.mark.gpu


# with 4 query heads a key head: 32 rows, 128 rows and more
@pytest.mark.parametrize("max_q", [7, 8, 9, 32, 33, 64, 700])
@pytest.mark.parametrize("D,P,dtype", [(64, 16, FP16), (128, 64, BF16), (256, 16, BF16)])
def test_max_q_is_only_a_bound(max_q, D, P, dtype):
    c = Case([333, 0, 90], [7, 3, 0], 8, 2, D, P, dtype, seed=max_q)
    c.check(run_window(c, 200, 3, max_q=max_q), window_sees(c, 200, 3), D ** -0.5)
    if max_q <= 64:
        masks = [m for n in c.ns for m in random_tree(n, c.g)]
        c.check(run_tree(c, masks, max_q=max_q), tree_sees(c, masks), D ** -0.5)


@pytest.mark.parametrize("entries,n,ctx,hq,hkv,D", [
    (1, 1, 5000, 8, 2, 128), (3, 8, 2500, 8, 2, 64), (2, 20, 3000, 8, 2, 128), (70, 9, 300, 16, 16, 64),
    (2, 64, 2000, 12, 2, 256), (1, 64, 3000, 16, 1, 128), (40, 40, 200, 16, 16, 256)])
def test_the_workspace_is_not_left(entries, n, ctx, hq, hkv, D):
    ctxs = [ctx - 13 * e if ctx > 13 * e else 0 for e in range(entries)]
    c = Case(ctxs, [n] * entries, hq, hkv, D, 16, BF16, seed=entries)
    masks = [m for _ in range(entries) for m in random_tree(n, c.g)]
    q = c.to_device()
    k, v, table, lengths, _ = c.args
    cache, index = tq._kv_cache(k, v, False)
    state = tq._kv_state(table, lengths, None, cache.pages, index)
    lib, shapes = tq.load_library(), (entries, q.shape[0], hq, n)
    by = ctypes.byref
    sizes = (lib.trellis_tree_attention_workspace_bytes(by(cache), by(state), *shapes),
             lib.trellis_window_attention_workspace_bytes(by(cache), by(state), *shapes, 0, 0))
    for size, call in zip(sizes, (
            lambda ws: tq.tree_attention(q, *c.args, signed(masks), n, workspace=ws),
            lambda ws: tq.window_attention(q, *c.args, n, workspace=ws))):
        buffer = torch.full((size + (1 << 20),), 0x5A, dtype=torch.uint8, device=q.device)
        want = call(None)
        got = call(buffer[:size])
        assert (buffer[size:] == 0x5A).all()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        with pytest.raises(tq.TrellisError, match="workspace"):
            call(buffer[:size - 1])
