"""tree_attention_kv8 and window_attention_kv8 against plain 64-bit attention
over what the codes and scales stand for.  Codes times scales are exact in both
16-bit types here, so the bounds are those of the 16-bit cache's tests."""
import pytest
import torch

import trellis_coded_quantized_amd as tq
from tests import kv_reference as ref
from tests.kv8_reference import E4M3, E8M0, Case8
from tests.test_gpu_attention import BF16, FP16, random_tree, signed, tree_sees, window_sees
from tests.test_gpu_attention_lists import unlike

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def run_tree(c, masks, max_q=None, scale=None, **kw):
    q = c.to_device()
    return tq.tree_attention_kv8(q, *c.args, signed(masks), max_q or max(c.ns), scale=scale, **kw)


def run_window(c, window, sinks, max_q=None, scale=None, **kw):
    q = c.to_device()
    return tq.window_attention_kv8(q, *c.args, max_q or max(c.ns), window=window, sinks=sinks, scale=scale, **kw)


def test_every_code_under_every_scale():
    """One key, one row: the output is the value itself, for all 256 codes and scales from 2^-126 up to where bf16 ends."""
    P, D = 16, 256
    for dt, bytes_ in ((BF16, list(range(1, 248)) + [254, 255]), (FP16, list(range(1, 160)))):
        n = len(bytes_)
        code = torch.arange(256, dtype=torch.uint8)
        k = torch.zeros((n, 1, D // 16, P, 16), dtype=torch.uint8, device=DEV)
        v = torch.full((n, 1, P // 16, D, 16), 0x7F, dtype=torch.uint8, device=DEV)
        v[:, 0, 0, :, 0] = code.to(DEV)
        ks = torch.full((n, 1, 1), 127, dtype=torch.uint8, device=DEV)
        vs = torch.tensor(bytes_, dtype=torch.uint8, device=DEV).view(n, 1, 1)
        table = torch.arange(n, dtype=torch.int32, device=DEV).view(n, 1)
        starts = torch.arange(n + 1, dtype=torch.int32, device=DEV)
        q = torch.ones((n, 1, D), dtype=dt, device=DEV)
        got = tq.window_attention_kv8(q, k.view(E4M3), v.view(E4M3), ks.view(E8M0), vs.view(E8M0), table,
                                      torch.zeros(n, dtype=torch.int32, device=DEV), starts, 1)[:, 0].cpu()
        scale = 2.0 ** (torch.tensor(bytes_, dtype=torch.float64) - 127)
        scale[torch.tensor(bytes_) == 255] = float("nan")
        # rounded to the 16-bit type, as documented (exact but below its normal numbers and past its end)
        want = (code.view(E4M3).double() * scale[:, None]).to(dt)
        same = (got == want) | (got.isnan() & want.isnan())
        # past the type's end there is no right value to compare with
        bad = ~same & torch.isfinite(want)
        assert not bad.any(), [(dt, bytes_[i], j) for i, j in bad.nonzero().tolist()[:5]]


@pytest.mark.parametrize("hq,hkv,D,P,dtype", [
    (24, 4, 256, 16, BF16), (32, 8, 128, 32, FP16), (16, 16, 64, 64, BF16), (8, 1, 128, 256, BF16),
    (6, 2, 64, 16, FP16), (5, 5, 256, 128, FP16)])
@pytest.mark.parametrize("ns", [[1, 1, 1, 1, 1], [4, 1, 3, 2, 4], [64, 1, 33, 0, 17]])
def test_tree(hq, hkv, D, P, dtype, ns):
    c = Case8([0, 1, 31, 100, 257], ns, hq, hkv, D, P, dtype, seed=D + P)
    masks = [m for n in ns for m in random_tree(n, c.g)]
    c.check(run_tree(c, masks), tree_sees(c, masks), D ** -0.5)


@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 1000])
@pytest.mark.parametrize("n,D", [(1, 128), (5, 64), (40, 128), (33, 256)])
def test_tree_lengths(ctx, n, D):
    c = Case8([ctx], [n], 8, 2, D, 16, BF16, seed=ctx)
    masks = random_tree(n, c.g)
    c.check(run_tree(c, masks), tree_sees(c, masks), D ** -0.5)


@pytest.mark.parametrize("n,hq", [(3, 4), (50, 4)])
def test_rows_that_see_nothing_are_zero(n, hq):
    c = Case8([0, 0, 20], [n, 2, 1], hq, 2, 128, 16, BF16)
    masks = [0] * n + [0, 2] + [0]
    got = run_tree(c, masks)
    assert not got[:n + 1].any()
    c.check(got, tree_sees(c, masks), 128 ** -0.5)


@pytest.mark.parametrize("n,D,P", [(4, 128, 16), (64, 64, 32), (40, 256, 16), (2, 64, 64)])
def test_nan_tokens_reach_only_rows_that_see_them(n, D, P):
    c = Case8([37], [n], 8, 2, D, P, BF16, seed=3)
    nan = float("nan")
    c.vals[0][38, 0, 3], c.vals[0][38, 1, D - 1] = nan, nan
    c.keys[0][38] = nan
    masks = [1 if i == 0 else 2 if i == 1 else (1 | 1 << i if i % 2 else 1 << i) for i in range(n)]
    sees = tree_sees(c, masks)
    got = run_tree(c, masks)
    hit = sees[0][:, 38]
    assert got[hit.to(DEV)].isnan().all()
    rest = [i for i in range(n) if not hit[i]]
    c.keys[0][38] = 0
    parts = ref.attend(c.q[rest], c.keys[0], c.vals[0], sees[0][rest], D ** -0.5)
    ref.assert_attention(got[rest], parts, 37 + n, D)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_nan_values_in_open_and_cut_tiles(D):
    for n, hq in ((1, 8), (1, 2), (30, 8), (40, 8)):
        c = Case8([200], [n], hq, 2, D, 16, FP16, seed=5)
        c.vals[0][10, 0, 1] = float("nan")           # seen by all
        c.vals[0][199, 1, 2] = float("nan")          # before a window's last rows
        c.vals[0][200 + n - 1, 0, 5] = float("nan")  # seen by the last token only
        for window, sinks in ((0, 0), (3, 0), (40, 12)):
            c.check(run_window(c, window, sinks), window_sees(c, window, sinks), D ** -0.5, f"n {n} window {window}")


@pytest.mark.parametrize("hq,hkv,D,P,dtype", [
    (24, 4, 256, 16, BF16), (32, 8, 128, 64, FP16), (16, 16, 64, 16, BF16), (3, 1, 64, 32, FP16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (7, 3), (32, 0), (65, 33), (100, 4), (100000, 4)])
def test_window(hq, hkv, D, P, dtype, window, sinks):
    c = Case8([0, 5, 300, 64, 129], [1, 2, 1, 0, 1], hq, hkv, D, P, dtype, seed=window)
    c.check(run_window(c, window, sinks), window_sees(c, window, sinks), D ** -0.5, "few")
    c = Case8([0, 5, 300, 64, 129], [70, 2, 129, 0, 33], hq, hkv, D, P, dtype, seed=window + 1)
    c.check(run_window(c, window, sinks), window_sees(c, window, sinks), D ** -0.5, "many")


@pytest.mark.parametrize("n", [1, 100])
def test_long_context_split_over_workgroups(n):
    c = Case8([9001, 40], [n, 1], 8, 2, 64, 16, BF16, seed=n)
    c.check(run_window(c, 0, 0), window_sees(c, 0, 0), 64 ** -0.5)


@pytest.mark.parametrize("entries,most,longest,hq,hkv,D,P,dtype", [
    (70, 60, 200, 12, 2, 256, 16, FP16), (130, 50, 150, 4, 2, 64, 16, BF16), (90, 2, 2000, 8, 8, 128, 16, FP16),
    (3, 400, 900, 12, 2, 128, 64, BF16), (2, 300, 500, 8, 1, 64, 32, BF16)])
@pytest.mark.parametrize("filled", [0x00, 0xFF])
def test_unlike_entries_and_workspaces_of_any_content(entries, most, longest, hq, hkv, D, P, dtype, filled):
    ctxs, ns = unlike(entries, most, longest, D)
    c = Case8(ctxs, ns, hq, hkv, D, P, dtype, seed=entries)
    workspace = torch.full((1 << 28,), filled, dtype=torch.uint8, device=DEV)
    c.check(run_window(c, 300, 3, workspace=workspace), window_sees(c, 300, 3), D ** -0.5, "window")
    if max(ns) <= 64:
        masks = [m for n in ns for m in random_tree(n, c.g)]
        workspace.fill_(filled)
        c.check(run_tree(c, masks, workspace=workspace), tree_sees(c, masks), D ** -0.5, "tree")


@pytest.mark.parametrize("n", [2, 60])
def test_sequence_numbers_row_strides_and_scale(n):
    c = Case8([50, 3, 90], [n, 1, n], 8, 2, 128, 16, BF16, seqs=6, ids=[4, 0, 2])
    q = c.to_device()
    wide = torch.full((q.shape[0], 8 + 3, 128), float("nan"), dtype=BF16, device=DEV)
    wide[:, 1:9] = q
    ids = torch.tensor(c.ids, dtype=torch.int32, device=DEV)
    got = tq.window_attention_kv8(wide[:, 1:9], *c.args, n, window=60, sinks=2, scale=0.3, seq_ids=ids)
    c.check(got, window_sees(c, 60, 2), 0.3)


@pytest.mark.parametrize("n", [1, 40])
def test_blocks_of_far_apart_scales(n):
    """Neighbouring blocks differ by up to 2^40 in keys and values; the loud ones decide."""
    c = Case8([500], [n], 4, 2, 64, 16, BF16, exponents=(85, 125))
    c.check(run_window(c, 0, 0), window_sees(c, 0, 0), 64 ** -0.5)


@pytest.mark.parametrize("n", [2, 40])
def test_bad_pages_lengths_and_sequences_stay_inside_the_arrays(n):
    c = Case8([60, 30, 20], [n, n, n], 4, 2, 64, 16, BF16, seqs=4, ids=[0, 1, 2])
    q = c.to_device()
    *pools, table, lengths, starts = c.args
    table[0, :] = torch.tensor([2 ** 31 - 1, -5] * 8, dtype=torch.int32, device=DEV)[:table.shape[1]]
    lengths[1] = 2 ** 31 - 1
    out = torch.zeros_like(q)
    ids = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    tq.window_attention_kv8(q, *pools, table, lengths, starts, n, seq_ids=ids, out=out)
    a, b = c.starts[2], c.starts[3]
    parts = ref.attend(c.q[a:b], c.keys[2], c.vals[2], window_sees(c, 0, 0)[2], 64 ** -0.5)
    ref.assert_attention(out[a:b], parts, 20 + n, 64)
    assert not out[:c.starts[1]].any()                         # no page of its own: nothing is seen
    bad = torch.tensor([9, -1, 2], dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 3.0)
    tq.window_attention_kv8(q, *pools, table, lengths, starts, n, seq_ids=bad, out=out)
    assert (out[:a] == 3.0).all()
    ref.assert_attention(out[a:b], parts, 20 + n, 64)


def test_rows_past_max_q_are_left_and_no_tokens():
    c = Case8([10], [6], 4, 2, 64, 16, BF16)
    q = c.to_device()
    out = torch.full_like(q, 2.0)
    tq.window_attention_kv8(q, *c.args, 4, out=out)
    assert (out[4:] == 2.0).all()
    parts = ref.attend(c.q[:4], c.keys[0][:14], c.vals[0][:14], ref.window_see(10, 4, 14, 0, 0), 64 ** -0.5)
    ref.assert_attention(out[:4], parts, 14, 64)
    q = torch.empty((0, 4, 64), dtype=BF16, device=DEV)
    assert tq.window_attention_kv8(q, *c.args, 1).shape == (0, 4, 64)


@pytest.mark.parametrize("n", [2, 40])
def test_offsets_past_32_bits(n):
    """Pages at the far end of a pool of more than 2^32 bytes."""
    P, D, hkv = 16, 128, 2
    pages = (1 << 32) // (P * D * hkv) + 50
    c = Case8([100], [n], 4, hkv, D, P, BF16)
    q = c.to_device()
    *small, table, lengths, starts = c.args
    held = small[0].shape[0]
    pools = []
    for s in small:
        pool = torch.empty((pages,) + s.shape[1:], dtype=torch.uint8, device=DEV)
        pool[-held:] = s.view(torch.uint8)
        pools.append(pool.view(s.dtype))
    table = torch.where(table >= 0, table + (pages - held), table).int()
    got = tq.window_attention_kv8(q, *pools, table, lengths, starts, n)
    c.check(got, window_sees(c, 0, 0), D ** -0.5)


@pytest.mark.parametrize("n", [1, 60])
def test_same_bits_on_another_stream_and_in_a_graph(n):
    c = Case8([700, 90], [n, n], 8, 2, 128, 16, BF16)
    q = c.to_device()
    want = tq.window_attention_kv8(q, *c.args, n, window=500, sinks=4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = tq.window_attention_kv8(q, *c.args, n, window=500, sinks=4)
    side.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.window_attention_kv8(q, *c.args, n, window=500, sinks=4, out=out)
    lengths = c.args[5]
    for rep in range(4):
        out.zero_()
        lengths[1] = 90 - 7 * rep
        eager = tq.window_attention_kv8(q, *c.args, n, window=500, sinks=4)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16)), rep


def test_refusals():
    c = Case8([10], [2], 4, 2, 64, 16, BF16)
    q = c.to_device()
    k, v, ks, vs, table, lengths, starts = c.args
    with pytest.raises(TypeError, match="q: dtype"):
        tq.window_attention_kv8(q.float(), *c.args, 2)
    with pytest.raises(TypeError, match="k_cache: dtype"):
        tq.window_attention_kv8(q, k.view(torch.uint8), v, ks, vs, table, lengths, starts, 2)
    with pytest.raises(TypeError, match="v_scale: dtype"):
        tq.window_attention_kv8(q, k, v, ks, vs.view(torch.uint8), table, lengths, starts, 2)
    with pytest.raises(ValueError, match="v_cache: shape"):
        tq.window_attention_kv8(q, k, v[:, :1].contiguous(), ks, vs, table, lengths, starts, 2)
    with pytest.raises(ValueError, match="k_scale: shape"):
        tq.window_attention_kv8(q, k, v, ks[:-1], vs, table, lengths, starts, 2)
    with pytest.raises(ValueError, match="one layer"):
        tq.window_attention_kv8(q, k[None], v[None], ks[None], vs[None], table, lengths, starts, 2)
    with pytest.raises(tq.TrellisError, match="multiple of the cache's"):
        tq.window_attention_kv8(q[:, :3].contiguous(), *c.args, 2)
    with pytest.raises(tq.TrellisError, match="max_q"):
        tq.tree_attention_kv8(q, *c.args, signed([1, 3]), 65)
    with pytest.raises(ValueError, match="ancestors"):
        tq.tree_attention_kv8(q, *c.args, signed([1]), 2)
    with pytest.raises(tq.TrellisError, match="workspace"):
        tq.window_attention_kv8(q, *c.args, 2, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
