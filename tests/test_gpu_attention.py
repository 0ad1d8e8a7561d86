"""tree_attention and window_attention against plain 64-bit attention, at the
sizes, masks and contents where an attention over a paged cache goes wrong."""
import pytest
import torch

import trellis_coded_quantized_amd as tq
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, FP16 = torch.bfloat16, torch.float16


class Case:
    """A cache that is NaN wherever no token was written, and a batch of entries."""

    def __init__(self, ctxs, ns, hq, hkv, D, P, dtype, seed=0, extra_pages=3, seqs=None, ids=None, pad=1):
        g = torch.Generator().manual_seed(seed)
        self.ctxs, self.ns, self.hq, self.hkv, self.D, self.P, self.dtype = ctxs, ns, hq, hkv, D, P, dtype
        self.g = g
        seqs = len(ctxs) if seqs is None else seqs
        self.ids = list(range(len(ctxs))) if ids is None else ids
        need = [-(-(c + n) // P) for c, n in zip(ctxs, ns)]
        total = sum(need) + extra_pages
        order = torch.randperm(total, generator=g).int()
        self.table = torch.full((seqs, max(need) + pad), -1, dtype=torch.int32)
        self.lengths = torch.full((seqs,), 7, dtype=torch.int32)
        at = 0
        for e, s in enumerate(self.ids):
            self.table[s, :need[e]] = order[at:at + need[e]]
            self.lengths[s] = ctxs[e]
            at += need[e]
        self.k = torch.full((total, hkv, D // 8, P, 8), float("nan"), dtype=dtype)
        self.v = torch.full((total, hkv, P // 8, D, 8), float("nan"), dtype=dtype)
        self.keys, self.vals = [], []
        for e, s in enumerate(self.ids):
            n = ctxs[e] + ns[e]
            self.keys.append(torch.randn((n, hkv, D), generator=g).to(dtype))
            self.vals.append(torch.randn((n, hkv, D), generator=g).to(dtype))
        starts = [0]
        for n in ns:
            starts.append(starts[-1] + n)
        self.starts = starts
        self.q = torch.randn((starts[-1], hq, D), generator=g).to(dtype)

    def to_device(self):
        for e, s in enumerate(self.ids):
            n = self.ctxs[e] + self.ns[e]
            ref.put_tokens(self.k, self.v, ref.seq_slots(self.table[s], n, self.P), self.keys[e], self.vals[e])
        self.args = (self.k.to(DEV), self.v.to(DEV), self.table.to(DEV), self.lengths.to(DEV),
                     torch.tensor(self.starts, dtype=torch.int32, device=DEV))
        return self.q.to(DEV)

    def check(self, got, sees, scale, what=""):
        for e in range(len(self.ns)):
            a, b = self.starts[e], self.starts[e + 1]
            if a == b:
                continue
            parts = ref.attend(self.q[a:b], self.keys[e], self.vals[e], sees[e], scale)
            ref.assert_attention(got[a:b], parts, self.ctxs[e] + self.ns[e], self.D, f"{what} entry {e}")


def random_tree(n, g, own=True):
    masks = []
    for i in range(n):
        up = masks[int(torch.randint(max(0, i - 4), i, (1,), generator=g))] if i else 0
        masks.append(up | (1 << i))
    return masks


def signed(masks):
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device=DEV)


def run_tree(c, masks, max_q=None, scale=None, **kw):
    q = c.to_device()
    return tq.tree_attention(q, *c.args, signed(masks), max_q or max(c.ns), scale=scale, **kw)


def tree_sees(c, masks):
    return [ref.tree_see(c.ctxs[e], masks[c.starts[e]:c.starts[e + 1]], c.ctxs[e] + c.ns[e])
            for e in range(len(c.ns))]


def run_window(c, window, sinks, max_q=None, scale=None, **kw):
    q = c.to_device()
    return tq.window_attention(q, *c.args, max_q or max(c.ns), window=window, sinks=sinks, scale=scale, **kw)


def window_sees(c, window, sinks):
    return [ref.window_see(x, n, x + n, window, sinks) for x, n in zip(c.ctxs, c.ns)]


# contexts and node counts around tiles of 32 and 64 keys and around pages
@pytest.mark.parametrize("hq,hkv,D,P,dtype", [
    (24, 4, 256, 16, BF16), (32, 8, 128, 32, FP16), (16, 16, 64, 64, BF16), (8, 1, 128, 256, BF16),
    (6, 2, 64, 16, FP16), (5, 5, 256, 128, FP16)])
@pytest.mark.parametrize("ns", [[1, 1, 1, 1, 1], [4, 1, 3, 2, 4], [64, 1, 33, 0, 17]])
def test_tree(hq, hkv, D, P, dtype, ns):
    c = Case([0, 1, 31, 100, 257], ns, hq, hkv, D, P, dtype, seed=D + P)
    masks = [m for n in ns for m in random_tree(n, c.g)]
    got = run_tree(c, masks)
    c.check(got, tree_sees(c, masks), D ** -0.5)


@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 1000])
@pytest.mark.parametrize("n", [1, 5, 40])
def test_tree_lengths(ctx, n):
    c = Case([ctx], [n], 8, 2, 128, 16, BF16, seed=ctx)
    masks = random_tree(n, c.g)
    c.check(run_tree(c, masks), tree_sees(c, masks), 128 ** -0.5)


@pytest.mark.parametrize("n,hq", [(3, 4), (50, 4)])
def test_tree_rows_that_see_nothing_are_zero(n, hq):
    c = Case([0, 0, 20], [n, 2, 1], hq, 2, 128, 16, BF16)
    masks = [0] * n + [0, 2] + [0]
    got = run_tree(c, masks)
    assert not got[:n + 1].any()
    c.check(got, tree_sees(c, masks), 128 ** -0.5)


@pytest.mark.parametrize("n", [3, 64])
def test_tree_bits_without_a_token_and_arbitrary_masks(n):
    c = Case([9, 70], [n, 2], 4, 2, 64, 16, FP16)
    masks = [(0x9E3779B97F4A7C15 * (i + 1)) & (2 ** 64 - 1) for i in range(n)] + [2 ** 64 - 1, 2 ** 63]
    c.check(run_tree(c, masks), tree_sees(c, masks), 64 ** -0.5)


@pytest.mark.parametrize("n,D", [(4, 128), (64, 64), (40, 256)])
def test_tree_nonfinite_tokens_reach_only_rows_that_see_them(n, D):
    c = Case([37], [n], 8, 2, D, 16, BF16, seed=3)
    inf = float("inf")
    c.vals[0][37 + 1, 0, 3], c.vals[0][37 + 1, 1, D - 1] = inf, float("nan")
    c.vals[0][37 + 2, 0, 3], c.vals[0][37 + 2, 1, 40] = -inf, -inf
    c.keys[0][37 + 1] = float("nan")
    masks = [1 if i == 0 else 2 if i == 1 else (1 | 1 << i if i % 2 else 1 << i) for i in range(n)]
    sees = tree_sees(c, masks)
    got = run_tree(c, masks)
    # rows that see token 1 (a NaN key) are NaN; the others as if it were not there
    hit = sees[0][:, 38]
    assert got[hit.to(DEV)].isnan().all()
    rest = [i for i in range(n) if not hit[i]]
    c.keys[0][38] = 0
    parts = ref.attend(c.q[rest], c.keys[0], c.vals[0], sees[0][rest], D ** -0.5)
    ref.assert_attention(got[rest], parts, 37 + n, D)


def test_nonfinite_values_in_open_and_cut_tiles():
    inf = float("inf")
    for n, hq in ((1, 8), (1, 2), (30, 8)):
        c = Case([200], [n], hq, 2, 64, 16, FP16, seed=5)
        c.vals[0][10, 0, 1] = inf                    # seen by all
        c.vals[0][199, 1, 2] = -inf                  # before a window's last rows
        c.vals[0][200 + n - 1, 0, 5] = float("nan")  # seen by the last token only
        for window, sinks in ((0, 0), (3, 0), (40, 12)):
            got = run_window(c, window, sinks)
            c.check(got, window_sees(c, window, sinks), 64 ** -0.5, f"n {n} window {window}")


@pytest.mark.parametrize("hq,hkv,D,P,dtype", [
    (24, 4, 256, 16, BF16), (32, 8, 128, 64, FP16), (16, 16, 64, 16, BF16), (3, 1, 64, 32, FP16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (7, 3), (32, 0), (65, 33), (100, 4), (100000, 4)])
def test_window(hq, hkv, D, P, dtype, window, sinks):
    c = Case([0, 5, 300, 64, 129], [1, 2, 1, 0, 1], hq, hkv, D, P, dtype, seed=window)
    c.check(run_window(c, window, sinks), window_sees(c, window, sinks), D ** -0.5, "few")
    c = Case([0, 5, 300, 64, 129], [70, 2, 129, 0, 33], hq, hkv, D, P, dtype, seed=window + 1)
    c.check(run_window(c, window, sinks), window_sees(c, window, sinks), D ** -0.5, "many")


@pytest.mark.parametrize("sinks", [0, 1, 31, 32, 33, 64, 70, 200, 2 ** 31 - 1])
@pytest.mark.parametrize("n", [1, 90])
def test_sinks_around_tiles(sinks, n):
    c = Case([330], [n], 8, 2, 128, 16, BF16, seed=sinks % 1000)
    c.check(run_window(c, 50, sinks), window_sees(c, 50, sinks), 128 ** -0.5)


def test_window_largest_numbers():
    c = Case([40], [3], 4, 2, 64, 16, BF16)
    c.check(run_window(c, 2 ** 31 - 1, 2 ** 31 - 1), window_sees(c, 0, 0), 64 ** -0.5)


@pytest.mark.parametrize("n", [1, 100])
def test_long_context_split_over_workgroups(n):
    c = Case([9001, 40], [n, 1], 8, 2, 64, 16, BF16, seed=n)
    c.check(run_window(c, 0, 0), window_sees(c, 0, 0), 64 ** -0.5)


def test_many_entries():
    ns = [1 + (s % 2) for s in range(150)]
    ctxs = [(37 * s) % 400 for s in range(150)]
    c = Case(ctxs, ns, 4, 2, 64, 16, FP16)
    masks = [m for n in ns for m in random_tree(n, c.g)]
    c.check(run_tree(c, masks), tree_sees(c, masks), 64 ** -0.5)


@pytest.mark.parametrize("n", [2, 60])
def test_sequence_numbers_row_strides_and_scale(n):
    c = Case([50, 3, 90], [n, 1, n], 8, 2, 128, 16, BF16, seqs=6, ids=[4, 0, 2])
    q = c.to_device()
    wide = torch.full((q.shape[0], 8 + 3, 128), float("nan"), dtype=BF16, device=DEV)
    wide[:, 1:9] = q
    ids = torch.tensor(c.ids, dtype=torch.int32, device=DEV)
    got = tq.window_attention(wide[:, 1:9], *c.args, n, window=60, sinks=2, scale=0.3, seq_ids=ids)
    c.check(got, window_sees(c, 60, 2), 0.3)


def test_large_scores_stay_finite_and_right():
    for n in (1, 40):
        c = Case([300], [n], 4, 2, 64, 16, BF16)
        c.q *= 40
        c.check(run_window(c, 0, 0), window_sees(c, 0, 0), 64 ** -0.5)


@pytest.mark.parametrize("n", [1, 40])
def test_rising_scores_move_the_running_bound(n):
    """Keys grow along the cache, so every tile raises the maximum by more than the kernels' step."""
    c = Case([500], [n], 4, 2, 64, 16, FP16)
    c.keys[0] = torch.ones_like(c.keys[0]) * (torch.arange(500 + n)[:, None, None] / 64).to(FP16)
    c.q = c.q.abs()
    c.check(run_window(c, 0, 0), window_sees(c, 0, 0), 64 ** -0.5)


def test_bad_pages_lengths_and_sequences_stay_inside_the_arrays():
    """Entries of the table outside the pool, lengths past the table, unknown sequences: nothing outside is touched;
    well-formed entries of the same call are not disturbed."""
    for n in (2, 40):
        c = Case([60, 30, 20], [n, n, n], 4, 2, 64, 16, BF16, seqs=4, ids=[0, 1, 2])
        q = c.to_device()
        k, v, table, lengths, starts = c.args
        table[0, :] = torch.tensor([2 ** 31 - 1, -5] * 8, dtype=torch.int32, device=DEV)[:table.shape[1]]
        lengths[1] = 2 ** 31 - 1
        out = torch.zeros_like(q)
        ids = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
        tq.window_attention(q, k, v, table, lengths, starts, n, seq_ids=ids, out=out)
        a, b = c.starts[2], c.starts[3]
        parts = ref.attend(c.q[a:b], c.keys[2], c.vals[2], window_sees(c, 0, 0)[2], 64 ** -0.5)
        ref.assert_attention(out[a:b], parts, 20 + n, 64)
        bad = torch.tensor([9, -1, 2], dtype=torch.int32, device=DEV)
        out = torch.full_like(q, 3.0)
        tq.window_attention(q, k, v, table, lengths, starts, n, seq_ids=bad, out=out)
        assert (out[:a] == 3.0).all()
        ref.assert_attention(out[a:b], parts, 20 + n, 64)


def test_rows_past_max_q_are_left():
    c = Case([10], [6], 4, 2, 64, 16, BF16)
    q = c.to_device()
    out = torch.full_like(q, 2.0)
    tq.window_attention(q, *c.args, 4, out=out)
    assert (out[4:] == 2.0).all()
    parts = ref.attend(c.q[:4], c.keys[0][:14], c.vals[0][:14], ref.window_see(10, 4, 14, 0, 0), 64 ** -0.5)
    ref.assert_attention(out[:4], parts, 14, 64)


def test_no_tokens():
    c = Case([10], [1], 4, 2, 64, 16, BF16)
    c.to_device()
    q = torch.empty((0, 4, 64), dtype=BF16, device=DEV)
    assert tq.window_attention(q, *c.args, 1).shape == (0, 4, 64)
    assert tq.tree_attention(q, *c.args, torch.empty(0, dtype=torch.int64, device=DEV), 1).shape == (0, 4, 64)


@pytest.mark.parametrize("n", [2, 40])
def test_offsets_past_32_bits(n):
    """Pages at the far end of a pool of more than 2^32 bytes (and elements)."""
    P, D, hkv = 16, 128, 2
    pages = (1 << 32) // (P * D * hkv) + 50
    c = Case([100], [n], 4, hkv, D, P, BF16)
    q = c.to_device()
    small_k, small_v, table, lengths, starts = c.args
    k = torch.empty((pages,) + small_k.shape[1:], dtype=BF16, device=DEV)
    v = torch.empty((pages,) + small_v.shape[1:], dtype=BF16, device=DEV)
    held = small_k.shape[0]
    k[-held:], v[-held:] = small_k, small_v
    table = torch.where(table >= 0, table + (pages - held), table).int()
    got = tq.window_attention(q, k, v, table, lengths, starts, n)
    c.check(got, window_sees(c, 0, 0), D ** -0.5)


@pytest.mark.parametrize("n", [1, 60])
def test_same_bits_on_another_stream_and_in_a_graph(n):
    c = Case([700, 90], [n, n], 8, 2, 128, 16, BF16)
    q = c.to_device()
    want = tq.window_attention(q, *c.args, n, window=500, sinks=4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = tq.window_attention(q, *c.args, n, window=500, sinks=4)
    side.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.window_attention(q, *c.args, n, window=500, sinks=4, out=out)
    lengths = c.args[3]
    for rep in range(4):
        out.zero_()
        lengths[1] = 90 - 7 * rep                       # the graph reads lengths on the device
        eager = tq.window_attention(q, *c.args, n, window=500, sinks=4)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16)), rep


def test_refusals():
    c = Case([10], [2], 4, 2, 64, 16, BF16)
    q = c.to_device()
    k, v, table, lengths, starts = c.args
    anc = signed([1, 3])
    with pytest.raises(TypeError, match="dtype"):
        tq.window_attention(q.half(), *c.args, 2)
    with pytest.raises(ValueError, match="not one cache"):
        tq.window_attention(q, k, v[:, :, :1].contiguous(), table, lengths, starts, 2)
    with pytest.raises(ValueError, match="one layer"):
        tq.window_attention(q, k[None], v[None], table, lengths, starts, 2)
    with pytest.raises(ValueError, match="contiguous"):
        tq.window_attention(q.transpose(0, 1).contiguous().transpose(0, 1), *c.args, 2)
    with pytest.raises(tq.TrellisError, match="q_stride"):
        wide = torch.zeros((2, 4 * 64 + 4), dtype=BF16, device=DEV)
        tq.window_attention(wide[:, :256].unflatten(1, (4, 64)), *c.args, 2)
    with pytest.raises(tq.TrellisError, match="multiple of the cache's"):
        tq.window_attention(q[:, :3].contiguous(), *c.args, 2)
    with pytest.raises(tq.TrellisError, match="max_q"):
        tq.tree_attention(q, *c.args, anc, 65)
    with pytest.raises(tq.TrellisError, match="scale"):
        tq.tree_attention(q, *c.args, anc, 2, scale=0.0)
    with pytest.raises(tq.TrellisError, match="window"):
        tq.window_attention(q, *c.args, 2, window=-1)
    with pytest.raises(ValueError, match="ancestors"):
        tq.tree_attention(q, *c.args, anc[:1], 2)
    with pytest.raises(ValueError, match="entries"):
        tq.window_attention(q, k, v, table, lengths, torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV), 2)
    with pytest.raises(TypeError, match="dtype"):
        tq.window_attention(q, k, v, table.long(), lengths, starts, 2)
