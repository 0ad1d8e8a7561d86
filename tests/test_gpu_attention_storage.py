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


class Holes(Case):
    """A case whose pool has one more page in front, page 0, which is another sequence's; some pages of the tables
    are taken away."""

    def __init__(self, *args, page0, **kw):
        super().__init__(*args, **kw)
        self.page0 = page0
        self.held = [torch.ones(c + n, dtype=torch.bool) for c, n in zip(self.ctxs, self.ns)]
        self.missing = []

    def take(self, entry, at, entry_is):
        """Table entry `at` of an entry becomes entry_is."""
        self.missing.append((self.ids[entry], at, entry_is))
        self.held[entry][at * self.P:(at + 1) * self.P] = False

    def to_device(self):
        q = super().to_device()
        k, v, table, lengths, starts = self.args
        k, v = (torch.cat([torch.full_like(x[:1], self.page0), x]) for x in (k, v))
        table = torch.where(table >= 0, table + 1, table).int()
        for s, at, entry_is in self.missing:
            table[s, at] = k.shape[0] if entry_is == "pages" else entry_is
        self.args = (k, v, table, lengths, starts)
        return q

    def check(self, got, sees, scale, what=""):
        super().check(got, [see & h[None] for see, h in zip(sees, self.held)], scale, what)


NO_PAGE = [-1, "pages", 2 ** 31 - 1, -2 ** 31]


def both(c, scale, windows=((0, 0), (70, 20))):
    q = c.to_device()
    n = max(c.ns)
    for window, sinks in windows:
        got = tq.window_attention(q, *c.args, n, window=window, sinks=sinks)
        c.check(got, window_sees(c, window, sinks), scale, f"window {window}")
    if n <= 64:
        masks = [m for x in c.ns for m in random_tree(x, c.g)]
        c.check(tq.tree_attention(q, *c.args, signed(masks), n), tree_sees(c, masks), scale, "tree")


@pytest.mark.parametrize("page0", [float("nan"), float("inf"), 300.0])
@pytest.mark.parametrize("n", [2, 40])
@pytest.mark.parametrize("hq,hkv,D,P,dtype", [
    (8, 2, 64, 16, BF16), (32, 8, 128, 32, FP16), (12, 2, 256, 16, BF16), (8, 1, 128, 128, BF16)])
def test_keys_without_storage_are_not_seen(hq, hkv, D, P, dtype, n, page0):
    c = Holes([300, 0, 129, 64], [n, n, 1, n], hq, hkv, D, P, dtype, seed=D + n, page0=page0)
    c.take(0, 0, NO_PAGE[0])                                       # first tokens
    c.take(0, 150 // P, NO_PAGE[1])                                # amid the context
    c.take(0, 299 // P, NO_PAGE[2])                                # the window's first keys, new tokens
    c.take(1, 0, NO_PAGE[3])
    c.take(3, 64 // P, NO_PAGE[0])                                 # the new tokens, as after a refused reservation
    both(c, D ** -0.5)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (256, 32)])
def test_sequences_without_any_page_give_zeros(n, D, P):
    c = Holes([700, 90], [n, n], 8, 2, D, P, BF16, page0=float("nan"))
    for at in range(-(-(700 + n) // P)):
        c.take(0, at, NO_PAGE[at % 4])
    q = c.to_device()
    for got in (tq.window_attention(q, *c.args, n), tq.window_attention(q, *c.args, n, window=64, sinks=4),
                tq.tree_attention(q, *c.args, signed([1] * (2 * n)), n)):
        assert not got[:n].any()
        assert got[n:].isfinite().all() and got[n:].any()


@pytest.mark.parametrize("n", [1, 100])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_holes_in_long_contexts(n, D):
    """Keys that are split over workgroups: whole parts without storage, and holes in others."""
    c = Holes([9001, 40], [n, 1], 8, 2, D, 16, BF16, seed=n, page0=float("inf"))
    for at in list(range(0, 130)) + list(range(200, 563, 7)):
        c.take(0, at, -1)
    both(c, D ** -0.5, windows=((0, 0), (5000, 3)))


def test_infinities_among_holes():
    """Values that some rows see, beside pages that none does."""
    for n in (3, 40):
        c = Holes([200], [n], 8, 2, 64, 16, FP16, page0=float("nan"))
        c.vals[0][10, 0, 1], c.vals[0][199, 1, 2] = float("inf"), float("-inf")
        c.vals[0][200 + n - 1, 0, 5] = float("nan")
        c.take(0, 1, -1)
        c.take(0, 11, "pages")
        both(c, 64 ** -0.5, windows=((0, 0), (20, 12)))


@pytest.mark.parametrize("n", [3, 40])
def test_a_refused_reservation_shows_nobody_elses_keys(n):
    """reserve, append and attend as a captured step runs them: the host does not know that an entry was refused."""
    P, D, hq, hkv = 16, 64, 8, 2
    i32 = dict(dtype=torch.int32, device=DEV)
    k, v = tq.kv_cache(1, 8, hkv, D, P, BF16, DEV)
    table, lengths, refs = tq.kv_state(2, 8, 8, DEV)
    g = torch.Generator().manual_seed(n)

    def step(ids, counts):
        total = sum(counts)
        starts = torch.tensor([0] + [sum(counts[:i + 1]) for i in range(len(counts))], **i32)
        ids = torch.tensor(ids, **i32)
        slots, granted = tq.cache_reserve(table, lengths, refs, P, ids, starts, total)
        x = torch.randn((total, hq + 2 * hkv, D), generator=g).to(BF16).to(DEV)
        ones = torch.ones(D, dtype=BF16, device=DEV)
        q = tq.qk_norm_rope(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], ones, ones, torch.zeros(total, **i32),
                            torch.empty(0, device=DEV), slots, k[0], v[0])
        return granted, tq.window_attention(q, k[0], v[0], table, lengths, starts, max(counts), seq_ids=ids)

    granted, _ = step([0], [112])                                  # 7 of 8 pages
    lengths[0] += 112
    v[0] += 100                                                    # what nobody else may see
    granted, out = step([0, 1], [n, 16 + n])                       # 1 asks for more than the one page left
    assert granted.tolist() == ([1, 0] if n <= 16 else [0, 0])
    assert out[:n].float().min() > 10
    assert not out[n:].any()
