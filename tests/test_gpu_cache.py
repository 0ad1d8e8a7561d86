"""The cache's page operations against lists in Python: tables, lengths and
reference counts have to be equal, copied pages and rows bit for bit."""
import pytest
import torch

import trellis_coded_quantized_amd as tq
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, FP16 = torch.bfloat16, torch.float16


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def starts(counts):
    s = [0]
    for n in counts:
        s.append(s[-1] + n)
    return ints(s)


class World:
    """Device state and its mirror in lists; k and v hold distinct bits everywhere."""

    def __init__(self, seqs=8, width=6, pages=40, P=16, layers=3, heads=2, D=64, dtype=BF16, pool=True):
        self.P = P
        self.table, self.lengths, self.refs = tq.kv_state(seqs, width, pages, DEV)
        if pool:
            self.k, self.v = tq.kv_cache(layers, pages, heads, D, P, dtype, DEV)
            for t in (self.k, self.v):
                t.view(torch.int16).copy_(torch.randint(-32768, 32767, t.shape, device=DEV, dtype=torch.int16))
        self.mirror = ref.Pages(self.table, self.lengths, self.refs, P)

    def reserve(self, ids, counts, grow=True):
        slots, granted = tq.cache_reserve(self.table, self.lengths, self.refs, self.P, ints(ids), starts(counts),
                                          sum(counts))
        want = self.mirror.reserve(ids, counts)
        assert slots.tolist() == want[0]
        assert granted.tolist() == want[1]
        if grow:
            done = set()
            for s, n, ok in zip(ids, counts, want[1]):
                if ok and s not in done:
                    self.lengths[s] += n
                    self.mirror.lengths[s] += n
                    done.add(s)
        self.same()

    def fork(self, parents, children):
        k, v = self.k.clone(), self.v.clone()
        granted = tq.cache_fork(self.k, self.v, self.table, self.lengths, self.refs, ints(parents), ints(children))
        want, copies = self.mirror.fork(parents, children)
        assert granted.tolist() == want
        for src, dst in copies:
            k[:, dst], v[:, dst] = k[:, src].clone(), v[:, src].clone()
        assert torch.equal(self.k.view(torch.int16), k.view(torch.int16))
        assert torch.equal(self.v.view(torch.int16), v.view(torch.int16))
        self.same()

    def free(self, ids):
        tq.cache_free(self.table, self.lengths, self.refs, ints(ids))
        self.mirror.free(list(dict.fromkeys(ids)))
        self.same()

    def same(self):
        self.mirror.same_as(self.table, self.lengths, self.refs)


@pytest.mark.parametrize("P", [16, 64, 256])
def test_reserve_grows_sequences(P):
    w = World(P=P, pool=False)
    w.reserve([3, 0, 5], [1, 0, 2 * P])
    w.reserve([0, 3], [P - 1, P])
    w.reserve([0], [1])                          # the last place of a page it holds
    w.reserve([0], [1])                          # the first of the next
    w.reserve([5, 1], [P, 1], grow=False)        # drafts: pages held beyond the length
    w.reserve([5, 1], [1, 2], grow=False)        # are not taken twice
    w.reserve([7], [6 * P])


def test_reserve_refusals():
    w = World(seqs=6, width=5, pages=10, pool=False)
    w.reserve([0, 1], [50, 81])                  # past the table's width
    w.reserve([2, 2, 7, -1], [16, 16, 4, 4])     # repeated and unknown sequences
    w.reserve([3, 4, 5], [48, 16 * 4, 16])       # 5 left: 3 fit, 4 do not, 1 after them does not count as fitting
    w.reserve([5], [16])
    w.reserve([4], [16 * 2])
    w.reserve([1], [1])                          # none left


def test_reserve_many_sequences_and_pages():
    w = World(seqs=1100, width=40, pages=40000, pool=False)
    ids = [(7 * s) % 1100 for s in range(1024)]
    w.reserve(ids, [(13 * s) % 600 for s in range(1024)])
    w.free(ids[::3])
    w.reserve(ids[1::3], [17] * len(ids[1::3]))
    w.reserve(ids[::3], [200] * len(ids[::3]))


def test_reserve_a_long_prompt():
    w = World(seqs=2, width=9000, pages=70001, pool=False)
    w.reserve([0], [5])
    w.reserve([1], [131071])
    w.free([0])
    w.reserve([0], [9000 * 16])


def test_fork_shares_full_pages_and_copies_the_partial_one():
    w = World()
    w.reserve([0, 1], [16 * 2 + 5, 16])
    w.fork([0, 0, 1], [2, 3, 4])
    w.reserve([2, 3, 0, 4], [12, 1, 1, 1])       # each writes behind its own copy
    w.free([0])
    w.fork([2, 2], [2, 0])                       # its own parent; a freed child
    w.free([2, 3, 4, 0, 1])
    assert not w.refs.any()


@pytest.mark.parametrize("D,P,heads,dtype", [(128, 32, 1, FP16), (256, 16, 4, BF16)])
def test_fork_layouts(D, P, heads, dtype):
    w = World(P=P, D=D, heads=heads, dtype=dtype, layers=5)
    w.reserve([6], [2 * P + 7])
    w.fork([6] * 4, [0, 1, 2, 3])


def test_fork_replaces_children_and_parents():
    """Beam search: parents are replaced in the call that copies them."""
    w = World(pages=16)
    w.reserve([0, 1, 2], [20, 40, 33])
    w.fork([1, 0, 1], [0, 1, 2])
    w.fork([2, 2, 0, 1], [0, 1, 2, 3])
    w.fork([3, 0], [0, 3])
    for s in range(4):
        w.free([s])
    assert not w.refs.any()


def test_fork_refusals():
    w = World(pages=6, width=4)
    w.reserve([0, 1], [20, 16 * 3])
    w.fork([0, 0, 0, 1], [2, 3, 4, 5])           # one free page: 3, 4 refused and left empty, 5 has no partial page
    w.fork([0, 9, 1, 1, 1, 0], [6, 7, 7, -1, 8, 6])
    w.fork([9], [2])                             # an unknown parent empties the child
    w.table[0, 1] = -1                           # a parent without the page of its length
    w.mirror.table[0][1] = -1
    w.fork([0], [5])


def test_fork_twice_is_the_same():
    w = World()
    w.reserve([0, 1], [21, 37])
    w.fork([0, 1, 0], [5, 6, 7])
    before = (w.table.clone(), w.refs.clone())
    w.fork([0, 1, 0], [5, 6, 7])
    assert torch.equal(before[0], w.table) and torch.equal(before[1], w.refs)


def test_free_repeated_unknown_and_shared():
    w = World()
    w.reserve([0, 1], [50, 16])
    w.fork([0], [2])
    w.free([0, 0, 5, -3, 99, 0])
    w.free([2])
    assert int(w.refs.sum()) == 1


@pytest.mark.parametrize("D,P,heads,dtype", [(64, 16, 2, BF16), (128, 64, 1, FP16), (256, 16, 3, BF16)])
def test_accept(D, P, heads, dtype):
    layers = 3
    w = World(P=P, D=D, heads=heads, dtype=dtype, layers=layers)
    ids, ctx = [4, 1, 0, 6, 2], [P - 3, 0, 5, 2 * P + 1, 1]
    w.reserve(ids, ctx)
    w.reserve(ids, [20, 3, 64, 9, 1], grow=False)
    path = [[0, 2, 3, 7, 19], [0, 1, 2, 0, 0], [1, 5, 6, 40, 63], [3, 4, 0, 0, 0], [0, 0, 0, 0, 0]]
    counts = [5, 3, 5, 2, 0]
    want_k, want_v = w.k.clone(), w.v.clone()
    for b, s in enumerate(ids):
        for layer in range(layers):
            at = lambda i: ref.seq_slots(w.table[s].long(), ctx[b] + i + 1, P)[-1:]     # noqa: E731
            rows = [ref.take_tokens(w.k[layer], w.v[layer], at(path[b][j])) for j in range(counts[b])]
            for j, (k, v) in enumerate(rows):
                ref.put_tokens(want_k[layer], want_v[layer], at(j), k, v)
    new = torch.empty_like(w.lengths)
    old = w.lengths.clone()
    tq.cache_accept(w.k, w.v, w.table, w.lengths, ints(ids), ints(path), ints(counts), new_lengths=new)
    assert torch.equal(w.k.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(w.v.view(torch.int16), want_v.view(torch.int16))
    assert torch.equal(w.lengths, old)
    for s, n in zip(ids, counts):
        old[s] += n
    assert torch.equal(new, old)


def test_accept_in_place_of_lengths_repeats_and_rows_without_storage():
    w = World(layers=1)
    w.reserve([0, 1], [10, 16])
    w.reserve([0], [4], grow=False)
    k, v = w.k.clone(), w.v.clone()
    ids, path = ints([0, 0, 1, 9, -1]), ints([[0, 1], [1, 3], [0, 5], [0, 1], [0, 1]])
    got = tq.cache_accept(w.k, w.v, w.table, w.lengths, ids, path, ints([2, 2, 2, 2, 2]))
    assert got is w.lengths
    assert w.lengths.tolist()[:3] == [12, 18, 0]
    assert torch.equal(w.k.view(torch.int16), k.view(torch.int16))   # identity paths, and 1 + 5 has no page
    assert torch.equal(w.v.view(torch.int16), v.view(torch.int16))


def test_accept_64_rows_of_256():
    w = World(layers=1, D=256, heads=1, width=20)
    w.reserve([0], [3])
    w.reserve([0], [130], grow=False)
    slots = ref.seq_slots(w.table[0].long(), 133, 16)
    k, v = ref.take_tokens(w.k[0], w.v[0], slots)
    path = list(range(0, 128, 2))
    tq.cache_accept(w.k, w.v, w.table, w.lengths, ints([0]), ints([path]), ints([64]))
    gk, gv = ref.take_tokens(w.k[0], w.v[0], slots)
    assert torch.equal(gk[3:67].view(torch.int16), k[3:131:2].view(torch.int16))
    assert torch.equal(gv[3:67].view(torch.int16), v[3:131:2].view(torch.int16))
    assert torch.equal(gk[67:].view(torch.int16), k[67:].view(torch.int16))
    assert w.lengths.tolist()[0] == 67


def test_steps_in_a_graph():
    """reserve, accept and fork, captured once, replayed with the state of the moment."""
    w = World(seqs=4, width=12, pages=60, layers=2)
    w.reserve([0, 1], [10, 3])
    ids, st, path, counts = ints([0, 1]), starts([4, 4]), ints([[0, 1, 2], [0, 1, 2]]), ints([3, 2])
    slots, granted, kids = ints([0] * 8), ints([0, 0]), ints([2, 3])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        tq.cache_reserve(w.table, w.lengths, w.refs, 16, ids, st, 8, slots=slots, granted=granted)
        tq.cache_accept(w.k, w.v, w.table, w.lengths, ids, path, counts)
        tq.cache_fork(w.k, w.v, w.table, w.lengths, w.refs, ids, kids, granted=granted)
    for rep in range(5):
        want = w.mirror.reserve([0, 1], [4, 4])
        for s, n in ((0, 3), (1, 2)):
            w.mirror.lengths[s] += n
        w.mirror.fork([0, 1], [2, 3])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert slots.tolist() == want[0], rep
        w.same()


def test_refusals():
    w = World()
    with pytest.raises(tq.TrellisError, match="sequences outside"):
        tq.cache_free(w.table, w.lengths, w.refs, ints([0] * 1025))
    with pytest.raises(tq.TrellisError, match="sequences outside"):
        tq.cache_free(w.table, w.lengths, w.refs, ints([]))
    with pytest.raises(ValueError, match="shape"):
        tq.cache_fork(w.k, w.v, w.table, w.lengths, w.refs, ints([0, 1]), ints([2]))
    with pytest.raises(ValueError, match="shape"):
        tq.cache_fork(w.k, w.v, w.table, w.lengths, w.refs[:-1], ints([0]), ints([2]))
    with pytest.raises(tq.TrellisError, match="page_size"):
        tq.cache_reserve(w.table, w.lengths, w.refs, 24, ints([0]), starts([1]), 1)
    with pytest.raises(tq.TrellisError, match="max_path"):
        tq.cache_accept(w.k, w.v, w.table, w.lengths, ints([0]), ints([[0] * 65]), ints([1]))
    with pytest.raises(ValueError, match="shape"):
        tq.cache_accept(w.k, w.v, w.table, w.lengths, ints([0]), ints([[0], [0]]), ints([1]))
    with pytest.raises(ValueError, match="workspace"):
        tq.cache_fork(w.k, w.v, w.table, w.lengths, w.refs, ints([0]), ints([2]),
                      workspace=torch.empty(1 << 16, dtype=torch.uint8))
