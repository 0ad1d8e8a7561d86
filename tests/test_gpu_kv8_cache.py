"""cache_fork_kv8 and cache_accept_kv8 against lists and blocks worked out on
the host, to the bit."""
import pytest
import torch

import trellis_coded_quantized_amd as tq
from tests import kv8_reference as r8
from tests import kv_reference as ref
from tests.kv8_reference import E4M3, E8M0

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


class World:
    def __init__(self, layers=2, heads=2, D=64, P=16, pages=40, seqs=6, width=6, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.P, self.D, self.layers, self.heads = P, D, layers, heads
        self.host = [r8.codes((60 * torch.randn(s, generator=g)).clamp(-448, 448)) for s in
                     ((layers, pages, heads, D // 16, P, 16), (layers, pages, heads, P // 16, D, 16))]
        self.host += [torch.randint(110, 130, (layers, pages, heads, P // 16), generator=g, dtype=torch.uint8)
                      for _ in range(2)]
        self.table, self.lengths, self.refs = tq.kv_state(seqs, width, pages, device=DEV)

    def upload(self):
        self.dev = [t.to(DEV).view(d) for t, d in zip(self.host, (E4M3, E4M3, E8M0, E8M0))]
        return self.dev

    def download(self):
        return [t.view(torch.uint8).cpu() for t in self.dev]

    def reserve(self, seqs, counts):
        starts = [0]
        for n in counts:
            starts.append(starts[-1] + n)
        _, granted = tq.cache_reserve(self.table, self.lengths, self.refs, self.P, ints(seqs), ints(starts), starts[-1])
        assert granted.all()
        for s, n in zip(seqs, counts):
            self.lengths[s] += n


@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (256, 32)])
def test_fork_copies_codes_and_scales(D, P):
    w = World(D=D, P=P, layers=3)
    w.reserve([0, 1, 2], [2 * P + 5, P, 3])
    lists = ref.Pages(w.table.cpu(), w.lengths.cpu(), w.refs.cpu(), P)
    pools = w.upload()
    granted = tq.cache_fork_kv8(*pools, w.table, w.lengths, w.refs, ints([0, 1, 2, 0, 9]), ints([3, 4, 5, 3, 2]))
    want, copies = lists.fork([0, 1, 2, 0, 9], [3, 4, 5, 3, 2])
    assert granted.tolist() == want
    lists.same_as(w.table.cpu(), w.lengths.cpu(), w.refs.cpu())
    for got, host in zip(w.download(), w.host):
        for a, b in copies:
            host[:, b] = host[:, a]
        assert torch.equal(got, host)


def expected_accept(w, table, length, path):
    """The pools after rows path[j] of one sequence moved to length + j, block by block."""
    P, pools = w.P, [t.clone() for t in w.host]

    def place(at):
        page = table[at // P] if 0 <= at // P < len(table) else -1
        return (page * P + at % P) // 16 if 0 <= page < w.host[0].shape[1] else None

    kinds = ((r8.block_of_keys, r8.put_block_of_keys, 0, 2), (r8.block_of_values, r8.put_block_of_values, 1, 3))
    moves = {}
    for j, p in enumerate(path):
        if p != j and p >= 0 and place(length + p) is not None and place(length + j) is not None:
            moves.setdefault(place(length + j), []).append((j, p))
    for layer in range(w.layers):
        for get, put, pool, scale in kinds:
            for block, rows in moves.items():
                code, byte = get(w.host[pool][layer], w.host[scale][layer], block, P)
                came = [get(w.host[pool][layer], w.host[scale][layer], place(length + p), P) for _, p in rows]
                now = byte
                for _, b in came:
                    now = torch.maximum(now, b)
                out = r8.rescale(code, byte[:, None, None], now[:, None, None])
                out = torch.where((now == byte)[:, None, None], code, out)
                for (j, p), (c, b) in zip(rows, came):
                    out[:, :, (length + j) % 16] = r8.rescale(c[:, :, (length + p) % 16], b[:, None], now[:, None])
                put(pools[pool][layer], pools[scale][layer], block, P, out, now)
    return pools


@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (256, 32)])
@pytest.mark.parametrize("length,path", [
    (0, [0, 1, 2]), (7, [0, 2, 5]), (13, [1, 2, 9, 30]), (16, [3]), (30, list(range(5, 60, 2))),
    (5, [63]), (20, [0, 1, 2, 3, 20, 21, 22, 40]), (15, list(range(64)))])
def test_accept(D, P, length, path):
    w = World(D=D, P=P, layers=2, width=-(-100 // P) + 1, seed=length + D)
    w.reserve([0, 2], [length + 64 if length + 64 <= 90 else 90, 20])
    w.lengths[0], w.lengths[2] = length, 4
    other = [1, 3]
    counts = [len(path), len(other)]
    rows = torch.zeros((2, 64), dtype=torch.int32)
    rows[0, :len(path)], rows[1, :2] = torch.tensor(path), torch.tensor(other)
    table = w.table.tolist()
    want = expected_accept(w, table[0], length, path)
    w.host, keep = want, w.host
    want = expected_accept(w, table[2], 4, other)
    w.host = keep
    for in_place in (False, True):
        pools = w.upload()
        lengths = w.lengths.clone()
        new = None if in_place else torch.full_like(lengths, -3)
        got = tq.cache_accept_kv8(*pools, w.table, lengths, ints([0, 2]), rows.to(DEV), ints(counts), new_lengths=new)
        assert got.tolist()[:3] == [length + counts[0], 0, 4 + counts[1]]
        for a, b, name in zip(w.download(), want, ("k", "v", "k_scale", "v_scale")):
            assert torch.equal(a, b), (name, in_place)


def test_accept_of_rows_without_storage_repeated_and_unknown_sequences():
    w = World(width=3)
    w.reserve([0], [40])
    w.lengths[0] = 10
    w.table[0, 2] = -1                                         # tokens 32 .. are gone
    path = [2, 25, 30, 4]
    want = expected_accept(w, w.table[0].tolist(), 10, path)
    pools = w.upload()
    rows = torch.tensor([path, path, path], dtype=torch.int32, device=DEV)
    got = tq.cache_accept_kv8(*pools, w.table, w.lengths, ints([0, 0, 77]), rows, ints([4, 4, 4]))
    assert got.tolist()[0] == 14
    for a, b in zip(w.download(), want):
        assert torch.equal(a, b)


def test_accept_in_a_graph():
    w = World(width=6, seed=4)
    w.reserve([0], [50])
    w.lengths[0] = 12
    rows = torch.tensor([[1, 4, 9, 20]], dtype=torch.int32, device=DEV)
    want = expected_accept(w, w.table[0].tolist(), 12, [1, 4, 9, 20])
    pools, new = w.upload(), torch.zeros_like(w.lengths)
    ids, counts = ints([0]), ints([4])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.cache_accept_kv8(*pools, w.table, w.lengths, ids, rows, counts, new_lengths=new)
    for _ in range(4):
        for p, h in zip(pools, w.host):
            p.view(torch.uint8).copy_(h.to(DEV))
        new.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert new.tolist()[0] == 16
        for a, b in zip(w.download(), want):
            assert torch.equal(a, b)


def test_refusals():
    w = World()
    k, v, ks, vs = w.upload()
    one, path = ints([0]), ints([[0]])
    with pytest.raises(TypeError, match="k_cache: dtype"):
        tq.cache_fork_kv8(k.view(torch.uint8), v, ks, vs, w.table, w.lengths, w.refs, one, one)
    with pytest.raises(ValueError, match="refs"):
        tq.cache_fork_kv8(k, v, ks, vs, w.table, w.lengths, w.refs[:-1], one, one)
    with pytest.raises(ValueError, match="children"):
        tq.cache_fork_kv8(k, v, ks, vs, w.table, w.lengths, w.refs, one, ints([1, 2]))
    with pytest.raises(tq.TrellisError, match="max_path"):
        tq.cache_accept_kv8(k, v, ks, vs, w.table, w.lengths, one, torch.zeros((1, 65), dtype=torch.int32, device=DEV), one)
    with pytest.raises(ValueError, match="v_scale: shape"):
        tq.cache_accept_kv8(k, v, ks, vs[:, :-1], w.table, w.lengths, one, path, one)
