"""Page operations on long lists: names repeated far apart, more sequences than
one workgroup has threads, lengths written to another array."""
import pytest
import torch

import trellis_coded_quantized_amd as tq
from tests.test_gpu_cache import World, ints

pytestmark = pytest.mark.gpu


def repeated(n, seqs):
    """n names out of `seqs` with repeats 1, 63, 64, 65 and 200 entries away, and unknown ones."""
    ids = [(11 * i) % seqs for i in range(n)]
    for at, back in ((70, 1), (130, 63), (131, 64), (132, 65), (n - 1, 200)):
        ids[at] = ids[at - back]
    ids[5], ids[66], ids[200] = -1, seqs, 2 ** 31 - 1
    return ids


@pytest.mark.parametrize("tokens", [2, 6])                   # slots with the plan, and by a launch of their own
def test_reserve_repeats_far_apart(tokens):
    w = World(seqs=331, width=3, pages=1200, pool=False)
    w.reserve(repeated(300, 331), [tokens - i % 2 for i in range(300)])
    w.reserve(repeated(300, 331), [16] * 300)


def test_fork_repeats_far_apart():
    w = World(seqs=331, width=2, pages=800, layers=1, heads=1)
    w.reserve([0, 1, 2], [20, 16, 1])
    w.fork([i % 3 for i in range(300)], repeated(300, 331))


@pytest.mark.parametrize("in_place", [False, True])
def test_accept_lengths_of_many_sequences(in_place):
    w = World(seqs=331, width=2, pages=800, layers=2, heads=2)
    ids = repeated(300, 331)
    start = [(5 * s) % 29 for s in range(331)]
    w.lengths.copy_(ints(start))
    new = w.lengths if in_place else torch.full_like(w.lengths, -9)
    counts = [(i * 3) % 5 - 1 for i in range(300)]
    k, v = w.k.clone(), w.v.clone()
    tq.cache_accept(w.k, w.v, w.table, w.lengths, ints(ids), ints([[0, 1, 2, 3]] * 300), ints(counts), new_lengths=new)
    want, seen = list(start), set()
    for s, n in zip(ids, counts):
        if 0 <= s < 331 and s not in seen:
            want[s] = min(start[s] + max(n, 0), 32)
            seen.add(s)
    assert new.tolist() == want
    assert torch.equal(w.k.view(torch.int16), k.view(torch.int16))
    assert torch.equal(w.v.view(torch.int16), v.view(torch.int16))
    if not in_place:
        assert w.lengths.tolist() == start


def test_fork_that_takes_page_0_beside_a_parent_of_full_pages():
    w = World(seqs=6, width=4, pages=12, layers=3)
    w.reserve([0, 1, 2], [5, 33, 32])                        # page 0, pages 1 to 3, pages 4 and 5
    w.free([0])
    w.fork([1, 2, 1], [3, 4, 5])                             # copies into pages 0 and 6, nothing for the second
    assert w.table[3].tolist()[2] == 0
