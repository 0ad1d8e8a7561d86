"""Forks of parents that lack pages of their length: refused, the child left
empty, whichever page it is."""
import pytest
import torch

import trellis_coded_quantized_amd as tq
from tests.test_gpu_cache import World, ints

pytestmark = pytest.mark.gpu


def fork(w, parents, children):
    return tq.cache_fork(w.k, w.v, w.table, w.lengths, w.refs, ints(parents), ints(children)).tolist()


def holds(w, s):
    return [p for p in w.table[s].tolist() if p >= 0]


@pytest.mark.parametrize("tokens", [32, 37, 96])                   # whole pages, a partial one, the whole table
@pytest.mark.parametrize("no_page", [-1, 40, -2 ** 31, 2 ** 31 - 1])
def test_a_missing_full_page(tokens, no_page):
    for at in range(tokens // 16):
        w = World()
        w.reserve([0, 1, 2], [tokens, 20, 40])
        lost = w.table[0, at].item()
        w.table[0, at] = no_page
        before, k = w.refs.clone(), w.k.clone()
        assert fork(w, [0, 1, 0], [2, 3, 4]) == [0, 1, 0]
        for kid in (2, 4):
            assert holds(w, kid) == [] and w.lengths[kid] == 0
        assert w.lengths[3] == 20 and w.table[3, 0] == w.table[1, 0]
        # child 2's old pages are back, of the parent nothing is shared or held on to
        want = before.clone()
        mine = w.table[1, 0].item()
        want[mine] += 1
        copy = w.table[3, 1].item()
        for p in range(len(want)):
            if before[p] == 1 and p not in holds(w, 0) + holds(w, 1) + [lost]:
                want[p] -= 1                                       # pages of child 2
        want[copy] = 1
        assert torch.equal(w.refs, want)
        other = torch.arange(40, device=k.device) != copy
        assert torch.equal(w.k[:, other].view(torch.int16), k[:, other].view(torch.int16))


def test_a_length_without_any_page():
    w = World()
    w.lengths[:3] = ints([32, 5, 16])
    assert fork(w, [0, 1, 2], [3, 4, 2]) == [0, 0, 1]              # the last is its own parent: left as it is
    assert (w.table == -1).all() and not w.refs.any()
    assert w.lengths.tolist()[:5] == [32, 5, 16, 0, 0]


@pytest.mark.parametrize("length", [97, 112, 2 ** 31 - 1])
def test_a_length_past_the_table(length):
    w = World()
    w.reserve([0], [96])
    w.lengths[0] = length
    before = w.refs.clone()
    assert fork(w, [0], [1]) == [0]
    assert holds(w, 1) == [] and w.lengths[1] == 0
    assert torch.equal(w.refs, before)


def test_holes_past_the_length_do_not_matter():
    w = World()
    w.reserve([0], [40])
    w.table[0, 5] = 2 ** 31 - 1
    assert fork(w, [0], [1]) == [1]
    assert w.lengths[1] == 40 and len(holds(w, 1)) == 3


def test_a_parent_with_a_hole_that_is_replaced_itself():
    w = World()
    w.reserve([0, 1], [50, 20])
    lost = w.table[0, 1].item()
    w.table[0, 1] = -1
    assert fork(w, [0, 1], [2, 0]) == [0, 1]
    assert holds(w, 2) == [] and w.lengths.tolist()[:3] == [20, 20, 0]
    held = sorted(holds(w, 0) + holds(w, 1))
    want = [held.count(p) + (p == lost) for p in range(40)]
    assert w.refs.tolist() == want
