"""Adapters, the 8-bit append, attention, fork and accept as a server runs them
together: trees of drafts against decoding one by one."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompts,steps,nodes", [((70, 41, 150), 3, 7), ((3,), 4, 2), ((300, 17, 5, 64), 2, 20)])
def test_trees_and_single_tokens_agree(prompts, steps, nodes):
    from examples.adapters import run
    # u: half a step of bf16, w: of e4m3, both relative.  The two ways round
    # in other places, so either one is off by what its roundings can do:
    # attention: projections, adapters, heads, weights, outputs (as in the
    # drafted trees without adapters: 2.25 * 6 u + 8 u, here with two more for
    # the adapters' sums) and, new, codes: half a step w in every key, which
    # moves a score by at most 2.25 w (norms 1.5 sqrt(D), a dot product of
    # unaligned errors, scaled by 1 / sqrt(D)), and w in every value: 3.25 w on
    # either way.
    # gated half: weights rounded to bf16 on one way only, gate and up rounded
    # once on one way, the output on both: 4 u, each of gate and up passed on
    # by at most 1.1 and the other's size.
    u, w = torch.finfo(torch.bfloat16).eps / 2, 2.0 ** -4
    attention, gated = run("cuda:0", prompts, steps, nodes)
    assert attention <= 2.25 * 6 * u + 10 * u + 2 * 3.25 * w
    assert gated <= 2 * 4 * u
