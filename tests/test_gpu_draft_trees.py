"""The operators together: trees of drafts against decoding one by one."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompt,steps,nodes", [(700, 4, 8), (17, 3, 2), (1030, 2, 33)])
def test_trees_and_single_tokens_agree(prompt, steps, nodes):
    from examples.draft_trees import run
    # Both ways round weights (bf16 expansion of the packed ones for many rows
    # only), projections, rotated heads, softmax weights and outputs, half a
    # step u = eps / 2 each, in other places.  Scores: heads of norm up to 1.5 sqrt(D), each
    # off by 3 u on either way, so at most 1.5^2 sqrt(D) 6 u if all of it were
    # aligned; roundings are not, which divides by sqrt(D): 2.25 * 6 u.  A
    # score's error is its weight's relative error.  Values, weights, the
    # sum's output and the projection: 4 u on either way.  The largest error
    # and the largest output spread over the same range, so their ratio is
    # that of the typical ones.
    u = torch.finfo(torch.bfloat16).eps / 2
    assert run("cuda:0", prompt, steps, nodes) <= 2.25 * 6 * u + 8 * u
