"""A layer's attention between its packed projections, as a server would run it:
a prompt, a fork of it, then steps that verify trees of drafted tokens.

    python examples/draft_trees.py

The weights and the tokens are random, so the drafts and the accepted paths
are drawn instead of sampled.  At the end every accepted token is decoded
again, one at a time, in a sequence that never saw a draft; both ways have to
give the same rows (the largest difference is printed and returned).
"""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import trellis_coded_quantized_amd as tq
import trellis_inputs as ti

HIDDEN, HEADS, KV_HEADS, DIM, PAGE, BITS = 2048, 16, 4, 128, 16, 4
EPS = 1e-6


class Layer:
    """Packed qkv and output projections and the norm weights of one layer."""

    def __init__(self, rng, device):
        def packed(rows, cols):
            codes = torch.from_numpy(ti.codes(rng, rows, cols, BITS).view(np.int32)).to(device)
            scales = torch.from_numpy(ti.scales(rng, rows).view(np.int16)).to(device).view(torch.float16)
            return codes, scales

        def weight():
            return torch.from_numpy(rng.uniform(0.5, 1.5, DIM)).to(device, torch.bfloat16)

        self.qkv = packed((HEADS + 2 * KV_HEADS) * DIM, HIDDEN)
        self.o = packed(HIDDEN, HEADS * DIM)
        self.q_norm, self.k_norm = weight(), weight()
        self.inv_freq = (10000.0 ** (-torch.arange(0, DIM, 2, device=device) / DIM)).float()

    def project(self, packed, x):
        if x.shape[0] <= 4:
            return tq.matvec_axis1(*packed, x, BITS)
        return tq.prefill(*packed, x, BITS, algo=tq.PREFILL_AUTO)

    def heads(self, x, positions, slots, k_cache, v_cache):
        """Rotated queries of x; its keys and values are in the cache afterwards."""
        qkv = self.project(self.qkv, x).unflatten(1, (-1, DIM))
        q, k, v = qkv.split((HEADS, KV_HEADS, KV_HEADS), 1)          # views: the call takes their strides
        return tq.qk_norm_rope(q, k, v, self.q_norm, self.k_norm, positions, self.inv_freq, slots, k_cache, v_cache,
                               eps=EPS)

    def out(self, attended):
        return self.project(self.o, attended.flatten(1))


def draw_tree(rng, nodes):
    """Parents of a tree in draft order (-1: a root), the mask of every node's
    ancestors with itself, and its depth."""
    parents = [-1] + [int(rng.integers(-1, i)) for i in range(1, nodes)]
    masks, depth = [], []
    for i, p in enumerate(parents):
        masks.append((masks[p] if p >= 0 else 0) | 1 << i)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return parents, masks, depth


def run(device="cuda", prompt=700, steps=4, nodes=8, window=256, sinks=4, seed=0):
    """Largest difference between tree steps and decoding one by one, relative to the largest output."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=device).manual_seed(seed)
    i32 = dict(dtype=torch.int32, device=device)
    layer = Layer(rng, device)
    width = -(-(prompt + (steps + 1) * nodes) // PAGE)
    pages = 4 * width
    k, v = tq.kv_cache(1, pages, KV_HEADS, DIM, PAGE, device=device)
    table, lengths, refs = tq.kv_state(4, width, pages, device=device)

    def states(n):
        return torch.randn((n, HIDDEN), generator=gen, device=device).to(torch.bfloat16)

    # the prompt, in two chunks, into sequence 0: a window layer with sinks
    for at, n in ((0, prompt // 2), (prompt // 2, prompt - prompt // 2)):
        seq, starts = torch.tensor([0], **i32), torch.tensor([0, n], **i32)
        slots, granted = tq.cache_reserve(table, lengths, refs, PAGE, seq, starts, n)
        assert granted.all()
        q = layer.heads(states(n), torch.arange(at, at + n, **i32), slots, k[0], v[0])
        a = tq.window_attention(q, k[0], v[0], table, lengths, starts, n, window=window, sinks=sinks, seq_ids=seq)
        layer.out(a)
        lengths[0] += n

    # 1 and 2 continue the prompt with trees, 3 and later 0 decode what is accepted one by one
    assert tq.cache_fork(k, v, table, lengths, refs, torch.tensor([0, 0, 0], **i32), torch.tensor([1, 2, 3], **i32)).all()
    seqs, starts = torch.tensor([1, 2], **i32), torch.tensor([0, nodes, 2 * nodes], **i32)
    accepted = {1: [], 2: []}
    for _ in range(steps):
        trees = [draw_tree(rng, nodes) for _ in range(2)]
        x = states(2 * nodes)
        masks = torch.tensor(trees[0][1] + trees[1][1], device=device)
        depth = torch.tensor(trees[0][2] + trees[1][2], **i32)
        slots, granted = tq.cache_reserve(table, lengths, refs, PAGE, seqs, starts, 2 * nodes)
        assert granted.all()
        positions = lengths[1:3].repeat_interleave(nodes) + depth
        q = layer.heads(x, positions, slots, k[0], v[0])
        y = layer.out(tq.tree_attention(q, k[0], v[0], table, lengths, starts, masks, nodes, seq_ids=seqs))
        # keep one path: a node and its ancestors
        path, counts = torch.zeros((2, nodes), **i32), []
        for e, (_, mask, _) in enumerate(trees):
            end = int(rng.integers(nodes))
            kept = [i for i in range(nodes) if mask[end] >> i & 1]
            path[e, :len(kept)] = torch.tensor(kept, **i32)
            counts.append(len(kept))
            accepted[e + 1] += [(x[e * nodes + i], y[e * nodes + i]) for i in kept]
        tq.cache_accept(k, v, table, lengths, seqs, path, torch.tensor(counts, **i32))

    # once more, token by token
    worst = top = 0.0
    for twin, seq in ((3, 1), (0, 2)):
        one, starts = torch.tensor([twin], **i32), torch.tensor([0, 1], **i32)
        for x, y in accepted[seq]:
            slots, granted = tq.cache_reserve(table, lengths, refs, PAGE, one, starts, 1)
            assert granted.all()
            q = layer.heads(x[None], lengths[twin:twin + 1].clone(), slots, k[0], v[0])
            a = tq.window_attention(q, k[0], v[0], table, lengths, starts, 1, seq_ids=one)
            worst = max(worst, (layer.out(a)[0].float() - y.float()).abs().max().item())
            top = max(top, y.float().abs().max().item())
            lengths[twin] += 1
        assert lengths[twin] == lengths[seq]

    tq.cache_free(table, lengths, refs, torch.arange(4, **i32))
    assert not refs.any()
    return worst / top


if __name__ == "__main__":
    print(f"trees against one by one: largest difference {run():.2e} of the largest output")
