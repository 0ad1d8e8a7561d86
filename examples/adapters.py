"""One packed decoder layer for requests of several fine-tunes, over a cache held
in 8 bits: every request has its own low-rank adapter, or none.

    python examples/adapters.py

A prompt for each request, a fork of all of them, then steps that verify trees
of drafted tokens.  At the end every accepted token is decoded again, one at a
time, in the forks, which never saw a draft; both ways have to give the same
rows.  Weights, adapters and tokens are random.  Prints and returns the largest
differences, relative to the largest output, of the attention's half of the
layer and of its gated half.
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
from examples.draft_trees import draw_tree

HIDDEN, HEADS, KV_HEADS, DIM, WIDE, PAGE, BITS = 2048, 16, 4, 128, 2560, 16, 4
RANK, POOL = 16, 4
EPS = 1e-6
QKV = (HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM)


class Layer:
    """Packed projections of one layer, and the factors of POOL adapters beside them."""

    def __init__(self, rng, gen, device):
        def packed(rows, cols):
            codes = torch.from_numpy(ti.codes(rng, rows, cols, BITS).view(np.int32)).to(device)
            scales = torch.from_numpy(ti.scales(rng, rows).view(np.int16)).to(device).view(torch.float16)
            return codes, scales

        def normal(*shape, size):
            return (torch.randn(shape, generator=gen, device=device) * size).to(torch.bfloat16)

        def adapters(cols, rows):
            return ([normal(POOL, RANK, cols, size=cols ** -0.5) for _ in rows],
                    [normal(POOL, r, RANK, size=0.5) for r in rows])

        self.qkv, self.o = packed(sum(QKV), HIDDEN), packed(HIDDEN, HEADS * DIM)
        self.gate, self.up = packed(WIDE, HIDDEN), packed(WIDE, HIDDEN)
        self.qkv_ab, self.o_ab = adapters(HIDDEN, QKV), adapters(HEADS * DIM, (HIDDEN,))
        self.mlp_ab = adapters(HIDDEN, (WIDE, WIDE))
        self.scales = torch.linspace(0.5, 1.5, POOL, device=device)
        self.ranks = torch.tensor([RANK, RANK // 2, RANK, 5], dtype=torch.int32, device=device)
        self.q_norm, self.k_norm = (1 + normal(DIM, size=0.1) for _ in range(2))
        self.inv_freq = (10000.0 ** (-torch.arange(0, DIM, 2, device=device) / DIM)).float()

    def project(self, packed, x):
        if x.shape[0] <= 4:
            return tq.matvec_axis1(*packed, x, BITS)
        return tq.prefill(*packed, x, BITS, algo=tq.PREFILL_AUTO)

    def heads(self, x, starts, adapters, positions, slots, pools):
        """Rotated queries of x; its keys and values are in the cache afterwards."""
        qkv = self.project(self.qkv, x)
        parts = list(qkv.split(QKV, 1))                        # views: the adapters are added in place
        tq.lora_add(x, *self.qkv_ab, parts, starts, adapters, self.scales, ranks=self.ranks, outs=parts)
        q, k, v = (p.unflatten(1, (-1, DIM)) for p in parts)
        return tq.qk_norm_rope_kv8(q, k, v, self.q_norm, self.k_norm, positions, self.inv_freq, slots, *pools, eps=EPS)

    def out(self, attended, starts, adapters):
        a = attended.flatten(1)
        y = self.project(self.o, a)
        return tq.lora_add(a, *self.o_ab, [y], starts, adapters, self.scales, ranks=self.ranks, outs=[y])[0]

    def gated(self, x, starts, adapters):
        if x.shape[0] <= 4:
            gate, up = (torch.empty((x.shape[0], WIDE), dtype=torch.float32, device=x.device) for _ in range(2))
            tq.gateup_swiglu(*self.gate, *self.up, x, BITS, gate_f32=gate, up_f32=up)
        else:
            gate, up = self.project(self.gate, x), self.project(self.up, x)
        (ag, au), (bg, bu) = self.mlp_ab
        return tq.lora_swiglu(x, ag, bg, au, bu, gate, up, starts, adapters, self.scales, ranks=self.ranks)


def run(device="cuda", prompts=(70, 41, 150), steps=3, nodes=7, seed=0):
    """(attention half, gated half): largest differences between tree steps and decoding one by one, relative to the
    largest outputs."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=device).manual_seed(seed)
    i32 = dict(dtype=torch.int32, device=device)
    layer, count = Layer(rng, gen, device), len(prompts)
    adapters = torch.tensor([(0, 3, -1, 1)[s % 4] for s in range(count)], **i32)
    width = -(-(max(prompts) + (steps + 1) * nodes) // PAGE)
    pages = 2 * count * width
    caches = tq.kv8_cache(1, pages, KV_HEADS, DIM, PAGE, device=device)
    pools = [c[0] for c in caches]
    table, lengths, refs = tq.kv_state(2 * count, width, pages, device=device)
    seqs = torch.arange(count, **i32)

    def states(n):
        return torch.randn((n, HIDDEN), generator=gen, device=device).to(torch.bfloat16)

    def starts_of(counts):
        return torch.tensor([0] + list(np.cumsum(counts)), **i32)

    # the prompts, all in one call
    starts = starts_of(prompts)
    slots, granted = tq.cache_reserve(table, lengths, refs, PAGE, seqs, starts, sum(prompts))
    assert granted.all()
    x = states(sum(prompts))
    positions = torch.cat([torch.arange(n, **i32) for n in prompts])
    q = layer.heads(x, starts, adapters, positions, slots, pools)
    layer.out(tq.window_attention_kv8(q, *pools, table, lengths, starts, max(prompts), seq_ids=seqs), starts, adapters)
    layer.gated(x, starts, adapters)
    lengths[:count] = torch.tensor(prompts, **i32)
    assert tq.cache_fork_kv8(*caches, table, lengths, refs, seqs, seqs + count).all()

    # trees of drafts; of each one path is kept
    accepted = [[] for _ in prompts]
    starts = starts_of([nodes] * count)
    for _ in range(steps):
        trees = [draw_tree(rng, nodes) for _ in prompts]
        x = states(count * nodes)
        masks = torch.tensor([m for t in trees for m in t[1]], device=device)
        depth = torch.tensor([d for t in trees for d in t[2]], **i32)
        slots, granted = tq.cache_reserve(table, lengths, refs, PAGE, seqs, starts, count * nodes)
        assert granted.all()
        q = layer.heads(x, starts, adapters, lengths[:count].repeat_interleave(nodes) + depth, slots, pools)
        y = layer.out(tq.tree_attention_kv8(q, *pools, table, lengths, starts, masks, nodes, seq_ids=seqs), starts, adapters)
        z = layer.gated(x, starts, adapters)
        path, counts = torch.zeros((count, nodes), **i32), []
        for e, (_, mask, _) in enumerate(trees):
            end = int(rng.integers(nodes))
            kept = [i for i in range(nodes) if mask[end] >> i & 1]
            path[e, :len(kept)] = torch.tensor(kept, **i32)
            counts.append(len(kept))
            accepted[e] += [(x[e * nodes + i], y[e * nodes + i], z[e * nodes + i]) for i in kept]
        tq.cache_accept_kv8(*caches, table, lengths, seqs, path, torch.tensor(counts, **i32))

    # once more, token by token, in the forks
    worst, top = [0.0, 0.0], [0.0, 0.0]
    starts = torch.tensor([0, 1], **i32)
    for s in range(count):
        twin = torch.tensor([s + count], **i32)
        for x, *want in accepted[s]:
            slots, granted = tq.cache_reserve(table, lengths, refs, PAGE, twin, starts, 1)
            assert granted.all()
            mine = adapters[s:s + 1]
            q = layer.heads(x[None], starts, mine, lengths[s + count:s + count + 1].clone(), slots, pools)
            a = tq.window_attention_kv8(q, *pools, table, lengths, starts, 1, seq_ids=twin)
            got = layer.out(a, starts, mine), layer.gated(x[None], starts, mine)
            for i in range(2):
                worst[i] = max(worst[i], (got[i][0].float() - want[i].float()).abs().max().item())
                top[i] = max(top[i], want[i].float().abs().max().item())
            lengths[s + count] += 1
        assert lengths[s + count] == lengths[s]
    tq.cache_free(table, lengths, refs, torch.arange(2 * count, **i32))
    assert not refs.any()
    return worst[0] / top[0], worst[1] / top[1]


if __name__ == "__main__":
    print("trees against one by one, largest differences of the largest outputs: attention {:.2e}, gated {:.2e}".format(*run()))
