"""qk_norm_rope_kv8: queries against a 64-bit norm and rotation, the blocks
that tokens go into against a simulation of their scales and codes."""
import pytest
import torch

import trellis_coded_quantized_amd as tq
from tests import kv8_reference as r8
from tests import kv_reference as ref
from tests.kv8_reference import E4M3, E8M0

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, FP16 = torch.bfloat16, torch.float16


def consecutive(counts, firsts, P, pages, g):
    """Slots of sequences that hold `firsts` tokens and get `counts` more, pages in random order."""
    order, at, out = torch.randperm(pages, generator=g), 0, []
    for n, f in zip(counts, firsts):
        held = -(-(f + n) // P)
        row = order[at:at + held]
        at += held
        assert at <= pages
        j = f + torch.arange(n)
        out.append(row[j // P] * P + j % P)
    return torch.cat(out).int()


class World:
    """Inputs of a call and a cache of written blocks: codes of normal numbers, scales 2^-9 .. 2^-5."""

    def __init__(self, slots, hq, hkv, D, P, rot, dtype, pages, seed=0, far=100000):
        g = self.g = torch.Generator().manual_seed(seed)
        N = len(slots)
        self.dtype, self.P, self.D, self.slots = dtype, P, D, slots
        d = dict(q=torch.randn((N, hq, D), generator=g), k=torch.randn((N, hkv, D), generator=g),
                 v=torch.randn((N, hkv, D), generator=g), wq=1 + 0.2 * torch.randn(D, generator=g),
                 wk=1 + 0.2 * torch.randn(D, generator=g))
        for n, t in d.items():
            setattr(self, n, t.to(dtype))
        half = rot // 2
        self.inv = (1e6 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float()
        self.pos = torch.randint(0, far, (N,), generator=g).int()
        self.k8 = r8.codes((60 * torch.randn((pages, hkv, D // 16, P, 16), generator=g)).clamp(-448, 448))
        self.v8 = r8.codes((60 * torch.randn((pages, hkv, P // 16, D, 16), generator=g)).clamp(-448, 448))
        self.ks = torch.randint(118, 122, (pages, hkv, P // 16), generator=g, dtype=torch.uint8)
        self.vs = torch.randint(118, 122, (pages, hkv, P // 16), generator=g, dtype=torch.uint8)

    def run(self, eps=1e-6, interleaved=False, **kw):
        up = {n: getattr(self, n).to(DEV) for n in ("q", "k", "v", "wq", "wk", "pos", "inv", "slots")}
        self.pools = [self.k8.to(DEV).view(E4M3), self.v8.to(DEV).view(E4M3), self.ks.to(DEV).view(E8M0),
                      self.vs.to(DEV).view(E8M0)]
        return tq.qk_norm_rope_kv8(up["q"], up["k"], up["v"], up["wq"], up["wk"], up["pos"], up["inv"], up["slots"],
                                   *self.pools, eps=eps, interleaved=interleaved, **kw)

    def check(self, out, eps=1e-6, interleaved=False, queries=True):
        k8, v8, ks, vs = (p.view(torch.uint8).cpu() for p in self.pools)
        D, P, dt = self.D, self.P, self.dtype
        if queries:
            want, size = ref.norm_rope(self.q, self.wq, self.pos, self.inv, eps, interleaved)
            err = (out.cpu().double() - want).abs()
            assert (err <= ref.norm_rope_bound(want, size, D, dt)).all()
        keys, ksize = ref.norm_rope(self.k, self.wk, self.pos, self.inv, eps, interleaved)
        # f32 before the rounding to a code: the bound without its 16-bit half step
        slack = (D / 2 + 20) * ref.F32 * ksize
        want_k8, want_ks, want_v8, want_vs = (t.clone() for t in (self.k8, self.ks, self.v8, self.vs))
        known = self.slots.clone()
        known[(known < 0) | (known >= k8.shape[0] * P)] = -1
        for block, places in r8.by_blocks(known).items():
            tok, at = [t for t, _ in places], [p for _, p in places]
            code, byte = r8.append_block(*r8.block_of_values(self.v8, self.vs, block, P), at, self.v[tok].float(), dt)
            r8.put_block_of_values(want_v8, want_vs, block, P, code, byte)
            # keys: the scale as the 64-bit magnitudes want it (either one next to a border), the other rows' codes
            # as that scale makes them, the new rows' within half a step
            old, byte0 = r8.block_of_keys(self.k8, self.ks, block, P)
            got, byte = r8.block_of_keys(k8, ks, block, P)
            new = r8.tame(keys[tok], dt)
            top = r8.finite_top(new, (0, 2))
            lo, hi = r8.need_byte(top * (1 - 1e-5)), r8.need_byte(top * (1 + 1e-5))
            if 0 not in at:
                lo, hi = torch.maximum(lo, byte0), torch.maximum(hi, byte0)
            assert ((byte == lo) | (byte == hi)).all(), (block, byte, lo, hi)
            kept = [p for p in range(16) if p not in at]
            again = r8.rescale(old, byte0[:, None, None], byte[:, None, None])
            if 0 in at:
                again = old
            assert torch.equal(got[:, :, kept], again[:, :, kept]), block
            back = r8.value(got[:, :, at], byte[:, None, None]).permute(2, 0, 1)
            half_step = torch.maximum(new.abs() * 2.0 ** -4, 2.0 ** (byte.double() - 137)[None, :, None])
            assert torch.equal(back.isnan(), new.isnan())
            off = (back - new).abs() - half_step * (1 + 1e-6) - slack[tok]
            assert (torch.nan_to_num(off, nan=-1.0) <= 0).all(), (block, off.max())
            r8.put_block_of_keys(want_k8, want_ks, block, P, got, byte)
        # values to the bit, and nothing but the blocks' own bytes has changed
        assert torch.equal(vs, want_vs) and r8.same_codes(v8, want_v8)
        assert torch.equal(ks, want_ks) and r8.same_codes(k8, want_k8)


@pytest.mark.parametrize("hq,hkv,D,P,rot,dtype", [
    (24, 4, 256, 16, 64, BF16), (32, 8, 128, 64, 128, FP16), (16, 16, 64, 16, 32, BF16), (8, 1, 128, 256, 16, BF16),
    (1, 1, 64, 32, 64, FP16), (7, 7, 256, 128, 256, BF16), (6, 2, 64, 16, 0, FP16), (4, 2, 256, 32, 240, FP16)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("counts,firsts", [([1], [0]), ([1, 1, 1, 1], [3, 15, 16, 40]), ([37], [13]),
                                           ([5, 30, 1, 16, 2], [0, 9, 31, 16, 30])])
def test_parity(hq, hkv, D, P, rot, dtype, interleaved, counts, firsts):
    g = torch.Generator().manual_seed(sum(counts) + D)
    pages = sum(-(-(n + f) // P) for n, f in zip(counts, firsts)) + 2
    w = World(consecutive(counts, firsts, P, pages, g), hq, hkv, D, P, rot, dtype, pages, seed=D + P)
    w.check(w.run(interleaved=interleaved), interleaved=interleaved)


@pytest.mark.parametrize("N", [300, 5003])
def test_long_lists(N):
    """Several workgroups of runs; blocks that straddle them; single tokens between."""
    g = torch.Generator().manual_seed(N)
    counts, firsts = [N // 2, 1, 1, N // 3, 1, 17], [5, 0, 20, 0, 31, 8]
    pages = sum(-(-(n + f) // 64) for n, f in zip(counts, firsts)) + 2
    w = World(consecutive(counts, firsts, 64, pages, g), 2, 3, 64, 64, 32, BF16, pages, seed=N)
    w.check(w.run())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seed", range(8))
def test_lists_of_any_kind(D, seed):
    """Runs of any length at any place of a block, whole blocks, tokens that are not cached between them, and blocks
    that are much quieter than what comes."""
    g = torch.Generator().manual_seed(100 * seed + D)
    pick = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    P, pages = [16, 32, 64][seed % 3], 60
    blocks = torch.randperm(pages * P // 16, generator=g).tolist()
    slots = []
    for _ in range(pick(1, 40)):
        kind = pick(0, 3)
        if kind == 0:
            slots += [-1] * pick(1, 5)
            continue
        at = torch.randperm(16, generator=g)[:16 if kind == 1 else pick(1, 16) if kind == 2 else 1]
        block = blocks.pop()
        slots += [block * 16 + p for p in at.tolist()]
    w = World(torch.tensor(slots, dtype=torch.int32), 2, 3, D, P, 32, [BF16, FP16][seed % 2], pages, seed=seed)
    w.ks = torch.where(torch.rand(w.ks.shape, generator=g) < 0.3, torch.full_like(w.ks, 90), w.ks)
    w.vs = torch.where(torch.rand(w.vs.shape, generator=g) < 0.3, torch.full_like(w.vs, 90), w.vs)
    w.check(w.run())


def test_tokens_of_a_block_in_any_order_and_with_gaps():
    slots = torch.tensor([16 * 5 + p for p in (9, 2, 14, 3)] + [16 * 2 + p for p in range(15, -1, -1)] +
                         [16 * 7 + p for p in (0, 4)] + [16 * 5 + 16], dtype=torch.int32)
    for P in (16, 64):
        w = World(slots, 2, 2, 128, P, 64, BF16, 8 * 16 // P + 1, seed=P)
        w.check(w.run())


@pytest.mark.parametrize("D,P", [(64, 16), (128, 32), (256, 16)])
def test_scales_grow_with_louder_tokens(D, P):
    """One token at a time, each twice as loud as the one before: earlier ones are rounded again at every step."""
    g = torch.Generator().manual_seed(D)
    w = World(torch.zeros(1, dtype=torch.int32), 2, 2, D, P, 32, BF16, 4, seed=D)
    for step in range(16):
        w.slots = torch.tensor([2 * P + step], dtype=torch.int32)
        w.k = torch.randn((1, 2, D), generator=g).to(BF16)
        w.v = (torch.randn((1, 2, D), generator=g) * 2.0 ** (step - 8)).to(BF16)
        w.wk = torch.full((D,), 2.0 ** (step - 8), dtype=BF16)
        w.check(w.run())
        w.k8, w.v8, w.ks, w.vs = (p.view(torch.uint8).cpu() for p in w.pools)
    # a quieter token leaves the scale; a block's first slot begins it anew
    before = w.vs.clone()
    w.slots, w.v = torch.tensor([2 * P + 3], dtype=torch.int32), torch.full((1, 2, D), 2.0 ** -20, dtype=BF16)
    w.check(w.run())
    assert torch.equal(w.pools[3].view(torch.uint8).cpu(), before)
    w.slots = torch.tensor([2 * P], dtype=torch.int32)
    w.check(w.run())
    assert (w.pools[3].view(torch.uint8).cpu()[2, :, 0] < before[2, :, 0]).all()


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_zeros_infinities_nan_and_the_ends_of_the_type(dtype):
    slots = torch.tensor([0, 1, 2, 16, 17, 32, 48, 64, 80], dtype=torch.int32)
    w = World(slots, 2, 2, 64, 16, 0, dtype, 7)
    inf, nan, fi = float("inf"), float("nan"), torch.finfo(dtype)
    w.v[0, 0, 5], w.v[1, 0, 6], w.v[2, 1, 0] = inf, nan, -inf
    w.v[3] = 0
    w.v[4] = 0
    w.v[5, 0, 0], w.v[5, 1, 1] = fi.max, -fi.max
    w.v[6] = nan
    w.v[7] = fi.smallest_normal / 8 if dtype == FP16 else 1e-39
    w.v[8] = 448.0
    w.k[3] = 0                                               # a norm of zeros
    w.k[6, 0, 3] = nan                                       # its whole head
    out = w.run(eps=1e-6)
    w.check(out)
    vs = w.pools[3].view(torch.uint8).cpu()
    assert (vs[1] == 1).all() and (vs[5, :, 0] == 127).all()


def test_a_garbage_scale_is_replaced_at_a_first_slot():
    w = World(torch.tensor([32, 33], dtype=torch.int32), 2, 2, 64, 16, 0, BF16, 4)
    w.ks[:], w.vs[:] = 0xFF, 0xFF
    w.check(w.run())


def test_slots_outside_the_cache_are_not_written():
    pages = 4
    w = World(torch.tensor([-1, 3, pages * 16, 2 ** 31 - 1, -2 ** 31, 40], dtype=torch.int32), 4, 2, 128, 16, 64, FP16,
              pages)
    w.check(w.run())


def test_rows_are_independent_and_strided_views():
    w = World(torch.arange(9, dtype=torch.int32) + 5, 4, 2, 128, 16, 128, BF16, 3)
    x = torch.full((9, 8 * 128 + 64), float("nan"), dtype=BF16, device=DEV)
    x[:, 64:] = torch.cat([w.q.flatten(1), w.k.flatten(1), w.v.flatten(1)], 1).to(DEV)
    q, k, v = (x[:, a:b].unflatten(1, (-1, 128)) for a, b in ((64, 576), (576, 832), (832, 1088)))
    want = w.run()
    pools = w.pools
    again = [w.k8.to(DEV).view(E4M3), w.v8.to(DEV).view(E4M3), w.ks.to(DEV).view(E8M0), w.vs.to(DEV).view(E8M0)]
    out = tq.qk_norm_rope_kv8(q, k, v, w.wq.to(DEV), w.wk.to(DEV), w.pos.to(DEV), w.inv.to(DEV), w.slots.to(DEV), *again)
    assert torch.equal(out, want)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(pools, again))


def test_queries_equal_those_of_the_16_bit_append():
    w = World(torch.arange(33, dtype=torch.int32), 6, 2, 128, 16, 64, BF16, 3)
    out = w.run()
    kc, vc = tq.kv_cache(1, 3, 2, 128, 16, dtype=BF16, device=DEV)
    args = [t.to(DEV) for t in (w.q, w.k, w.v, w.wq, w.wk, w.pos, w.inv, w.slots)]
    assert torch.equal(out, tq.qk_norm_rope(*args, kc[0], vc[0]))


def test_far_pages():
    """A block past 2^32 bytes of a pool."""
    P, D, hkv = 16, 256, 4
    pages = (1 << 32) // (P * D * hkv) + 3
    pools = [torch.zeros(s, dtype=torch.uint8, device=DEV) for s in
             ((pages, hkv, D // 16, P, 16), (pages, hkv, P // 16, D, 16), (pages, hkv, 1), (pages, hkv, 1))]
    w = World(torch.arange(16, dtype=torch.int32), 4, hkv, D, P, 64, BF16, 2)
    w.run()
    args = [t.to(DEV) for t in (w.q, w.k, w.v, w.wq, w.wk, w.pos, w.inv)]
    tq.qk_norm_rope_kv8(*args, (w.slots + (pages - 1) * P).to(DEV), pools[0].view(E4M3), pools[1].view(E4M3),
                        pools[2].view(E8M0), pools[3].view(E8M0))
    for far, near in zip(pools, w.pools):
        assert torch.equal(far[-1], near.view(torch.uint8)[0])
        assert not far[:-1].any()


def test_other_stream_and_graph():
    w = World(torch.arange(20, dtype=torch.int32) + 7, 4, 2, 64, 16, 64, BF16, 3)
    want = w.run()
    first = [p.clone() for p in w.pools]
    args = [t.to(DEV) for t in (w.q, w.k, w.v, w.wq, w.wk, w.pos, w.inv, w.slots)]
    pools = [w.k8.to(DEV).view(E4M3), w.v8.to(DEV).view(E4M3), w.ks.to(DEV).view(E8M0), w.vs.to(DEV).view(E8M0)]
    begin = [p.clone() for p in pools]
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        tq.qk_norm_rope_kv8(*args, *pools, out=out)
    side.synchronize()
    same = lambda: torch.equal(out, want) and all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                                                  for a, b in zip(pools, first))
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.qk_norm_rope_kv8(*args, *pools, out=out)
    for _ in range(4):
        out.zero_()
        for p, b in zip(pools, begin):
            p.view(torch.uint8).copy_(b.view(torch.uint8))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same()


def test_no_tokens_and_refusals():
    w = World(torch.arange(2, dtype=torch.int32), 4, 2, 64, 16, 32, BF16, 2)
    w.run()
    args = [t.to(DEV) for t in (w.q, w.k, w.v, w.wq, w.wk, w.pos, w.inv, w.slots)]
    none = [t[:0] if i in (0, 1, 2, 5, 7) else t for i, t in enumerate(args)]
    assert tq.qk_norm_rope_kv8(*none, *w.pools).shape == (0, 4, 64)
    with pytest.raises(TypeError, match="q: dtype"):
        tq.qk_norm_rope_kv8(args[0].float(), *args[1:], *w.pools)
    with pytest.raises(TypeError, match="k: dtype"):
        tq.qk_norm_rope_kv8(args[0], args[1].half(), *args[2:], *w.pools)
    with pytest.raises(ValueError, match="slots"):
        tq.qk_norm_rope_kv8(*args[:7], args[7][:1], *w.pools)
    with pytest.raises(ValueError, match="k_scale: shape"):
        tq.qk_norm_rope_kv8(*args, w.pools[0], w.pools[1], w.pools[2][:1], w.pools[3])
    with pytest.raises(ValueError, match="v_scale must be contiguous"):
        tq.qk_norm_rope_kv8(*args, *w.pools[:3], w.pools[3].transpose(0, 1).contiguous().transpose(0, 1))
