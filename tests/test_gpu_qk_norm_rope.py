"""qk_norm_rope against a 64-bit norm and rotation, and the cache it fills
element by element against the documented layout."""
import pytest
import torch

import trellis_coded_quantized_amd as tq
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, FP16 = torch.bfloat16, torch.float16


def make(N, hq, hkv, D, P, rot, dtype, seed=0, far=100000, pages=None):
    g = torch.Generator().manual_seed(seed)
    pages = pages or -(-N // P) + 3
    d = dict(q=torch.randn((N, hq, D), generator=g), k=torch.randn((N, hkv, D), generator=g),
             v=torch.randn((N, hkv, D), generator=g), wq=1 + 0.2 * torch.randn(D, generator=g),
             wk=1 + 0.2 * torch.randn(D, generator=g))
    d = {n: t.to(dtype) for n, t in d.items()}
    half = rot // 2
    d["inv"] = (1e6 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float()
    d["pos"] = torch.randint(0, far, (N,), generator=g).int()
    d["slots"] = torch.randperm(pages * P, generator=g)[:N].int()
    d["kc"] = torch.full((pages, hkv, D // 8, P, 8), 5.0, dtype=dtype)
    d["vc"] = torch.full((pages, hkv, P // 8, D, 8), 5.0, dtype=dtype)
    return d


def check(d, out, kc, vc, dtype, eps, interleaved):
    """Queries, keys in the cache and values in the cache; everything else of the cache as it was."""
    D = d["q"].shape[2]
    for x, w, got in ((d["q"], d["wq"], out), (d["k"], d["wk"], None)):
        want, size = ref.norm_rope(x, w, d["pos"], d["inv"], eps, interleaved)
        if got is None:
            slots = d["slots"]
            keep = slots >= 0
            gk, gv = ref.take_tokens(kc.cpu(), vc.cpu(), slots[keep])
            got, want, size = gk, want[keep], size[keep]
            assert torch.equal(gv.view(torch.int16), d["v"][keep].view(torch.int16))
        err = (got.cpu().double() - want).abs()
        tol = ref.norm_rope_bound(want, size, D, dtype)
        assert (err <= tol).all(), f"worst {(err / tol).max():.3g} of the bound"
    slots = d["slots"][d["slots"] >= 0]
    rest_k, rest_v = kc.cpu().clone(), vc.cpu().clone()
    five = torch.full((slots.numel(),) + tuple(d["k"].shape[1:]), 5.0, dtype=dtype)
    ref.put_tokens(rest_k, rest_v, slots, five, five)
    assert (rest_k == 5).all() and (rest_v == 5).all()


def run(d, eps=1e-6, interleaved=False, **kw):
    dev = {n: t.to(DEV) for n, t in d.items()}
    out = tq.qk_norm_rope(dev["q"], dev["k"], dev["v"], dev["wq"], dev["wk"], dev["pos"], dev["inv"], dev["slots"],
                          dev["kc"], dev["vc"], eps=eps, interleaved=interleaved, **kw)
    return out, dev["kc"], dev["vc"]


@pytest.mark.parametrize("hq,hkv,D,P,rot,dtype", [
    (24, 4, 256, 16, 64, BF16), (32, 8, 128, 64, 128, FP16), (16, 16, 64, 16, 32, BF16), (8, 1, 128, 256, 16, BF16),
    (1, 1, 64, 32, 64, FP16), (7, 7, 256, 128, 256, BF16), (6, 2, 64, 16, 0, FP16), (16, 2, 256, 32, 240, FP16)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N", [1, 4, 37])
def test_parity(hq, hkv, D, P, rot, dtype, interleaved, N):
    d = make(N, hq, hkv, D, P, rot, dtype, seed=N + D)
    check(d, *run(d, interleaved=interleaved), dtype, 1e-6, interleaved)


@pytest.mark.parametrize("first,N", [(0, 64), (3, 64), (13, 200), (8, 9), (15, 1)])
@pytest.mark.parametrize("P", [16, 64])
def test_runs_of_consecutive_slots(first, N, P):
    """A chunk that starts anywhere in a page and crosses pages in random order."""
    d = make(N, 4, 2, 128, P, 128, BF16, seed=N + first)
    order = torch.randperm(d["kc"].shape[0])
    at = first + torch.arange(N)
    keep = at // P < len(order)
    d["slots"] = torch.where(keep, order[(at // P).clamp(max=len(order) - 1)] * P + at % P, -1).int()
    check(d, *run(d), BF16, 1e-6, False)


def test_far_positions_and_negative_ones():
    d = make(5, 2, 1, 64, 16, 64, BF16)
    d["pos"] = torch.tensor([2 ** 31 - 1, 10 ** 9 + 7, 1, 0, -12345], dtype=torch.int32)
    check(d, *run(d), BF16, 1e-6, False)


def test_slots_outside_the_cache_are_not_written():
    d = make(6, 4, 2, 128, 16, 64, FP16)
    pages = d["kc"].shape[0]
    d["slots"] = torch.tensor([-1, 3, pages * 16, 2 ** 31 - 1, -2 ** 31, 40], dtype=torch.int32)
    out, kc, vc = run(d)
    d["slots"] = torch.tensor([-1, 3, -1, -1, -1, 40], dtype=torch.int32)
    check(d, out, kc, vc, FP16, 1e-6, False)


def test_zero_and_extreme_heads():
    d = make(4, 2, 1, 64, 16, 32, BF16)
    d["q"][0], d["k"][0] = 0, 0
    d["q"][1] *= 1e-15
    d["q"][2] *= 1e15
    check(d, *run(d, eps=1e-6), BF16, 1e-6, False)


def test_views_of_one_projection():
    d = make(9, 4, 2, 128, 16, 128, BF16)
    x = torch.full((9, 8 * 128 + 64), float("nan"), dtype=BF16, device=DEV)
    x[:, 64:] = torch.cat([d["q"].flatten(1), d["k"].flatten(1), d["v"].flatten(1)], 1).to(DEV)
    q, k, v = (x[:, a:b].unflatten(1, (-1, 128)) for a, b in ((64, 576), (576, 832), (832, 1088)))
    dev = {n: t.to(DEV) for n, t in d.items()}
    out = tq.qk_norm_rope(q, k, v, dev["wq"], dev["wk"], dev["pos"], dev["inv"], dev["slots"], dev["kc"], dev["vc"])
    check(d, out, dev["kc"], dev["vc"], BF16, 1e-6, False)


def test_offsets_past_32_bits():
    P, D = 64, 256
    pages = (1 << 32) // (P * D) + 4
    d = make(3, 2, 1, D, P, 64, BF16, pages=4)
    dev = {n: t.to(DEV) for n, t in d.items()}
    kc = torch.full((pages, 1, D // 8, P, 8), 5.0, dtype=BF16, device=DEV)
    vc = torch.full((pages, 1, P // 8, D, 8), 5.0, dtype=BF16, device=DEV)
    slots = dev["slots"] + (pages - 4) * P
    out = tq.qk_norm_rope(dev["q"], dev["k"], dev["v"], dev["wq"], dev["wk"], dev["pos"], dev["inv"], slots, kc, vc)
    check(d, out, kc[-4:], vc[-4:], BF16, 1e-6, False)
    assert (kc[:-4] == 5).all() and (vc[:-4] == 5).all()


def test_stream_and_graph():
    d = make(70, 8, 2, 128, 16, 64, BF16)
    dev = {n: t.to(DEV) for n, t in d.items()}
    args = [dev[n] for n in ("q", "k", "v", "wq", "wk", "pos", "inv", "slots", "kc", "vc")]
    want = tq.qk_norm_rope(*args)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tq.qk_norm_rope(*args, out=out)
    for _ in range(3):
        dev["pos"] += 11
        eager = tq.qk_norm_rope(*args)
        kc = dev["kc"].clone()
        dev["kc"].zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16))
        slots = dev["slots"]
        assert torch.equal(ref.take_tokens(dev["kc"], dev["vc"], slots)[0], ref.take_tokens(kc, dev["vc"], slots)[0])


def test_refusals():
    d = make(3, 4, 2, 128, 16, 64, BF16)
    dev = {n: t.to(DEV) for n, t in d.items()}
    a = [dev[n] for n in ("q", "k", "v", "wq", "wk", "pos", "inv", "slots", "kc", "vc")]

    def call(**kw):
        b = list(a)
        for i, x in kw.items():
            b[int(i[1:])] = x
        return tq.qk_norm_rope(*b)

    with pytest.raises(tq.TrellisError, match="rotary_dim"):
        call(_6=dev["inv"][:4].contiguous())
    with pytest.raises(ValueError, match="tokens"):
        call(_1=dev["k"][:2])
    with pytest.raises(ValueError, match="entries"):
        call(_3=dev["wq"][:64])
    with pytest.raises(TypeError):
        call(_5=dev["pos"].long())
    with pytest.raises(ValueError, match="shape"):
        call(_7=dev["slots"][:2])
    with pytest.raises(TypeError):
        call(_0=dev["q"].half())
    with pytest.raises(tq.TrellisError, match="eps"):
        tq.qk_norm_rope(*a, eps=float("nan"))
    with pytest.raises(ValueError, match="shape"):
        tq.qk_norm_rope(*a, out=torch.empty((3, 4, 64), dtype=BF16, device=DEV))
    assert tq.qk_norm_rope(*[x[:0] if i in (0, 1, 2, 5, 7) else x for i, x in enumerate(a)]).shape == (0, 4, 128)
