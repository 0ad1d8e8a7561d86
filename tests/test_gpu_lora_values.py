"""lora_add and lora_swiglu at the ends of their numbers: infinities in the
factors, sums that need every bit of A x, numbers next to the largest."""
import pytest
import torch

import trellis_coded_quantized_amd as tq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
INF, NAN = float("inf"), float("nan")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def pieces(t):
    """f64 numbers of at most 24 bits -> three bf16 numbers that add up to each, along a new last dimension."""
    out = []
    for _ in range(3):
        out.append(t.to(F32).to(BF16))
        t = t - out[-1].double()
    assert not t.any()
    return torch.stack(out, -1)


def exactly(t, rank):
    """x bf16 [M, 8 M] and A [1, rank, 8 M] whose products A x are t [M, rank], rounded nowhere: row m has ones in
    eight columns of its own, where A holds t's pieces."""
    M = t.shape[0]
    x, a = torch.zeros((M, 8 * M), dtype=BF16), torch.zeros((1, rank, 8 * M), dtype=BF16)
    for m in range(M):
        x[m, 8 * m:8 * m + 3] = 1
        a[0, :, 8 * m:8 * m + 3] = pieces(t[m])
    return x, a


def add(x, a, b, y, scale=1.0, ranks=None):
    out = tq.lora_add(x.to(DEV), [a.to(DEV)], [b.to(DEV)], [y.to(DEV)], ints([0, x.shape[0]]), ints([0]),
                      torch.tensor([scale], device=DEV), ranks=None if ranks is None else ints(ranks))[0]
    return out.cpu()


def gated(x, a, b, gate, up, scale=1.0):
    """Both projections have the same factors."""
    a, b = a.to(DEV), b.to(DEV)
    return tq.lora_swiglu(x.to(DEV), a, b, a, b, gate.to(DEV), up.to(DEV), ints([0, x.shape[0]]), ints([0]),
                          torch.tensor([scale], device=DEV)).cpu()


def agree(got, want, tol):
    """The same infinities and NaN, the others within tol."""
    got = got.double()
    assert torch.equal(got.isnan(), want.isnan())
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf])
    rest = ~(inf | want.isnan())
    assert not rest.any() or ((got - want).abs() - tol)[rest].max() <= 0


# ---- infinities in B ------------------------------------------------------
# t: on a bf16 number, above one, below one, above one by a second part that is
# itself above a bf16 number, and zero
T = [1.5, 1 + 2.0 ** -9, 1 - 2.0 ** -10, 1 + 2.0 ** -7 + 2.0 ** -9 + 2.0 ** -18, 0.0]


@pytest.mark.parametrize("rank", [8, 16, 32, 64])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [5, 70])
@pytest.mark.parametrize("R", [8, 200, 77])
def test_infinite_entries_of_b(rank, dtype, M, R):
    g = torch.Generator().manual_seed(rank + M + R)
    at = torch.randint(0, len(T), (M, rank), generator=g)
    t = torch.tensor(T, dtype=torch.float64)[at] * (torch.randint(0, 2, (M, rank), generator=g) * 2 - 1)
    b = torch.randn((1, R, rank), generator=g).to(BF16)
    for i in range(0, R, 3):                                   # rows of B with one infinity, two, or a NaN
        for _ in range(1 + i % 2):
            b[0, i, int(torch.randint(0, rank, (1,), generator=g))] = [INF, -INF, INF, NAN][i // 3 % 4]
    y = torch.randn((M, R), generator=g).to(dtype)
    x, a = exactly(t, rank)
    d = (t[:, None] * b[0].double()).sum(-1)                   # a product for each, so that none hides another's NaN
    # t enters with 16 bits at least, sums are f32
    off = (t.abs()[:, None] * b[0].double().abs()).sum(-1) * (2.0 ** -17 + (3 * rank + 4) * 2.0 ** -24)
    want = y.double() + d
    agree(add(x, a, b, y), want, off + (U[dtype] + 2.0 ** -23) * want.abs())

    up = torch.randn((M, R), generator=g).to(dtype)
    gate = y.double() + d
    silu, u = gate / (1 + torch.exp(-gate)), up.double() + d
    want = silu * u
    # |silu'| <= 1.1; the exponential's argument is rounded
    tol = 1.1 * off * u.abs() + silu.abs() * off + 1.2 * off * off + (gate.abs() + 8) * 2.0 ** -22 * want.abs()
    agree(gated(x, a, b, y, up), want, 1.01 * tol + U[BF16] * want.abs() + 1e-38)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [3, 70])
def test_infinities_and_nan_of_a_and_y(dtype, M):
    """A's reach the outputs through the ranks that hold them, y's stay where they are."""
    g = torch.Generator().manual_seed(M)
    x = torch.randint(-2, 3, (M, 32), generator=g).to(BF16)
    a = torch.randint(-2, 3, (1, 8, 32), generator=g).to(BF16)
    a[0, 1, 5], a[0, 3, 7], a[0, 6, 2] = INF, -INF, NAN
    b = torch.zeros((1, 24, 8), dtype=BF16)
    for i in range(24):                                        # one rank each: zeros of B meet what t has of others
        b[0, i, i % 8] = 1 - 2 * (i // 8 % 2)
    y = torch.randint(-3, 4, (M, 24), generator=g).to(dtype)
    y[0, 1], y[1, 2], y[2, 3] = INF, NAN, -INF
    # element by element: sums of products as they stand, infinities and NaN among them
    t = (x.double()[:, None] * a[0].double()).sum(-1)
    want = y.double() + (t[:, None] * b[0].double()).sum(-1)
    agree(add(x, a, b, y), want, torch.zeros_like(want))
    a[0, 6, 2] = 1
    t = (x.double()[:, None] * a[0].double()).sum(-1)
    want = y.double() + (t[:, None] * b[0].double()).sum(-1)
    agree(add(x, a, b, y), want, torch.zeros_like(want))
    agree(add(x, a, b, y, ranks=[1]), y.double() + t[:, :1] * b[0, :, 0].double(), torch.zeros_like(want))


@pytest.mark.parametrize("rank", [8, 64])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_infinite_entries_of_b_beside_many_single_rows(rank, dtype):
    """Wide outputs of many short entries, where a wave takes several blocks of columns."""
    g = torch.Generator().manual_seed(rank)
    M, R = 64, 8192
    t = torch.tensor([[1 + 2.0 ** -9] * rank], dtype=torch.float64)
    x, a = exactly(t, rank)
    x = x.expand(M, -1).contiguous()
    b = torch.randn((1, R, rank), generator=g).to(BF16)
    bad = torch.randint(0, R, (R // 50,), generator=g)
    b[0, bad, bad % rank] = INF
    b[0, bad[::2], bad[::2] % rank] = -INF
    starts, ids, s = ints(list(range(M + 1))), ints([0] * M), torch.ones(1, device=DEV)
    y = torch.randn((M, R), generator=g).to(dtype)
    d = (t * b[0].double()).sum(-1)
    off = (t * b[0].double().abs()).sum(-1) * (2.0 ** -17 + (3 * rank + 4) * 2.0 ** -24)
    want = y.double() + d
    got = tq.lora_add(x.to(DEV), [a.to(DEV)], [b.to(DEV)], [y.to(DEV)], starts, ids, s)[0].cpu()
    agree(got, want, off + (U[dtype] + 2.0 ** -23) * want.abs())
    a, b, y = a.to(DEV), b.to(DEV), y.to(DEV)
    got = tq.lora_swiglu(x.to(DEV), a, b, a, b, y, y, starts, ids, s).cpu()
    silu = want / (1 + torch.exp(-want))
    tol = (1.1 * want.abs() + silu.abs()) * off + 1.2 * off * off + (want.abs() + 8) * 2.0 ** -22 * (silu * want).abs()
    agree(got, silu * want, 1.01 * tol + U[BF16] * (silu * want).abs() + 1e-38)


def test_what_lies_past_a_rank_stays_out():
    """NaN past the adapter's rank beside infinities within it."""
    t = torch.tensor([[1 + 2.0 ** -9] * 16], dtype=torch.float64)
    b = torch.ones((1, 40, 16), dtype=BF16)
    b[0, ::2, 4], b[0, :, 5:] = INF, NAN
    x, a = exactly(t, 16)
    a[0, 5:] = NAN
    out = add(x, a, b, torch.zeros((1, 40)), ranks=[5])
    assert (out[0, ::2] == INF).all() and (out[0, 1::2] == 5 * (1 + 2.0 ** -9)).all()


# ---- every bit of A x -----------------------------------------------------
# Whole numbers below 2^24 in every sum, in any order: f32 is exact, and a bit
# of t that is dropped shows where another rank or y takes the rest away.

@pytest.mark.parametrize("rank", [8, 16, 32, 64])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [3, 70])
@pytest.mark.parametrize("R", [24, 31])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -8])
def test_sums_that_cancel(rank, dtype, M, R, scale):
    g = torch.Generator().manual_seed(rank + M + R)
    t = torch.randint(-2 ** 22, 2 ** 22, (M, rank), generator=g).double()
    t[:, 1::2] = t[:, ::2] + torch.randint(-300, 301, (M, rank // 2), generator=g)
    b = torch.zeros((1, R, rank), dtype=BF16)                  # three ranks at most: two that cancel, and any one
    for i in range(R):
        j = int(torch.randint(0, rank // 2, (1,), generator=g)) * 2
        b[0, i, j], b[0, i, j + 1] = 1, -1
        if i % 3 == 2:
            b[0, i, int(torch.randint(0, rank, (1,), generator=g))] = 1
    x, a = exactly(t, rank)
    d = t @ b[0].double().T * scale
    y = (-d).to(dtype)
    y[:, ::2] = 0
    want = y.double() + d                                      # exact in f64, and in f32
    assert torch.equal(want.float().double(), want)
    assert torch.equal(add(x, a, b, y, scale), want.to(F32).to(dtype))
    if scale < 1:
        silu = want / (1 + torch.exp(-want))
        tol = (want.abs() + 8) * 2.0 ** -22 + U[BF16]
        keep = want > -80                                      # where the exponential is far from f32's end
        agree(gated(x, a, b, y, y, scale)[keep], (silu * want)[keep], 1.01 * (tol * (silu * want).abs())[keep])


@pytest.mark.parametrize("rank", [8, 64])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [2, 50])
def test_finite_sums_past_the_largest_bf16(rank, dtype, M):
    """A x = +-2^127 (2 - 2^-10) and neighbours, times small numbers: f32 holds all of it, bf16 only up to 2^127 (2 - 2^-8)."""
    tops = torch.tensor([2 - 2.0 ** -7, 2 - 2.0 ** -8, 2 - 2.0 ** -10, 2 - 2.0 ** -23], dtype=torch.float64)
    t = torch.zeros((M, rank), dtype=torch.float64)
    t[:, rank - 2] = tops.repeat(M)[:M] * torch.tensor([1.0, 1, 1, 1, -1, -1, -1, -1]).repeat(M)[:M] * 2.0 ** 63
    x = torch.zeros((M, 8 * M), dtype=BF16)
    a = torch.zeros((1, rank, 8 * M), dtype=BF16)
    for m in range(M):                                         # two pieces of at most 16 bits and one below
        x[m, 8 * m:8 * m + 3] = 2.0 ** 64
        one = t[m, rank - 2].clamp(-(2 - 2.0 ** -7) * 2.0 ** 63, (2 - 2.0 ** -7) * 2.0 ** 63)
        a[0, rank - 2, 8 * m] = one
        a[0, rank - 2, 8 * m + 1:8 * m + 3] = pieces(t[m, rank - 2] - one)[:2]
    b = torch.zeros((1, 24, rank), dtype=BF16)
    b[0, :, rank - 2] = 2.0 ** -torch.arange(4.0, 28.0)
    want = t * 2.0 ** 64 @ b[0].double().T
    assert torch.equal(add(x, a, b, torch.zeros((M, 24), dtype=dtype)), want.to(F32).to(dtype))


# ---- the gated activation -------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [1, 70])
@pytest.mark.parametrize("loud", [0, 60, 100])
@pytest.mark.parametrize("R", [512, 509])
def test_gates_far_below_zero(dtype, M, loud, R):
    """-60 to -130: e^-g passes the end of f32, g / (1 + e^-g) times an up of 2^loud does not reach zero, or is a
    subnormal number."""
    g = torch.Generator().manual_seed(loud + M)
    gate = (-60 - 70 * torch.rand((M, R), generator=g)).to(dtype)
    up = (torch.randn((M, R), generator=g) * 2.0 ** loud).to(dtype)
    x, a, b = torch.zeros((M, 8), dtype=BF16), torch.zeros((1, 8, 8), dtype=BF16), torch.zeros((1, R, 8), dtype=BF16)
    want = gate.double() / (1 + torch.exp(-gate.double())) * up.double()
    # the exponential's argument is rounded; half a step of bf16, of its subnormals 2^-133, and a few of f32's 2^-149
    tol = (U[BF16] + (gate.double().abs() + 8) * 2.0 ** -22) * want.abs() + 2.0 ** -134 + 2.0 ** -146
    agree(gated(x, a, b, gate, up), want, tol)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gates_of_any_size(dtype):
    gate = torch.tensor([[0.0, -0.0, 1e-30, -1e-30, 1e30, -1e30, 88.0, -88.0, 300.0, -300.0, INF, NAN, 3e38, -3e38]]).to(dtype)
    x, a = torch.zeros((1, 8), dtype=BF16), torch.zeros((1, 8, 8), dtype=BF16)
    b = torch.zeros((1, gate.shape[1], 8), dtype=BF16)
    for size in (1.0, -3.0, 1e-20, 0.0):
        up = torch.full_like(gate, size)
        want = torch.nn.functional.silu(gate.double()) * up.double()
        got = gated(x, a, b, gate, up)
        tol = (U[BF16] + torch.minimum(gate.double().abs() + 8, torch.tensor(400.0)) * 2.0 ** -22) * want.abs() + 2.0 ** -133
        agree(got, want.to(BF16).double(), tol + U[BF16] * want.abs())


# ---- no adapter -----------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts", [[1, 2], [70, 30]])
@pytest.mark.parametrize("R", [40, 33])
def test_rows_without_an_adapter_keep_every_bit(dtype, counts, R):
    """Zeros of either sign, subnormal numbers, infinities: out = y, beside an entry with an adapter."""
    M = sum(counts)
    y = torch.tensor([0.0, -0.0, 2.0 ** -133, -2.0 ** -133, INF, -INF, 1.5]).repeat(M * R)[:M * R].view(M, R).to(dtype)
    x, a, b = torch.ones((M, 8), dtype=BF16), torch.ones((1, 8, 8), dtype=BF16), torch.ones((1, R, 8), dtype=BF16)
    kind = torch.int16 if dtype is BF16 else torch.int32
    for ids, rows in (([-1, 0], slice(0, counts[0])), ([-1, -1], slice(0, M)), ([0, 1], slice(counts[0], M))):
        out = tq.lora_add(x.to(DEV), [a.to(DEV)], [b.to(DEV)], [y.to(DEV)], ints([0, counts[0], M]), ints(ids),
                          torch.ones(1, device=DEV))[0].cpu()
        assert torch.equal(out[rows].view(kind), y[rows].view(kind))


# ---- lists of long and short entries ---------------------------------------

@pytest.mark.parametrize("rank", [8, 16, 32, 64])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("more", [0, 1])
def test_a_prompt_among_single_rows(rank, dtype, more):
    """Means of 128 / rank rows, and one row more: single rows, none, and one entry with all the others."""
    g = torch.Generator().manual_seed(rank + more)
    entries, pool, C, R = 24, 5, 264, 136
    M = 128 // rank * entries + more
    counts = [1] * entries
    counts[3], counts[7] = 0, M - (entries - 2)
    ids = [i % (pool + 1) - 1 for i in range(entries)]
    x, y = torch.randn((M, C), generator=g).to(BF16), torch.randn((M, R), generator=g).to(dtype)
    a, b = torch.randn((pool, rank, C), generator=g).to(BF16), torch.randn((pool, R, rank), generator=g).to(BF16)
    scales = torch.rand(pool, generator=g) + 0.5
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    d, off = torch.zeros((M, R), dtype=torch.float64), torch.zeros((M, R), dtype=torch.float64)
    for e, i in enumerate(ids):
        if i < 0:
            continue
        rows, s = slice(starts[e], starts[e + 1]), scales[i].double()
        d[rows] = s * (x[rows].double() @ a[i].double().T) @ b[i].double().T
        # sums of C products and at most 32 chunks, the scale, and sums over 3 ranks
        off[rows] = (s * (x[rows].double().abs() @ a[i].double().abs().T) @ b[i].double().abs().T *
                     (C + 32 + 1 + 3 * rank + 4) * 2.0 ** -24)
    args = [ints(starts), ints(ids), scales.to(DEV)]
    want = y.double() + d
    got = tq.lora_add(x.to(DEV), [a.to(DEV)], [b.to(DEV)], [y.to(DEV)], *args)[0].cpu()
    agree(got, want, U[dtype] * want.abs() + (off + 2.0 ** -24 * want.abs()) * (1 + 2 * U[dtype]))
    a, b = a.to(DEV), b.to(DEV)
    got = tq.lora_swiglu(x.to(DEV), a, b, a, b, y.to(DEV), y.to(DEV), *args).cpu()
    silu, off = want / (1 + torch.exp(-want)), off + 2.0 ** -24 * want.abs()
    tol = (1.1 * want.abs() + silu.abs()) * off + 1.2 * off * off + (want.abs() + 8) * 2.0 ** -22 * (silu * want).abs()
    agree(got, silu * want, 1.01 * tol + U[BF16] * (silu * want).abs() + 1e-38)
