"""lora_add and lora_swiglu against 64-bit products, with the bounds that f32
sums and the output's rounding leave."""
import pytest
import torch

import trellis_coded_quantized_amd as tq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
NAN = float("nan")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Case:
    """counts[e] rows and adapter ids[e] of every entry; `first` rows before the first one and `after` behind the last."""

    def __init__(self, counts, ids, C, Rs, rank, dtype, pool=6, ranks=None, first=0, after=0, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.counts, self.ids, self.C, self.Rs, self.rank, self.dtype = counts, ids, C, Rs, rank, dtype
        self.starts = [first]
        for n in counts:
            self.starts.append(self.starts[-1] + n)
        self.M = self.starts[-1] + after
        self.x = torch.randn((self.M, C), generator=g).to(BF16)
        self.a = [torch.randn((pool, rank, C), generator=g).to(BF16) for _ in Rs]
        self.b = [torch.randn((pool, R, rank), generator=g).to(BF16) for R in Rs]
        self.y = [torch.randn((self.M, R), generator=g).to(dtype) for R in Rs]
        self.scales = torch.rand(pool, generator=g) + 0.5
        self.ranks = [rank] * pool if ranks is None else ranks
        for i, r in enumerate(self.ranks):                     # what lies past an adapter's rank is not looked at
            for a, b in zip(self.a, self.b):
                a[i, r:], b[i, :, r:] = NAN, NAN

    def up(self):
        x = [t.to(DEV) for t in self.a], [t.to(DEV) for t in self.b], [t.to(DEV) for t in self.y]
        return (self.x.to(DEV), *x, ints(self.starts), ints(self.ids), self.scales.to(DEV))

    def kw(self):
        return {} if all(r == self.rank for r in self.ranks) else dict(ranks=ints(self.ranks))

    def deltas(self, k):
        """(the adapters' part of target k, what f32 may be off in it), 64 bits."""
        d = torch.zeros((self.M, self.Rs[k]), dtype=torch.float64)
        off = torch.zeros_like(d)
        for e, i in enumerate(self.ids):
            r = self.ranks[i] if 0 <= i < len(self.ranks) else 0
            if r == 0:
                continue
            rows = slice(self.starts[e], self.starts[e + 1])
            x, a, b = self.x[rows].double(), self.a[k][i, :r].double(), self.b[k][i, :, :r].double()
            s = self.scales[i].double()
            d[rows] = s * (x @ a.T) @ b.T
            # the sums of A x (C products and at most 32 column chunks), the scale, the three parts of a sum's 24 bits,
            # and the sums over 3 r products
            off[rows] = s * (x.abs() @ a.abs().T) @ b.abs().T * (self.C + 32 + 1 + 1 + 3 * r + 4) * 2.0 ** -24
        return d, off

    def check_add(self, outs, before=None):
        for k, out in enumerate(outs):
            d, off = self.deltas(k)
            y = self.y[k].double()
            want = y + d
            tol = U[self.dtype] * want.abs() + (off + 2.0 ** -24 * want.abs()) * (1 + 2 * U[self.dtype])
            got = out.double().cpu()
            lo, hi = self.starts[0], self.starts[-1]
            err = (got - want).abs()[lo:hi] - tol[lo:hi]
            assert not err.numel() or err.max() <= 0, f"target {k}: worst over the bound by {err.max():.3g}"
            for e, i in enumerate(self.ids):                   # no adapter: y itself
                if not 0 <= i < len(self.ranks) or self.ranks[i] == 0:
                    rows = slice(self.starts[e], self.starts[e + 1])
                    assert torch.equal(out[rows].cpu(), self.y[k][rows])
            if before is not None:
                assert torch.equal(out[:lo].cpu(), before[k][:lo]) and torch.equal(out[hi:].cpu(), before[k][hi:])

    def check_swiglu(self, out):
        (dg, og), (du, ou) = self.deltas(0), self.deltas(1)
        g, u = self.y[0].double() + dg, self.y[1].double() + du
        og, ou = og + 2.0 ** -24 * g.abs(), ou + 2.0 ** -24 * u.abs()
        silu = g / (1 + torch.exp(-g))
        want = silu * u
        # |silu'| <= 1.1; the exponential: its argument's rounding, |g| 2^-23, and a few units of its own
        tol = U[BF16] * want.abs() + (1.1 * og * u.abs() + silu.abs() * ou + (g.abs() + 8) * 2.0 ** -22 * want.abs()) * 1.01
        lo, hi = self.starts[0], self.starts[-1]
        err = ((out.double().cpu() - want).abs() - tol - 1e-38)[lo:hi]
        assert err.max() <= 0, f"worst over the bound by {err.max():.3g}"


@pytest.mark.parametrize("rank", [8, 16, 32, 64])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts,ids", [([1], [2]), ([1, 1, 1, 1, 1], [0, -1, 5, 0, 2]), ([4, 0, 13, 1], [1, 2, 3, 4]),
                                        ([70, 1, 130, 0, 65], [3, 0, -1, 1, 5])])
@pytest.mark.parametrize("C,Rs", [(256, [96, 40, 8]), (640, [512])])
def test_add(rank, dtype, counts, ids, C, Rs):
    c = Case(counts, ids, C, Rs, rank, dtype, seed=rank + C)
    c.check_add(tq.lora_add(*c.up()))


@pytest.mark.parametrize("rank", [16, 64])
@pytest.mark.parametrize("counts", [[1, 2], [100, 3]])
def test_four_projections_of_unlike_widths(rank, counts):
    c = Case(counts, [2, 0], 1024, [1024, 8, 264, 2048], rank, BF16, ranks=[rank, 3, rank - 5, 1, 1, 1], seed=rank)
    c.check_add(tq.lora_add(*c.up(), **c.kw()))


@pytest.mark.parametrize("seed", range(12))
def test_lists_of_any_kind(seed):
    """Entries from none to hundreds of rows, most of them short or most of them long, any ranks and widths."""
    g = torch.Generator().manual_seed(seed)
    pick = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    entries, rank, pool = pick(1, 40), [8, 16, 32, 64][seed % 4], pick(1, 9)
    counts = [pick(0, [1, 3, 40, 200][pick(0, 3)]) for _ in range(entries)]
    ids = [pick(-1, pool) for _ in range(entries)]
    Rs = [pick(1, 90) * [1, 8][pick(0, 1)] for _ in range(pick(1, 4))]
    c = Case(counts, ids, 8 * pick(1, 100), Rs, rank, [BF16, F32][pick(0, 1)], pool=pool,
             ranks=[pick(0, rank) for _ in range(pool)], first=pick(0, 5), after=pick(0, 5), seed=seed)
    filled = [torch.full_like(y, 9.0) for y in c.up()[3]]
    c.check_add(tq.lora_add(*c.up(), **c.kw(), outs=filled), before=[torch.full_like(y, 9.0) for y in c.y])


@pytest.mark.parametrize("rank", [8, 16, 32, 64])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts,ids", [([1], [2]), ([3, 1, 2], [0, -1, 5]), ([70, 1, 130], [3, 9, 1])])
def test_swiglu(rank, dtype, counts, ids):
    c = Case(counts, ids, 256, [200, 200], rank, dtype, seed=rank)
    x, a, b, y, starts, adapters, scales = c.up()
    c.check_swiglu(tq.lora_swiglu(x, a[0], b[0], a[1], b[1], y[0], y[1], starts, adapters, scales))


@pytest.mark.parametrize("C", [8, 24, 40, 264, 1000, 5120])
@pytest.mark.parametrize("counts", [[1, 2], [90]])
def test_odd_widths(C, counts):
    """Inputs that end inside a step, outputs that end inside a granule, rows that are not 16-byte aligned."""
    for Rs in ([1], [7, 129, 33], [331]):
        for dtype in (BF16, F32):
            c = Case(counts, [1, 0][:len(counts)], C, Rs, 16, dtype, seed=C)
            c.check_add(tq.lora_add(*c.up()))
    c = Case(counts, [1, 0][:len(counts)], C, [331, 331], 32, BF16, seed=C)
    x, a, b, y, *rest = c.up()
    c.check_swiglu(tq.lora_swiglu(x, a[0], b[0], a[1], b[1], y[0], y[1], *rest))


@pytest.mark.parametrize("counts", [[1, 1, 1, 1, 1, 1], [40, 3, 64, 9, 1, 100]])
@pytest.mark.parametrize("rank", [8, 16, 32, 64])
def test_ranks_below_the_pools(counts, rank):
    c = Case(counts, [0, 1, 2, 3, 4, 5], 320, [72, 16], rank, F32, ranks=[rank, 0, 1, rank // 2, rank - 1, rank // 2 + 3])
    c.check_add(tq.lora_add(*c.up(), **c.kw()))
    c = Case(counts, [0, 1, 2, 3, 4, 5], 320, [72, 72], rank, BF16, ranks=[rank, 0, 1, rank // 2, rank - 1, rank // 2 + 3])
    x, a, b, y, *rest = c.up()
    c.check_swiglu(tq.lora_swiglu(x, a[0], b[0], a[1], b[1], y[0], y[1], *rest, **c.kw()))


@pytest.mark.parametrize("counts", [[2, 1, 3], [80, 1, 70]])
def test_in_place_and_rows_of_no_entry(counts):
    for ids in ([0, -1, 3], [-1, -1, -1], [6, 2, -7]):
        c = Case(counts, ids, 128, [64, 24], 16, BF16, first=3, after=5)
        args = c.up()
        outs = tq.lora_add(*args, outs=args[3])
        assert outs is args[3]
        c.check_add(outs, before=c.y)
        filled = [torch.full_like(y, 9.0) for y in args[3]]
        args = c.up()
        c.check_add(tq.lora_add(*args, outs=filled), before=[torch.full_like(y, 9.0) for y in c.y])
        mixed = [args[3][0], torch.full_like(args[3][1], 9.0)]
        c.check_add(tq.lora_add(*args, outs=mixed))


@pytest.mark.parametrize("counts", [[2, 1], [80, 20]])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_views_of_one_projection(counts, dtype):
    """Queries, keys and values in one tensor, inputs in a wider one; in place."""
    for Rs in ([64, 16, 16], [61, 13, 9]):
        c = Case(counts, [4, 1], 128, Rs, 16, dtype)
        x, a, b, y, *rest = c.up()
        wide = torch.full((c.M, 8 + 128 + 8), NAN, dtype=BF16, device=DEV)
        wide[:, 8:136] = x
        qkv = torch.cat(y, 1)
        views = list(qkv.split(Rs, 1))
        guard = torch.full((c.M, sum(Rs) + 3), 5.0, dtype=dtype, device=DEV)
        guard[:, :-3] = qkv
        outs = tq.lora_add(wide[:, 8:136], a, b, views, *rest, outs=list(guard[:, :-3].split(Rs, 1)))
        c.check_add(outs)
        assert (guard[:, -3:] == 5.0).all()
        tq.lora_add(wide[:, 8:136], a, b, views, *rest, outs=views)
        assert torch.equal(qkv, guard[:, :-3])


def test_swiglu_into_its_gate():
    c = Case([3, 70], [1, -1], 128, [96, 96], 16, BF16)
    x, a, b, y, *rest = c.up()
    want = tq.lora_swiglu(x, a[0], b[0], a[1], b[1], y[0], y[1], *rest)
    c.check_swiglu(want)
    got = tq.lora_swiglu(x, a[0], b[0], a[1], b[1], y[0], y[1], *rest, out=y[0])
    assert torch.equal(got, want) and got is y[0]


@pytest.mark.parametrize("counts", [[1, 2, 1], [70, 2, 3]])
def test_infinities_and_nan_stay_in_their_rows(counts):
    c = Case(counts, [0, 1, 2], 256, [48], 32, F32)
    bad = counts[0]
    c.x[bad, 17], c.x[bad + 1, 3] = float("inf"), NAN
    out = tq.lora_add(*c.up())[0].cpu()
    assert not torch.isfinite(out[bad:bad + 2]).any()
    c.x[bad:bad + 2] = 0
    keep = [m for m in range(c.M) if m not in (bad, bad + 1)]
    d, off = c.deltas(0)
    want = c.y[0].double() + d
    assert ((out.double() - want).abs() <= off + 2.0 ** -23 * want.abs())[keep].all()


def test_an_infinite_sum_stays_infinite():
    """t = A x past bf16's end, times zeros and ones: infinities where f32 has them, no NaN."""
    c = Case([1], [0], 8, [8], 8, F32, pool=1)
    c.x[:], c.a[0][:], c.b[0][:] = 0, 0, 0
    c.x[0, 0], c.a[0][0, 0, 0], c.b[0][0, :, 0] = 2.0 ** 100, 2.0 ** 100, 1.0
    out = tq.lora_add(*c.up())[0]
    assert (out == float("inf")).all()


@pytest.mark.parametrize("entries,most", [(200, 3), (130, 90), (1000, 1)])
def test_many_entries(entries, most):
    g = torch.Generator().manual_seed(entries)
    counts = torch.randint(0, most + 1, (entries,), generator=g).tolist()
    ids = torch.randint(-2, 8, (entries,), generator=g).tolist()
    c = Case(counts, ids, 64, [40], 16, F32)
    c.check_add(tq.lora_add(*c.up()))


@pytest.mark.parametrize("filled", [0x00, 0xFF])
def test_workspaces_of_any_content(filled):
    for counts in ([1, 0, 2], [100, 0, 33]):
        c = Case(counts, [2, 1, 0], 2048, [64, 64], 16, F32, ranks=[16, 9, 3, 16, 16, 16])
        ws = torch.full((1 << 24,), filled, dtype=torch.uint8, device=DEV)
        c.check_add(tq.lora_add(*c.up(), **c.kw(), workspace=ws))


def test_large_pools_reach_past_32_bits():
    """The last adapter of a pool of more than 2^32 bytes."""
    C, R, rank = 5120, 64, 64
    pool = (1 << 32) // (2 * C * rank) + 2
    c = Case([2], [0], C, [R], rank, F32, pool=1)
    x, a, b, y, starts, _, scales = c.up()
    big = torch.empty((pool, rank, C), dtype=BF16, device=DEV)
    big[-1] = a[0][0]
    bb = torch.empty((pool, R, rank), dtype=BF16, device=DEV)
    bb[-1] = b[0][0]
    c.check_add(tq.lora_add(x, [big], [bb], y, starts, ints([pool - 1]), scales.expand(pool).contiguous()))


@pytest.mark.parametrize("counts", [[1, 2], [90, 40]])
def test_other_stream_and_graph(counts):
    c = Case(counts, [1, 4], 512, [64, 32], 16, BF16)
    x, a, b, y, starts, adapters, scales = c.up()
    want = tq.lora_add(x, a, b, y, starts, adapters, scales)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = tq.lora_add(x, a, b, y, starts, adapters, scales)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    outs = [torch.empty_like(t) for t in y]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.lora_add(x, a, b, y, starts, adapters, scales, outs=outs)
    for ids in ([1, 4], [-1, 2], [0, 0], [5, -1]):
        adapters.copy_(ints(ids))                              # the graph reads who has which adapter on the device
        for o in outs:
            o.zero_()
        eager = tq.lora_add(x, a, b, y, starts, adapters, scales)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, eager))


@pytest.mark.parametrize("counts", [[3, 70], [1, 1, 2]])
def test_swiglu_into_its_up_and_add_into_x(counts):
    c = Case(counts, [1, -1, 2][:len(counts)], 96, [96, 96], 16, BF16)
    x, a, b, y, *rest = c.up()
    want = tq.lora_swiglu(x, a[0], b[0], a[1], b[1], y[0], y[1], *rest)
    got = tq.lora_swiglu(x, a[0], b[0], a[1], b[1], y[0], y[1], *rest, out=y[1])
    assert torch.equal(got, want) and got is y[1]
    (want,) = tq.lora_add(x, a[:1], b[:1], y[:1], *rest)
    (got,) = tq.lora_add(x, a[:1], b[:1], y[:1], *rest, outs=[x])              # x has been read by then
    assert torch.equal(got, want) and got is x


def test_two_calls_at_once():
    cases = [Case([90, 40], [1, 4], 512, [640, 32], 16, BF16, seed=1), Case([1] * 40, [0, 3] * 20, 512, [640, 32], 16, BF16, seed=2)]
    args = [c.up() for c in cases]
    want = [tq.lora_add(*t) for t in args]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for k, (t, side) in enumerate(zip(args, streams)):
            with torch.cuda.stream(side):
                got[k].append(tq.lora_add(*t))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(p, q) for outs in got[k] for p, q in zip(outs, want[k]))


def test_starts_outside_the_rows_touch_nothing_outside():
    c = Case([3, 4], [0, 1], 64, [16], 8, F32)
    x, a, b, y, _, adapters, scales = c.up()
    for starts in ([-5, 3, 900], [2 ** 31 - 1, -2 ** 31, 7], [5, 2, 7]):
        out = tq.lora_add(x, a, b, y, ints(starts), adapters, scales, outs=[torch.zeros_like(y[0])])[0]
        assert torch.isfinite(out).all()


def test_no_rows_and_refusals():
    c = Case([2], [0], 64, [16], 8, BF16)
    x, a, b, y, starts, adapters, scales = c.up()
    out = tq.lora_add(x[:0], a, b, [y[0][:0]], ints([0, 0]), adapters, scales)
    assert out[0].shape == (0, 16)
    with pytest.raises(TypeError, match="x: dtype"):
        tq.lora_add(x.half(), a, b, y, starts, adapters, scales)
    with pytest.raises(TypeError, match=r"y: dtype"):
        tq.lora_add(x, a, b, [y[0].half()], starts, adapters, scales)
    with pytest.raises(TypeError, match=r"ys\[1\]: dtype"):
        tq.lora_add(x, a * 2, b * 2, [y[0], y[0].float()], starts, adapters, scales)
    with pytest.raises(ValueError, match=r"a\[0\]: shape"):
        tq.lora_add(x, [a[0][:, :, :56].contiguous()], b, y, starts, adapters, scales)
    with pytest.raises(ValueError, match=r"b\[0\]: shape"):
        tq.lora_add(x, a, [b[0][:-1]], y, starts, adapters, scales)
    with pytest.raises(ValueError, match="adapters: shape"):
        tq.lora_add(x, a, b, y, starts, ints([0, 1]), scales)
    with pytest.raises(ValueError, match="scales: shape"):
        tq.lora_add(x, a, b, y, starts, adapters, scales[:-1])
    with pytest.raises(ValueError, match="row must be contiguous"):
        tq.lora_add(x, a, b, [y[0].T.contiguous().T], starts, adapters, scales)
    with pytest.raises(tq.TrellisError, match="x_stride"):
        tq.lora_add(x[:1].expand(2, 64), a, b, y, starts, adapters, scales)
    with pytest.raises(tq.TrellisError, match="out_stride"):
        tq.lora_add(x, a, b, y, starts, adapters, scales, outs=[y[0][:1].expand(2, 16)])
    with pytest.raises(tq.TrellisError, match="workspace"):
        tq.lora_add(x, a, b, y, starts, adapters, scales, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    with pytest.raises(tq.TrellisError, match="gate has"):
        tq.lora_swiglu(x, a[0], b[0], a[0], b[0][:, :8].contiguous(), y[0], y[0][:, :8], starts, adapters, scales)
