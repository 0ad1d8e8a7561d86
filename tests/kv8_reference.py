"""Plain forms of the 8-bit cache's blocks, and a batch over such a cache, for
its tests.  No code here is shared with the library."""
import torch

from tests import kv_reference as ref
from tests.test_gpu_attention import Case

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
TOP = {torch.bfloat16: 1.875 * 2.0 ** 127, torch.float16: 61440.0}
NAN_CODE, NAN_SCALE = 0x7F, 0xFF


def codes(x):
    """f32 magnitudes of at most 448 (or NaN) -> e4m3 bytes, nearest, ties to even."""
    return x.float().to(E4M3).view(torch.uint8)


def value(code, byte):
    """Bytes and the scales' bytes (broadcast) -> f64."""
    return code.view(E4M3).double() * 2.0 ** (byte.double() - 127)


def same_codes(a, b):
    """Whether two arrays of codes stand for the same values.  e4m3 has two NaN, 0x7F and 0xFF (S.1111.111), and the
    contract says NaN, not which."""
    nan = [(x & 0x7F) == NAN_CODE for x in (a, b)]
    return torch.equal(nan[0], nan[1]) and torch.equal(a.masked_fill(nan[0], 0), b.masked_fill(nan[0], 0))


def need_byte(top):
    """The smallest b of 1..254 with 448 * 2^(b - 127) >= top, elementwise over f64."""
    b = torch.ones_like(top)
    for v in range(2, 255):
        b = torch.where(448.0 * 2.0 ** (v - 1 - 127) < top, torch.full_like(b, v), b)
    return b.to(torch.uint8)


def tame(x, dtype):
    """What a new element counts as: infinities are NaN, magnitudes end at the type's top."""
    x = torch.where(torch.isinf(x), torch.full_like(x, float("nan")), x)
    return x.clamp(-TOP[dtype], TOP[dtype])


def finite_top(x, dims):
    return torch.nan_to_num(x.abs(), nan=0.0).amax(dims)


def rescale(code, old, new):
    """Codes of blocks rounded again from scales `old` to `new` (bytes, broadcast)."""
    return codes((code.view(E4M3).double() * 2.0 ** (old.double() - new.double())).float())


def by_blocks(slots):
    """{block: [(token, place in the block)]} of a list of slots."""
    out = {}
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            out.setdefault(s // 16, []).append((t, s % 16))
    return out


def append_block(code, byte, places, new, dtype):
    """One block of one kind: code [heads, D, 16], byte [heads], new [n, heads, D] (f32) at `places`.
    Returns (codes, bytes)."""
    new = tame(new, dtype)
    need = need_byte(finite_top(new, (0, 2)).double())
    anew = 0 in places
    now = need if anew else torch.maximum(byte, need)
    out = code.clone() if anew else rescale(code, byte[:, None, None], now[:, None, None])
    out = torch.where((now == byte)[:, None, None], code, out)
    scaled = codes((new.double() * 2.0 ** (127 - now.double())[None, :, None]).float())
    for i, p in enumerate(places):
        out[:, :, p] = scaled[i]
    return out, now


def block_of_keys(k8, ks, block, P):
    """(codes [heads, D, 16], bytes [heads]) of a block of a key pool [pages, heads, D/16, P, 16]."""
    page, at = block * 16 // P, block * 16 % P
    return k8[page, :, :, at:at + 16].permute(0, 1, 3, 2).flatten(1, 2), ks[page, :, at // 16]


def block_of_values(v8, vs, block, P):
    page, at = block * 16 // P, block * 16 % P
    return v8[page, :, at // 16], vs[page, :, at // 16]


def put_block_of_keys(k8, ks, block, P, code, byte):
    page, at = block * 16 // P, block * 16 % P
    k8[page, :, :, at:at + 16] = code.unflatten(1, (-1, 16)).permute(0, 1, 3, 2)
    ks[page, :, at // 16] = byte


def put_block_of_values(v8, vs, block, P, code, byte):
    page, at = block * 16 // P, block * 16 % P
    v8[page, :, at // 16] = code
    vs[page, :, at // 16] = byte


class Case8(Case):
    """Case over a cache in 8 bits: keys and values are codes times their block's scale; where no token was written
    codes are NaN, and so are the scales of blocks without a token."""

    def __init__(self, *args, exponents=(119, 123), **kw):
        super().__init__(*args, **kw)
        pages, P, D = self.k.shape[0], self.P, self.D
        self.k8 = torch.full((pages, self.hkv, D // 16, P, 16), NAN_CODE, dtype=torch.uint8)
        self.v8 = torch.full((pages, self.hkv, P // 16, D, 16), NAN_CODE, dtype=torch.uint8)
        self.ks = torch.full((pages, self.hkv, P // 16), NAN_SCALE, dtype=torch.uint8)
        self.vs = torch.full((pages, self.hkv, P // 16), NAN_SCALE, dtype=torch.uint8)
        self.kb, self.vb = [], []
        for e in range(len(self.ids)):
            n = self.keys[e].shape[0]
            for values, bytes_ in ((self.keys, self.kb), (self.vals, self.vb)):
                b = torch.randint(*exponents, (-(-n // 16), self.hkv), generator=self.g, dtype=torch.uint8)
                per = b.repeat_interleave(16, 0)[:n, :, None]
                code = codes(64 * values[e].float())
                values[e] = value(code, per).to(self.dtype)
                bytes_.append(b)

    def to_device(self, dev="cuda:0"):
        P = self.P
        for e, s in enumerate(self.ids):
            n = self.keys[e].shape[0]
            slots = ref.seq_slots(self.table[s], n, P)
            page, off = slots // P, slots % P
            for values, bytes_, pool, scales in ((self.keys, self.kb, self.k8, self.ks),
                                                 (self.vals, self.vb, self.v8, self.vs)):
                per = bytes_[e].repeat_interleave(16, 0)[:n]
                code = codes((values[e].double() * 2.0 ** (127 - per.double())[:, :, None]).float())
                if pool is self.k8:
                    pool[page, :, :, off] = code.unflatten(2, (-1, 16))
                else:
                    pool[page, :, off // 16, :, off % 16] = code
                scales[page, :, off // 16] = per
        self.args = (self.k8.to(dev).view(E4M3), self.v8.to(dev).view(E4M3), self.ks.to(dev).view(E8M0),
                     self.vs.to(dev).view(E8M0), self.table.to(dev), self.lengths.to(dev),
                     torch.tensor(self.starts, dtype=torch.int32, device=dev))
        return self.q.to(dev)
