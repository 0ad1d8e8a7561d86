"""Plain 64-bit forms of the attention operators and page operations, and the
error bounds their tests use.  No code here is shared with the library."""
import torch

HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16)}
F32 = 2.0 ** -24


def put_tokens(k_cache, v_cache, slots, k, v):
    """Write k, v [n, heads, D] (any dtype of the caches) at slots, elementwise from the documented addresses."""
    P, D = k_cache.shape[-2], v_cache.shape[-2]
    page, t = (slots // P).long(), (slots % P).long()
    for d in range(D):
        k_cache[page, :, d // 8, t, d % 8] = k[:, :, d]
        v_cache[page, :, t // 8, d, t % 8] = v[:, :, d]


def take_tokens(k_cache, v_cache, slots):
    """(k, v) [n, heads, D] of the slots."""
    P = k_cache.shape[-2]
    page, t = (slots // P).long(), (slots % P).long()
    k = k_cache[page, :, :, t]                     # [n, heads, D/8, 8]
    v = v_cache[page, :, t // 8, :, t % 8]         # [n, heads, D]
    return k.flatten(2), v


def seq_slots(table_row, n, P):
    j = torch.arange(n, device=table_row.device)
    return table_row[j // P].long() * P + j % P


def attend(q, k, v, see, scale):
    """One entry, 64 bits.  q [n, Hq, D], k, v [keys, Hkv, D], see [n, keys].
    Returns (out [n, Hq, D], tolerance parts): sums of |weight * value|, of
    |value| per unit sum, and the largest sum of |q k| of a row's keys."""
    n, hq, D = q.shape
    g = hq // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    kk = k.repeat_interleave(g, 1).permute(1, 2, 0)
    vv = v.repeat_interleave(g, 1).permute(1, 0, 2)
    qq = q.permute(1, 0, 2)
    s = torch.matmul(qq, kk) * scale                                  # [Hq, n, keys]
    s = torch.where(see[None], s, torch.full_like(s, -torch.inf))
    m = s.amax(-1, keepdim=True) if s.shape[-1] else torch.full(s.shape[:-1] + (1,), -torch.inf, dtype=s.dtype)
    p = torch.exp(s - torch.where(m == -torch.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    ld = torch.where(l == 0, torch.ones_like(l), l)
    p = p / ld
    vz = torch.nan_to_num(vv, nan=0.0, posinf=0.0, neginf=0.0)
    o = torch.matmul(p, vz)
    bad = ~torch.isfinite(vv)
    if bad.any():                                                     # visible infinities and NaN, row by row
        for h, key, d in bad.nonzero().tolist():
            rows = see[:, key]
            o[h, rows, d] = o[h, rows, d] + vv[h, key, d]
    a = torch.matmul(p, vz.abs())
    b = torch.matmul(see.double()[None].expand(hq, -1, -1), vz.abs()) / ld
    qk = torch.matmul(qq.abs(), torch.nan_to_num(kk, nan=0.0, posinf=0.0, neginf=0.0).abs()) * scale
    qk = torch.where(see[None], qk, torch.zeros_like(qk))
    top = qk.amax(-1, keepdim=True) if qk.shape[-1] else torch.zeros_like(l)
    return [x.permute(1, 0, 2) for x in (o, a, b, top)]


def attention_bound(o, a, b, top, keys, D, dtype):
    """What a correct kernel may be off, per output:
      u |o|            the output's rounding (u: half a step of its type)
      u a              each weight's rounding, a = sum p |v|
      2 e a            scores in f32: a weight changes by e = (D + 4) 2^-24 of the sum of |q k| (products, sums,
                       scaling, exponent), and so does the sum that divides
      2 (keys + 16) 2^-24 a   f32 sums over the keys
      fp16 only: weights under 2^-14 step by 2^-24 (half: 2^-25), outputs likewise
    """
    u = HALF_STEP[dtype]
    e = (D + 4) * F32 * top
    tol = u * o.abs() + u * a + 2 * e * a + 2 * (keys + 16) * F32 * a
    tol = tol * (1 + 4 * u)
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25 * b + 2.0 ** -25
    return tol + 1e-38


def assert_attention(got, parts, keys, D, what=""):
    o, a, b, top = [x.cpu() for x in parts]
    g = got.double().cpu()
    fine = torch.isfinite(o)
    assert torch.equal(torch.isnan(g), torch.isnan(o)), f"{what}: NaN at other places"
    inf = torch.isinf(o)
    assert torch.equal(g[inf], o[inf]), f"{what}: infinities differ"
    tol = attention_bound(o, a, b, top.expand_as(o), keys, D, got.dtype)
    over = ((g - o).abs() - tol)[fine]
    assert over.numel() == 0 or over.max() <= 0, \
        f"{what}: {int((over > 0).sum())} of {over.numel()} outputs off, worst by {over.max():.3g}"


def tree_see(ctx, masks, keys):
    see = torch.zeros((len(masks), keys), dtype=torch.bool)
    see[:, :min(ctx, keys)] = True
    for i, m in enumerate(masks):
        for node in range(64):
            if (m >> node) & 1 and node < len(masks) and ctx + node < keys:
                see[i, ctx + node] = True
    return see


def window_see(ctx, n, keys, window, sinks):
    p = ctx + torch.arange(n)[:, None]
    j = torch.arange(keys)[None]
    see = j <= p
    if window:
        see = see & ((p - j < window) | (j < sinks))
    return see


def norm_rope(x, w, pos, inv_freq, eps, interleaved):
    """64-bit norm and rotation of x [n, heads, D]; also the bound's parts."""
    x, w = x.double(), w.double()
    y = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * w
    half = inv_freq.numel()
    ang = pos.double()[:, None] * inv_freq.double()[None]
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    out = y.clone()
    size = y.abs()
    if half:
        ia = torch.arange(half) * 2 if interleaved else torch.arange(half)
        ib = ia + 1 if interleaved else ia + half
        A, B = y[..., ia], y[..., ib]
        out[..., ia], out[..., ib] = A * c - B * s, B * c + A * s
        size = size.clone()
        size[..., ia] = size[..., ib] = A.abs() + B.abs()
    return out, size


def norm_rope_bound(out, size, D, dtype):
    """Output rounding, and f32: the sum of squares (D terms, halved by the root), root, division, two products with
    inv and w, cos and sin (at most 2^-21 off in all: argument rounding 2^-24 * pi, function 4 ulp), the rotation."""
    return HALF_STEP[dtype] * out.abs() * (1 + 1e-3) + (D / 2 + 8 + 8 + 4) * F32 * size + \
        (2.0 ** -25 if dtype == torch.float16 else 1e-40)


# ---- page operations, in whole numbers ------------------------------------

class Pages:
    """Lists in place of the device state."""

    def __init__(self, table, lengths, refs, P):
        self.table, self.lengths, self.refs, self.P = table.tolist(), lengths.tolist(), refs.tolist(), P
        self.width = len(self.table[0])

    def ok(self, p):
        return 0 <= p < len(self.refs)

    def free_list(self):
        return [i for i, r in enumerate(self.refs) if r == 0]

    def reserve(self, seq_ids, counts):
        free, asked, granted, slots = self.free_list(), 0, [], []
        done = set()
        for s, n in zip(seq_ids, counts):
            known = 0 <= s < len(self.table) and s not in done
            done.add(s)
            if not known or self.lengths[s] + n > self.width * self.P:
                granted.append(0)
                slots += [-1] * n
                continue
            at = range(self.lengths[s], self.lengths[s] + n)
            missing = sorted({a // self.P for a in at if not self.ok(self.table[s][a // self.P])})
            first, asked = asked, asked + len(missing)
            if asked > len(free):
                granted.append(0)
                slots += [-1] * n
                continue
            for j, p in enumerate(missing):
                self.table[s][p] = free[first + j]
                self.refs[free[first + j]] = 1
            granted.append(1)
            slots += [self.table[s][a // self.P] * self.P + a % self.P for a in at]
        return slots, granted

    def fork(self, parents, children):
        """Returns (granted, page copies (from, to))."""
        rows, lens = [list(r) for r in self.table], list(self.lengths)
        seen, jobs = set(), []
        for par, kid in zip(parents, children):
            known = 0 <= kid < len(rows) and kid not in seen
            if known:
                seen.add(kid)
            if not known:
                jobs.append(None)
            elif par == kid:
                jobs.append("same")
            else:
                full, part = (0, 0) if not 0 <= par < len(rows) else divmod(lens[par], self.P)
                good = 0 <= par < len(rows) and (not part or self.ok(rows[par][full]))
                jobs.append((par, kid, full, part, good))
        for j in jobs:
            if isinstance(j, tuple):
                for p in rows[j[1]]:
                    if self.ok(p):
                        self.refs[p] -= 1
        held = set()
        for j in jobs:
            if isinstance(j, tuple) and j[4]:
                for p in rows[j[0]][:j[2]]:
                    if self.ok(p):
                        self.refs[p] += 1
                if j[3]:
                    held.add(rows[j[0]][j[2]])
        free = [p for p in self.free_list() if p not in held]
        granted, copies, rank = [], [], 0
        for j in jobs:
            if not isinstance(j, tuple):
                granted.append(1 if j == "same" else 0)
                continue
            par, kid, full, part, good = j
            self.table[kid], self.lengths[kid] = [-1] * self.width, 0
            if not good:
                granted.append(0)
                continue
            if part:
                rank += 1
                if rank > len(free):
                    granted.append(0)
                    for p in rows[par][:full]:
                        if self.ok(p):
                            self.refs[p] -= 1
                    continue
                new = free[rank - 1]
                self.refs[new] = 1
                copies.append((rows[par][full], new))
                self.table[kid][full] = new
            for x in range(full):
                self.table[kid][x] = rows[par][x] if self.ok(rows[par][x]) else -1
            self.lengths[kid] = lens[par]
            granted.append(1)
        return granted, copies

    def free(self, seq_ids):
        for s in seq_ids:
            if 0 <= s < len(self.table):
                for p in self.table[s]:
                    if self.ok(p):
                        self.refs[p] -= 1
                self.table[s], self.lengths[s] = [-1] * self.width, 0

    def same_as(self, table, lengths, refs):
        assert table.tolist() == self.table
        assert lengths.tolist() == self.lengths
        assert refs.tolist() == self.refs
