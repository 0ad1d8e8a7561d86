"""Host-side checks of the attention and cache entry points (no GPU, no
launches): every invalid call is refused with a status and a message."""
import ctypes

import pytest

import trellis_coded_quantized_amd as tq

FAKE = ctypes.c_void_p(1 << 20)          # aligned, never dereferenced
MIS = ctypes.c_void_p((1 << 20) + 2)


def cache(k=1 << 20, v=1 << 20, pages=64, layers=1, heads=4, head_dim=128, page_size=16, dtype=tq.KV_BF16):
    return tq.KvCache(k, v, pages, layers, heads, head_dim, page_size, dtype)


def state(table=1 << 20, lengths=1 << 20, refs=1 << 20, seqs=8, width=4):
    return tq.KvState(table, lengths, refs, seqs, width)


def said(needle):
    msg = tq.load_library().trellis_last_error().decode()
    assert needle in msg, msg


BAD_CACHE = [
    (dict(head_dim=96), tq.EUNSUPPORTED, "head_dim=96"), (dict(page_size=8), tq.EUNSUPPORTED, "page_size=8"),
    (dict(page_size=24), tq.EUNSUPPORTED, "page_size=24"), (dict(page_size=512), tq.EUNSUPPORTED, "page_size=512"),
    (dict(dtype=2), tq.EINVAL, "dtype=2"), (dict(heads=0), tq.EINVAL, "heads=0"), (dict(pages=0), tq.EINVAL, "pages=0"),
    (dict(pages=1 << 27), tq.EINVAL, "pages="), (dict(layers=0), tq.EINVAL, "layers=0"),
    (dict(k=None), tq.EINVAL, "cache k is NULL"), (dict(v=(1 << 20) + 8), tq.EINVAL, "cache v not 16-byte"),
]
BAD_STATE = [
    (dict(seqs=0), "table of 0"), (dict(width=0), "x 0"), (dict(width=1 << 27), "width * page_size"),
    (dict(table=None), "table is NULL"), (dict(lengths=(1 << 20) + 4), "lengths not 16-byte"),
]


def window(c=None, s=None, q=FAKE, stride=32 * 128, ids=None, n=2, starts=FAKE, tokens=5, hq=32, max_q=3, win=0,
           sinks=0, scale=0.1, out=FAKE, ws=FAKE, wsb=1 << 40):
    c, s = c or cache(), s or state()
    return tq.load_library().trellis_window_attention(q, stride, ctypes.byref(c), ctypes.byref(s), ids, n, starts,
                                                      tokens, hq, max_q, win, sinks, scale, out, ws, wsb, None)


def tree(c=None, s=None, anc=FAKE, max_q=3, hq=32, tokens=5, scale=0.1, wsb=1 << 40):
    c, s = c or cache(), s or state()
    return tq.load_library().trellis_tree_attention(FAKE, 32 * 128, ctypes.byref(c), ctypes.byref(s), None, 2, FAKE, anc,
                                                    tokens, hq, max_q, scale, FAKE, FAKE, wsb, None)


@pytest.mark.parametrize("kw,status,needle", BAD_CACHE)
def test_bad_caches(kw, status, needle):
    assert window(c=cache(**kw)) == status
    said(needle)
    assert tree(c=cache(**kw)) == status
    said(needle)


@pytest.mark.parametrize("kw,needle", BAD_STATE)
def test_bad_states(kw, needle):
    assert window(s=state(**kw)) == tq.EINVAL
    said(needle)


@pytest.mark.parametrize("kw,needle", [
    (dict(hq=33), "heads_q=33"), (dict(hq=0), "heads_q=0"), (dict(stride=32 * 128 + 4), "q_stride"),
    (dict(stride=128), "q_stride"), (dict(n=0), "n=0"), (dict(n=70000), "n=70000"), (dict(max_q=0), "max_q=0"),
    (dict(win=-1), "window=-1"), (dict(sinks=-2), "sinks=-2"), (dict(scale=0.0), "scale"),
    (dict(scale=-1.0), "scale"), (dict(scale=float("inf")), "scale"), (dict(scale=float("nan")), "scale"),
    (dict(q=None), "q is NULL"), (dict(q=MIS), "q not 16-byte"), (dict(starts=None), "q_start is NULL"),
    (dict(ids=MIS), "seq_ids not 4-byte"), (dict(out=None), "out is NULL"), (dict(tokens=-1), "tokens=-1"),
    (dict(c=cache(layers=2)), "one layer")])
def test_window_refusals(kw, needle):
    assert window(**kw) == tq.EINVAL
    said(needle)


def test_tree_refusals():
    assert tree(max_q=65) == tq.EINVAL
    said("max_q=65")
    assert tree(anc=None) == tq.EINVAL
    said("ancestors is NULL")


def test_workspace_sizes():
    lib = tq.load_library()
    c, s = cache(), state(width=1000)
    cp, sp = ctypes.byref(c), ctypes.byref(s)
    need = lib.trellis_tree_attention_workspace_bytes(cp, sp, 2, 5, 32, 3)
    assert need > 0
    assert tree(s=s, wsb=need - 1) == tq.EWORKSPACE
    said("workspace")
    assert window(s=s, ws=MIS) == tq.EINVAL
    said("workspace not 256-byte")
    assert lib.trellis_tree_attention_workspace_bytes(cp, sp, 2, 0, 32, 3) == 0
    assert lib.trellis_tree_attention_workspace_bytes(cp, sp, 2, 5, 31, 3) == 0
    assert lib.trellis_window_attention_workspace_bytes(cp, sp, 2, 5, 32, 3, -1, 0) == 0
    assert window(tokens=0, q=None, out=None, ws=None, wsb=0) == tq.OK


def rope(c=None, q=FAKE, qs=32 * 128, ks=512, vs=512, wq=FAKE, pos=FAKE, inv=FAKE, rot=64, eps=1e-6, slots=FAKE,
         out=FAKE, tokens=3, hq=32):
    c = c or cache()
    return tq.load_library().trellis_qk_norm_rope(q, qs, FAKE, ks, FAKE, vs, wq, FAKE, pos, inv, rot, 0, eps, slots, out,
                                                  ctypes.byref(c), tokens, hq, None)


@pytest.mark.parametrize("kw,status,needle", BAD_CACHE)
def test_rope_bad_caches(kw, status, needle):
    assert rope(c=cache(**kw)) == status
    said(needle)


@pytest.mark.parametrize("kw,needle", [
    (dict(qs=32 * 128 + 1), "q_stride"), (dict(ks=504), "k_stride"), (dict(vs=0), "v_stride"), (dict(rot=8), "rotary_dim"),
    (dict(rot=144), "rotary_dim"), (dict(rot=-16), "rotary_dim"), (dict(eps=-1.0), "eps"), (dict(hq=0), "heads_q"),
    (dict(eps=float("nan")), "eps"), (dict(inv=None), "inv_freq"), (dict(pos=None), "positions"), (dict(slots=MIS), "slots"),
    (dict(out=MIS), "out"), (dict(wq=MIS), "q_weight"), (dict(tokens=1 << 31), "tokens")])
def test_rope_refusals(kw, needle):
    assert rope(**kw) == tq.EINVAL
    said(needle)


def test_rope_no_tokens():
    assert rope(tokens=0, q=None, out=None) == tq.OK


def test_cache_calls():
    lib = tq.load_library()
    c, s = cache(layers=3), state()
    cp, sp = ctypes.byref(c), ctypes.byref(s)
    for n in (0, 1025):
        assert lib.trellis_cache_free(cp, sp, FAKE, n, None) == tq.EINVAL
        said(f"n={n}")
    assert lib.trellis_cache_free(cp, sp, None, 2, None) == tq.EINVAL
    said("seq_ids is NULL")
    assert lib.trellis_cache_free(cp, ctypes.byref(state(refs=None)), FAKE, 2, None) == tq.EINVAL
    said("refs is NULL")
    need = lib.trellis_cache_fork_workspace_bytes(cp, sp, 5)
    assert need > 0
    assert lib.trellis_cache_fork(cp, sp, FAKE, FAKE, 5, FAKE, FAKE, need - 1, None) == tq.EWORKSPACE
    assert lib.trellis_cache_fork(cp, sp, FAKE, None, 5, FAKE, FAKE, need, None) == tq.EINVAL
    said("children is NULL")
    need = lib.trellis_cache_reserve_workspace_bytes(cp, sp, 5)
    assert lib.trellis_cache_reserve(cp, sp, FAKE, 5, FAKE, 9, FAKE, FAKE, FAKE, need - 1, None) == tq.EWORKSPACE
    assert lib.trellis_cache_reserve(cp, sp, FAKE, 5, FAKE, 9, None, FAKE, FAKE, need, None) == tq.EINVAL
    said("slots is NULL")
    assert lib.trellis_cache_reserve(cp, sp, FAKE, 5, FAKE, -1, FAKE, FAKE, FAKE, need, None) == tq.EINVAL
    for m in (0, 65):
        assert lib.trellis_cache_accept(cp, sp, FAKE, 5, FAKE, m, FAKE, FAKE, None) == tq.EINVAL
        said(f"max_path={m}")
    assert lib.trellis_cache_accept(cp, sp, FAKE, 5, None, 4, FAKE, FAKE, None) == tq.EINVAL
    said("path is NULL")
    big = ctypes.byref(state(width=1 << 22))
    assert lib.trellis_cache_free(cp, big, FAKE, 1000, None) == tq.EINVAL
    said("too many")


def test_binding_refuses_host_tensors_and_missing_devices():
    import torch
    t = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        tq.cache_free(t, t[0], t[0], t[0])
    with pytest.raises(TypeError, match="torch.Tensor"):
        tq.cache_free(t, t[0], [0], t[0])
