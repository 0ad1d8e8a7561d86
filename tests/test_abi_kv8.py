"""Host-side checks of the entry points over the 8-bit cache (no GPU, no
launches): every invalid call is refused with a status and a message."""
import ctypes

import pytest

import trellis_coded_quantized_amd as tq
from tests.test_abi_attention import BAD_STATE, FAKE, MIS, said, state

WS = ctypes.c_void_p(1 << 20)


def cache(k=1 << 20, v=1 << 20, ks=1 << 20, vs=(1 << 20) + 1, pages=64, layers=1, heads=4, head_dim=128, page_size=16,
          dtype=tq.KV_BF16):
    return tq.Kv8Cache(k, v, ks, vs, pages, layers, heads, head_dim, page_size, dtype)


BAD_CACHE = [
    (dict(head_dim=96), tq.EUNSUPPORTED, "head_dim=96"), (dict(page_size=8), tq.EUNSUPPORTED, "page_size=8"),
    (dict(page_size=24), tq.EUNSUPPORTED, "page_size=24"), (dict(page_size=512), tq.EUNSUPPORTED, "page_size=512"),
    (dict(dtype=2), tq.EINVAL, "dtype=2"), (dict(heads=0), tq.EINVAL, "heads=0"), (dict(pages=0), tq.EINVAL, "pages=0"),
    (dict(pages=1 << 27), tq.EINVAL, "pages="), (dict(layers=0), tq.EINVAL, "layers=0"),
    (dict(k=None), tq.EINVAL, "cache k is NULL"), (dict(v=(1 << 20) + 8), tq.EINVAL, "cache v not 16-byte"),
    (dict(ks=None), tq.EINVAL, "cache k_scale is NULL"), (dict(vs=None), tq.EINVAL, "cache v_scale is NULL"),
]


def refer(c):
    return None if c is False else ctypes.byref(c or cache())


def window(c=None, s=None, q=FAKE, stride=32 * 128, n=2, starts=FAKE, tokens=5, hq=32, max_q=3, win=0, sinks=0,
           scale=0.1, out=FAKE, ws=FAKE, wsb=1 << 40):
    s = s or state()
    return tq.load_library().trellis_window_attention_kv8(q, stride, refer(c), ctypes.byref(s), None, n, starts, tokens,
                                                          hq, max_q, win, sinks, scale, out, ws, wsb, None)


def tree(c=None, s=None, anc=FAKE, max_q=3, wsb=1 << 40):
    s = s or state()
    return tq.load_library().trellis_tree_attention_kv8(FAKE, 32 * 128, refer(c), ctypes.byref(s), None, 2, FAKE, anc, 5,
                                                        32, max_q, 0.1, FAKE, FAKE, wsb, None)


def append(c=None, q=FAKE, qs=32 * 128, ks=512, rotary=64, eps=1e-6, inv=FAKE, tokens=5, hq=32, slots=FAKE, out=FAKE):
    return tq.load_library().trellis_qk_norm_rope_kv8(q, qs, FAKE, ks, FAKE, 512, FAKE, FAKE, FAKE, inv, rotary, 0, eps,
                                                      slots, out, refer(c), tokens, hq, None)


def fork(c=None, s=None, parents=FAKE, n=2, wsb=1 << 40):
    s = s or state()
    return tq.load_library().trellis_cache_fork_kv8(refer(c), ctypes.byref(s), parents, FAKE, n, FAKE, FAKE, wsb, None)


def accept(c=None, s=None, path=FAKE, max_path=4, n=2, new=FAKE):
    s = s or state()
    return tq.load_library().trellis_cache_accept_kv8(refer(c), ctypes.byref(s), FAKE, n, path, max_path, FAKE, new, None)


@pytest.mark.parametrize("kw,status,needle", BAD_CACHE)
@pytest.mark.parametrize("call", [window, tree, append, fork, accept])
def test_bad_caches(call, kw, status, needle):
    assert call(c=cache(**kw)) == status
    said(needle)


@pytest.mark.parametrize("call", [window, tree, append, fork, accept])
def test_no_cache(call):
    assert call(c=False) == tq.EINVAL
    said("cache is NULL")


@pytest.mark.parametrize("kw,needle", BAD_STATE)
@pytest.mark.parametrize("call", [window, tree, fork, accept])
def test_bad_states(call, kw, needle):
    assert call(s=state(**kw)) == tq.EINVAL
    said(needle)


@pytest.mark.parametrize("call,kw,needle", [
    (window, dict(hq=33), "heads_q=33"), (window, dict(stride=4), "q_stride"), (window, dict(n=0), "n=0"),
    (window, dict(max_q=0), "max_q=0"), (window, dict(win=-1), "window=-1"), (window, dict(scale=float("nan")), "scale"),
    (window, dict(q=MIS), "q not 16-byte"), (window, dict(starts=None), "q_start is NULL"),
    (window, dict(out=None), "out is NULL"), (window, dict(tokens=-1), "tokens=-1"),
    (window, dict(c=cache(layers=2)), "one layer"), (tree, dict(max_q=65), "max_q=65"),
    (tree, dict(anc=None), "ancestors is NULL"), (append, dict(rotary=24), "rotary_dim=24"),
    (append, dict(eps=-1.0), "eps"), (append, dict(qs=12), "q_stride"), (append, dict(ks=128), "k_stride"),
    (append, dict(inv=None), "inv_freq is NULL"), (append, dict(slots=None), "slots is NULL"),
    (append, dict(out=MIS), "out not 16-byte"), (append, dict(c=cache(layers=3)), "one layer"),
    (append, dict(tokens=1 << 31), "tokens="), (fork, dict(parents=None), "parents is NULL"), (fork, dict(n=1025), "n=1025"),
    (accept, dict(max_path=65), "max_path=65"), (accept, dict(path=None), "path is NULL"),
    (accept, dict(new=MIS), "new_lengths not 4-byte")])
def test_refusals(call, kw, needle):
    assert call(**kw) == tq.EINVAL
    said(needle)


def test_workspaces():
    lib, c, s = tq.load_library(), ctypes.byref(cache()), ctypes.byref(state())
    need = lib.trellis_window_attention_kv8_workspace_bytes(c, s, 2, 5, 32, 3, 0, 0)
    assert need > 0 and window(wsb=need - 1) == tq.EWORKSPACE
    need = lib.trellis_tree_attention_kv8_workspace_bytes(c, s, 2, 5, 32, 3)
    assert need > 0 and tree(wsb=need - 1) == tq.EWORKSPACE
    need = lib.trellis_cache_fork_kv8_workspace_bytes(c, s, 2)
    assert need > 0 and fork(wsb=need - 1) == tq.EWORKSPACE
    assert lib.trellis_window_attention_kv8_workspace_bytes(None, s, 2, 5, 32, 3, 0, 0) == 0
    assert lib.trellis_cache_fork_kv8_workspace_bytes(ctypes.byref(cache(head_dim=32)), s, 2) == 0
    assert lib.trellis_window_attention_kv8_workspace_bytes(c, s, 2, 0, 32, 3, 0, 0) == 0


def test_no_tokens_is_no_work():
    assert window(tokens=0, q=None, out=None, ws=None, wsb=0) == tq.OK
    assert append(tokens=0, q=None, out=None) == tq.OK


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32 + 100, -2 ** 31 - 1])
def test_numbers_past_32_bits(value):
    for name in ("max_q", "window", "sinks"):
        with pytest.raises(ValueError, match=name):
            tq.window_attention_kv8(*[None] * 8, **{"max_q": 1, name: value})
    with pytest.raises(ValueError, match="max_q"):
        tq.tree_attention_kv8(*[None] * 9, value)
