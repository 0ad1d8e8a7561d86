"""Host-side checks of the adapters' entry points (no GPU, no launches)."""
import ctypes

import pytest

import trellis_coded_quantized_amd as tq
from tests.test_abi_attention import FAKE, MIS, said

P = 1 << 20


def target(a=P, b=P, y=P, out=P, R=96, y_stride=96, out_stride=96):
    return tq.LoraTarget(a, b, y, out, R, y_stride, out_stride)


def add(targets=None, count=None, x=FAKE, xs=64, y_dtype=tq.OUT_BF16, starts=FAKE, adapters=FAKE, n=2, scales=FAKE,
        ranks=None, pool=4, rank=16, M=5, C=64, ws=FAKE, wsb=1 << 40):
    targets = [target()] if targets is None else targets
    array = (tq.LoraTarget * len(targets))(*targets) if targets else None
    return tq.load_library().trellis_lora_add(x, xs, array, len(targets) if count is None else count, y_dtype, starts,
                                              adapters, n, scales, ranks, pool, rank, M, C, ws, wsb, None)


def swiglu(gate=None, up=None, out=ctypes.c_void_p(P + 4096), os=96, y_dtype=tq.OUT_BF16, wsb=1 << 40, **kw):
    g = None if gate is False else ctypes.byref(gate or target())
    u = None if up is False else ctypes.byref(up or target())
    return tq.load_library().trellis_lora_swiglu(FAKE, 64, g, u, out, os, y_dtype, FAKE, FAKE, 2, FAKE, None, 4, 16, 5, 64,
                                                 FAKE, wsb, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(targets=[]), tq.EINVAL, "targets is NULL"), (dict(count=0), tq.EINVAL, "n_targets=0"),
    (dict(targets=[target()] * 5), tq.EINVAL, "n_targets=5"), (dict(rank=128), tq.EUNSUPPORTED, "rank=128"),
    (dict(rank=12), tq.EUNSUPPORTED, "rank=12"), (dict(C=60, xs=64), tq.EUNSUPPORTED, "C=60"), (dict(C=0), tq.EINVAL, "C=0"),
    (dict(n=0), tq.EINVAL, "n=0"), (dict(n=65536), tq.EINVAL, "n=65536"), (dict(M=-1), tq.EINVAL, "M=-1"),
    (dict(M=(1 << 22) + 1), tq.EINVAL, "M="), (dict(y_dtype=2), tq.EINVAL, "y_dtype=2"), (dict(pool=0), tq.EINVAL, "pool=0"),
    (dict(xs=56), tq.EINVAL, "x_stride=56"), (dict(xs=68), tq.EINVAL, "x_stride=68"), (dict(x=None), tq.EINVAL, "x is NULL"),
    (dict(x=MIS), tq.EINVAL, "x not 16-byte"), (dict(starts=None), tq.EINVAL, "starts is NULL"),
    (dict(adapters=MIS), tq.EINVAL, "adapters not 4-byte"), (dict(scales=None), tq.EINVAL, "scales is NULL"),
    (dict(ranks=MIS), tq.EINVAL, "ranks not 4-byte"), (dict(wsb=100), tq.EWORKSPACE, "workspace 100"),
    (dict(ws=ctypes.c_void_p(P + 16)), tq.EINVAL, "workspace not 256-byte"),
    (dict(targets=[target(R=0)]), tq.EINVAL, "R=0"), (dict(targets=[target(R=1 << 19)]), tq.EINVAL, "R="),
    (dict(targets=[target(y_stride=95)]), tq.EINVAL, "y_stride=95"),
    (dict(targets=[target(out=P + 64, out_stride=95)]), tq.EINVAL, "out_stride=95"),
    (dict(targets=[target(out_stride=97)]), tq.EINVAL, "another stride"),
    (dict(targets=[target(), target(a=None)]), tq.EINVAL, "a is NULL"),
    (dict(targets=[target(b=P + 8)]), tq.EINVAL, "b not 16-byte"), (dict(targets=[target(y=P + 1)]), tq.EINVAL, "y not 2-byte"),
    (dict(targets=[target(out=None)]), tq.EINVAL, "out is NULL"),
    (dict(targets=[target(y=P + 2)], y_dtype=tq.OUT_F32), tq.EINVAL, "y not 4-byte")])
def test_add(kw, status, needle):
    assert add(**kw) == status
    said(needle)


@pytest.mark.parametrize("kw,needle", [
    (dict(gate=False), "gate is NULL"), (dict(up=False), "up is NULL"), (dict(up=target(R=95)), "95"),
    (dict(out=None), "out is NULL"), (dict(os=95), "out_stride=95"),
    (dict(out=ctypes.c_void_p(P), os=104), "out is gate with another stride"),
    (dict(up=target(y=P + 8192), out=ctypes.c_void_p(P + 8192), os=104), "out is up with another stride"),
    (dict(out=ctypes.c_void_p(P), y_dtype=tq.OUT_F32), "out is an f32 input")])
def test_swiglu(kw, needle):
    assert swiglu(**kw) == tq.EINVAL
    said(needle)


def test_no_rows_and_sizes():
    assert add(M=0, x=None, starts=None, ws=None, wsb=0) == tq.OK
    size = tq.load_library().trellis_lora_workspace_bytes
    need = size(5, 64, 2, 1, 16)
    assert need >= 5 * 16 * 4 and add(wsb=need - 1) == tq.EWORKSPACE
    assert size(0, 64, 2, 1, 16) == 0 and size(5, 60, 2, 1, 16) == 0 and size(5, 64, 2, 5, 16) == 0
    assert size(1 << 22, 64, 65535, 4, 64) >= (1 << 22) * 256 * 4


def test_binding():
    with pytest.raises(ValueError, match="projections"):
        tq.lora_add(None, [], [], [], None, None, None)
    with pytest.raises(ValueError, match="projections"):
        tq.lora_add(None, [None], [None, None], [None], None, None, None)
    with pytest.raises(TypeError, match="x must be"):
        tq.lora_add(None, [None], [None], [None], None, None, None)
