"""MI355X (gfx950) linear layer over packed trellis-coded weights.

A thin ctypes binding over libtrellis.so (include/trellis.h).  The functions
keep the C names without the ``trellis_`` prefix and only marshal
arguments: shapes and dtypes are checked, outputs and workspaces are
allocated with PyTorch on the input's device, and the call is enqueued on
the current PyTorch stream.  Every arithmetic step runs in the HIP library;
if libtrellis.so is missing the functions raise instead of computing
anything another way.

Tensor conventions (all CUDA/HIP device tensors, contiguous):
  codes  int32/uint32 [rows, cols*k/32]  packed code words
  scales float16 [rows]
  x      bfloat16 [M, in_features]

Attention between the projections (one paged key/value cache):
  k_cache  bfloat16/float16 [(layers,) pages, kv_heads, D/8, P, 8]
  v_cache  the same type    [(layers,) pages, kv_heads, P/8, D, 8]
  table    int32 [seqs, width] page numbers, -1: none
  lengths  int32 [seqs] cached tokens;  refs  int32 [pages] holders of a page

Low-rank adapters beside the projections:
  a  bfloat16 [pool, rank, in];  b  bfloat16 [pool, out, rank]

The same over a cache held in 8 bits (calls ending in _kv8):
  k_cache  float8_e4m3fn [(layers,) pages, kv_heads, D/16, P, 16]
  v_cache  float8_e4m3fn [(layers,) pages, kv_heads, P/16, D, 16]
  k_scale, v_scale  float8_e8m0fnu [(layers,) pages, kv_heads, P/16]
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtrellis.so")

OK, EINVAL, EUNSUPPORTED, EWORKSPACE, EHIP = 0, -1, -2, -3, -4
OUT_BF16, OUT_F32 = 0, 1
PREFILL_FUSED, PREFILL_EXPAND_GEMM, PREFILL_AUTO = 0, 1, 2
MATVEC_MAX_M = 4
GROUP_MAX = 4
KV_BF16, KV_F16 = 0, 1
TREE_MAX = 64
ACCEPT_MAX = 64
CACHE_MAX_SEQS = 1024
LORA_MAX = 4

# every symbol include/trellis.h declares
EXPORTS = (
    "trellis_matvec_axis1_workspace_bytes", "trellis_matvec_axis1", "trellis_matvec_axis1_group",
    "trellis_gateup_swiglu_workspace_bytes", "trellis_gateup_swiglu",
    "trellis_matvec_axis0_workspace_bytes", "trellis_matvec_axis0", "trellis_matvec_axis0_noalloc",
    "trellis_mlp_decode_workspace_bytes", "trellis_mlp_decode",
    "trellis_matvec_axis0_il", "trellis_expand_bf16_il",
    "trellis_expand_bf16", "trellis_prefill_workspace_bytes", "trellis_prefill",
    "trellis_prefill_axis0_workspace_bytes", "trellis_prefill_axis0", "trellis_prefill_axis0_il",
    "trellis_prefill_tune", "trellis_prefill_axis0_tune",
    "trellis_probe_decode_only", "trellis_probe_gateup_decode_free",
    "trellis_qk_norm_rope",
    "trellis_tree_attention_workspace_bytes", "trellis_tree_attention",
    "trellis_window_attention_workspace_bytes", "trellis_window_attention",
    "trellis_cache_reserve_workspace_bytes", "trellis_cache_reserve",
    "trellis_cache_fork_workspace_bytes", "trellis_cache_fork", "trellis_cache_accept", "trellis_cache_free",
    "trellis_qk_norm_rope_kv8",
    "trellis_tree_attention_kv8_workspace_bytes", "trellis_tree_attention_kv8",
    "trellis_window_attention_kv8_workspace_bytes", "trellis_window_attention_kv8",
    "trellis_cache_fork_kv8_workspace_bytes", "trellis_cache_fork_kv8", "trellis_cache_accept_kv8",
    "trellis_lora_workspace_bytes", "trellis_lora_add", "trellis_lora_swiglu",
    "trellis_decode_states", "trellis_last_error", "trellis_version",
)


class TrellisError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"[status {status}] {msg}")
        self.status = status


class LoraTarget(ctypes.Structure):
    """trellis_lora_target of include/trellis.h"""
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("y", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("R", ctypes.c_int64), ("y_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64)]


class KvCache(ctypes.Structure):
    """trellis_kv_cache of include/trellis.h"""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", ctypes.c_int64), ("layers", ctypes.c_int),
                ("heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int),
                ("dtype", ctypes.c_int)]


class Kv8Cache(ctypes.Structure):
    """trellis_kv8_cache of include/trellis.h"""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("layers", ctypes.c_int),
                ("heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int),
                ("dtype", ctypes.c_int)]


class KvState(ctypes.Structure):
    """trellis_kv_state of include/trellis.h"""
    _fields_ = [("table", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("seqs", ctypes.c_int64), ("width", ctypes.c_int64)]


_lib = None
_vp, _i64, _int, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t


def load_library():
    """Load libtrellis.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} not built; run trellis_coded_quantized_amd._build.build()")
    lib = ctypes.CDLL(LIB_PATH)
    sig = {
        "trellis_matvec_axis1_workspace_bytes": (_sz, [_i64, _i64, _int, _int, _int, _int]),
        "trellis_matvec_axis1": (_int, [_vp, _vp, _vp, _vp, _int, _i64, _i64, _int, _int, _int, _int,
                                        _vp, _sz, _vp]),
        "trellis_matvec_axis1_group": (_int, [_vp, _vp, _vp, _vp, _int, _vp, _int, _i64, _int, _int, _int, _int,
                                              _vp]),
        "trellis_gateup_swiglu_workspace_bytes": (_sz, [_i64, _i64, _int, _int, _int, _int]),
        "trellis_gateup_swiglu": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _int,
                                         _int, _int, _int, _vp, _sz, _vp]),
        "trellis_matvec_axis0_workspace_bytes": (_sz, [_i64, _i64, _int, _int, _int, _int]),
        "trellis_matvec_axis0": (_int, [_vp, _vp, _vp, _vp, _int, _i64, _i64, _int, _int, _int, _int,
                                        _vp, _sz, _vp]),
        "trellis_matvec_axis0_noalloc": (_int, [_vp, _vp, _vp, _vp, _int, _i64, _i64, _int, _int, _int, _int,
                                                _vp]),
        "trellis_mlp_decode_workspace_bytes": (_sz, [_i64, _i64, _i64, _int, _int, _int, _int, _int]),
        "trellis_mlp_decode": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int,
                                      _int, _int, _int, _int, _vp, _sz, _vp]),
        "trellis_expand_bf16": (_int, [_vp, _vp, _vp, _i64, _i64, _int, _int, _int, _vp]),
        "trellis_matvec_axis0_il": (_int, [_vp, _vp, _vp, _vp, _int, _i64, _i64, _int, _int, _int, _int,
                                           _vp, _sz, _vp]),
        "trellis_expand_bf16_il": (_int, [_vp, _vp, _vp, _i64, _i64, _int, _int, _int, _vp]),
        "trellis_prefill_workspace_bytes": (_sz, [_i64, _i64, _i64, _int, _int, _int, _int]),
        "trellis_prefill": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _int, _int,
                                   _vp, _sz, _vp]),
        "trellis_prefill_axis0_workspace_bytes": (_sz, [_i64, _i64, _i64, _int, _int, _int, _int]),
        "trellis_prefill_axis0": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _int, _int,
                                         _vp, _sz, _vp]),
        "trellis_prefill_axis0_il": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _int, _int,
                                            _vp, _sz, _vp]),
        "trellis_prefill_tune": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _int, _vp, _sz, _vp]),
        "trellis_prefill_axis0_tune": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _int, _vp, _sz,
                                              _vp]),
        "trellis_probe_decode_only": (_int, [_vp, _vp, _int, _int, _int, _vp]),
        "trellis_probe_gateup_decode_free": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _int, _int, _int,
                                                    _int, _vp]),
        "trellis_decode_states": (_int, [_vp, _i64, _i64, _int, _int, _int, _vp, _vp, _vp, _vp]),
        "trellis_qk_norm_rope": (_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _int, _int,
                                        ctypes.c_float, _vp, _vp, _vp, _i64, _int, _vp]),
        "trellis_tree_attention_workspace_bytes": (_sz, [_vp, _vp, _int, _i64, _int, _int]),
        "trellis_tree_attention": (_int, [_vp, _i64, _vp, _vp, _vp, _int, _vp, _vp, _i64, _int, _int,
                                          ctypes.c_float, _vp, _vp, _sz, _vp]),
        "trellis_window_attention_workspace_bytes": (_sz, [_vp, _vp, _int, _i64, _int, _int, _int, _int]),
        "trellis_window_attention": (_int, [_vp, _i64, _vp, _vp, _vp, _int, _vp, _i64, _int, _int, _int, _int,
                                            ctypes.c_float, _vp, _vp, _sz, _vp]),
        "trellis_cache_reserve_workspace_bytes": (_sz, [_vp, _vp, _int]),
        "trellis_cache_reserve": (_int, [_vp, _vp, _vp, _int, _vp, _i64, _vp, _vp, _vp, _sz, _vp]),
        "trellis_cache_fork_workspace_bytes": (_sz, [_vp, _vp, _int]),
        "trellis_cache_fork": (_int, [_vp, _vp, _vp, _vp, _int, _vp, _vp, _sz, _vp]),
        "trellis_cache_accept": (_int, [_vp, _vp, _vp, _int, _vp, _int, _vp, _vp, _vp]),
        "trellis_cache_free": (_int, [_vp, _vp, _vp, _int, _vp]),
        **{"trellis_" + name + "_kv8" + more: sig_of for name, more, sig_of in (
            ("tree_attention", "_workspace_bytes", (_sz, [_vp, _vp, _int, _i64, _int, _int])),
            ("tree_attention", "", (_int, [_vp, _i64, _vp, _vp, _vp, _int, _vp, _vp, _i64, _int, _int,
                                           ctypes.c_float, _vp, _vp, _sz, _vp])),
            ("window_attention", "_workspace_bytes", (_sz, [_vp, _vp, _int, _i64, _int, _int, _int, _int])),
            ("window_attention", "", (_int, [_vp, _i64, _vp, _vp, _vp, _int, _vp, _i64, _int, _int, _int, _int,
                                             ctypes.c_float, _vp, _vp, _sz, _vp])),
            ("qk_norm_rope", "", (_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _int, _int,
                                         ctypes.c_float, _vp, _vp, _vp, _i64, _int, _vp])),
            ("cache_fork", "_workspace_bytes", (_sz, [_vp, _vp, _int])),
            ("cache_fork", "", (_int, [_vp, _vp, _vp, _vp, _int, _vp, _vp, _sz, _vp])),
            ("cache_accept", "", (_int, [_vp, _vp, _vp, _int, _vp, _int, _vp, _vp, _vp])))},
        "trellis_lora_workspace_bytes": (_sz, [_i64, _i64, _int, _int, _int]),
        "trellis_lora_add": (_int, [_vp, _i64, _vp, _int, _int, _vp, _vp, _int, _vp, _vp, _i64, _int, _i64, _i64, _vp,
                                    _sz, _vp]),
        "trellis_lora_swiglu": (_int, [_vp, _i64, _vp, _vp, _vp, _i64, _int, _vp, _vp, _int, _vp, _vp, _i64, _int,
                                       _i64, _i64, _vp, _sz, _vp]),
        "trellis_last_error": (ctypes.c_char_p, []),
        "trellis_version": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def version() -> str:
    return load_library().trellis_version().decode()


def _check(status: int):
    if status != OK:
        raise TrellisError(status, load_library().trellis_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t, name, dtypes, ndim):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor")


_CODES = (torch.int32, torch.uint32)


def _geometry(codes, k):
    rows, words = codes.shape
    if (words * 32) % k:
        raise ValueError(f"{words} words are not a whole number of {k}-bit symbols")
    return rows, words * 32 // k


def _axis0_geometry(codes, k):
    """(rows, cols, interleaved) of axis-0 codes: row-major [R, C*k/32], or the
    block-interleaved k = 3 layout [C/512, R, 48] (identified by its shape)."""
    if codes.dim() == 3:
        groups, rows, words = codes.shape
        if k != 3 or words != 48:
            raise ValueError(f"interleaved codes must be k = 3 with 48 words per row pair, got k={k}, {words}")
        return rows, groups * 512, True
    rows, cols = _geometry(codes, k)
    return rows, cols, False


def _workspace(nbytes, device, workspace):
    if nbytes == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif not (isinstance(workspace, torch.Tensor) and workspace.device.type == "cuda" and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous device tensor")
    return workspace, workspace.numel() * workspace.element_size()


def _rows(scales, n, name="scales"):
    if scales.numel() != n:
        raise ValueError(f"{name} has {scales.numel()} entries, the matrix has {n} stored rows")


def _out(t, name, shape, dtypes, device):
    """A caller's output buffer (exactly `shape`, contiguous, on the device), or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtypes[0], device=device)
    _need(t, name, dtypes, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


_F = (torch.bfloat16, torch.float32)


def _odt(out_dtype):
    """output dtypes a matvec accepts, the requested one first"""
    if out_dtype not in _F:
        raise ValueError(f"out_dtype {out_dtype} not in {_F}")
    return (out_dtype,) + _F


def matvec_axis1(codes, scales, x, k, L=12, T=256, out_dtype=torch.bfloat16, out=None,
                 workspace=None):
    """y[m, r] = sum_c w(r, c) x[m, c]; codes [R, C*k/32] coded along inputs."""
    _need(codes, "codes", _CODES, 2)
    _need(scales, "scales", (torch.float16,), 1)
    _need(x, "x", (torch.bfloat16,), 2)
    R, C = _geometry(codes, k)
    _rows(scales, R)
    M = x.shape[0]
    if x.shape[1] != C:
        raise ValueError(f"x has {x.shape[1]} features, codes encode {C}")
    out = _out(out, "out", (M, R), _odt(out_dtype), x.device)
    od = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    lib = load_library()
    ws, wsb = _workspace(lib.trellis_matvec_axis1_workspace_bytes(R, C, M, k, L, T), x.device, workspace)
    _check(lib.trellis_matvec_axis1(_ptr(codes), _ptr(scales), _ptr(x), _ptr(out), od, R, C, M, k, L,
                                    T, _ptr(ws), wsb, _stream(x.device)))
    return out


def matvec_axis1_group(codes, scales, x, k, L=12, T=256, out_dtype=torch.bfloat16, outs=None):
    """matvec_axis1 of every matrix in `codes` (same C and k, same x) in one launch;
    returns the list of outputs [M, R_j]."""
    n = len(codes)
    if n != len(scales) or not 1 <= n <= GROUP_MAX:
        raise ValueError(f"{n} code tensors, {len(scales)} scale tensors (1..{GROUP_MAX} matrices)")
    _need(x, "x", (torch.bfloat16,), 2)
    Rs = []
    for c, s in zip(codes, scales):
        _need(c, "codes", _CODES, 2)
        _need(s, "scales", (torch.float16,), 1)
        R, C = _geometry(c, k)
        _rows(s, R)
        if x.shape[1] != C:
            raise ValueError(f"x has {x.shape[1]} features, codes encode {C}")
        Rs.append(R)
    M = x.shape[0]
    if outs is None:
        outs = [None] * n
    if len(outs) != n:
        raise ValueError(f"{len(outs)} outputs for {n} matrices")
    outs = [_out(o, f"outs[{j}]", (M, R), _odt(out_dtype), x.device) for j, (o, R) in enumerate(zip(outs, Rs))]
    od = OUT_F32 if outs[0].dtype == torch.float32 else OUT_BF16
    if any(o.dtype != outs[0].dtype for o in outs):
        raise ValueError("outputs of one grouped call share a dtype")
    P = ctypes.c_void_p * n
    _check(load_library().trellis_matvec_axis1_group(
        P(*[c.data_ptr() for c in codes]), P(*[s.data_ptr() for s in scales]), P(*[o.data_ptr() for o in outs]),
        (ctypes.c_int64 * n)(*Rs), n, _ptr(x), od, x.shape[1], M, k, L, T, _stream(x.device)))
    return outs


def gateup_swiglu(gcodes, gscales, ucodes, uscales, x, k, L=12, T=256, out=None,
                  gate_f32=None, up_f32=None, workspace=None):
    """bf16 silu(gate(x)) * up(x) with the bf16 cast chain; returns out [M, R]."""
    for t, n in ((gcodes, "gcodes"), (ucodes, "ucodes")):
        _need(t, n, _CODES, 2)
    for t, n in ((gscales, "gscales"), (uscales, "uscales")):
        _need(t, n, (torch.float16,), 1)
    _need(x, "x", (torch.bfloat16,), 2)
    if gcodes.shape != ucodes.shape:
        raise ValueError("gate and up codes differ in shape")
    R, C = _geometry(gcodes, k)
    _rows(gscales, R, "gscales")
    _rows(uscales, R, "uscales")
    M = x.shape[0]
    if x.shape[1] != C:
        raise ValueError(f"x has {x.shape[1]} features, codes encode {C}")
    out = _out(out, "out", (M, R), (torch.bfloat16,), x.device)
    if gate_f32 is not None:
        _out(gate_f32, "gate_f32", (M, R), (torch.float32,), x.device)
    if up_f32 is not None:
        _out(up_f32, "up_f32", (M, R), (torch.float32,), x.device)
    lib = load_library()
    ws, wsb = _workspace(lib.trellis_gateup_swiglu_workspace_bytes(R, C, M, k, L, T), x.device,
                         workspace)
    _check(lib.trellis_gateup_swiglu(_ptr(gcodes), _ptr(gscales), _ptr(ucodes), _ptr(uscales),
                                     _ptr(x), _ptr(out), _ptr(gate_f32), _ptr(up_f32), R, C, M, k, L,
                                     T, _ptr(ws), wsb, _stream(x.device)))
    return out


def matvec_axis0(codes_t, scales, x, k, L=12, T=256, out_dtype=torch.bfloat16, out=None,
                 workspace=None):
    """y[m, c] = sum_r w(r, c) x[m, r]; codes_t is the stored W^T [R_in, C_out*k/32],
    or for k = 3 the block-interleaved [C_out/512, R_in, 48]."""
    _need(codes_t, "codes", _CODES, codes_t.dim() if codes_t.dim() == 3 else 2)
    _need(scales, "scales", (torch.float16,), 1)
    _need(x, "x", (torch.bfloat16,), 2)
    R, C, il = _axis0_geometry(codes_t, k)
    _rows(scales, R)
    M = x.shape[0]
    if x.shape[1] != R:
        raise ValueError(f"x has {x.shape[1]} features, stored rows are {R}")
    out = _out(out, "out", (M, C), _odt(out_dtype), x.device)
    od = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    lib = load_library()
    ws, wsb = _workspace(lib.trellis_matvec_axis0_workspace_bytes(R, C, M, k, L, T), x.device,
                         workspace)
    fn = lib.trellis_matvec_axis0_il if il else lib.trellis_matvec_axis0
    _check(fn(_ptr(codes_t), _ptr(scales), _ptr(x), _ptr(out), od, R, C, M, k, L, T, _ptr(ws), wsb,
              _stream(x.device)))
    return out


def mlp_decode(gcodes, gscales, ucodes, uscales, dcodes_t, dscales, x, k_gu, k_down, L=12, T=256,
               hidden=None, out=None, workspace=None):
    """down(silu(gate(x)) * up(x)) for M <= 4 rows: the gate/up SwiGLU kernel,
    then the axis-0 down projection (dcodes_t is the stored W_down^T
    [R, C_out*k_down/32]).  `hidden` (bf16 [M, R]) receives the hidden
    vectors if given."""
    for t, n in ((gcodes, "gcodes"), (ucodes, "ucodes"), (dcodes_t, "dcodes")):
        _need(t, n, _CODES, 2)
    for t, n in ((gscales, "gscales"), (uscales, "uscales"), (dscales, "dscales")):
        _need(t, n, (torch.float16,), 1)
    _need(x, "x", (torch.bfloat16,), 2)
    R, C = _geometry(gcodes, k_gu)
    if _geometry(ucodes, k_gu) != (R, C):
        raise ValueError("gate and up codes differ in shape")
    Rd, C_out = _geometry(dcodes_t, k_down)
    if Rd != R:
        raise ValueError(f"down projection has {Rd} stored rows, the hidden width is {R}")
    M = x.shape[0]
    if x.shape[1] != C:
        raise ValueError(f"x has {x.shape[1]} features, gate/up take {C}")
    _rows(gscales, R, "gscales")
    _rows(uscales, R, "uscales")
    _rows(dscales, Rd, "dscales")
    out = _out(out, "out", (M, C_out), (torch.bfloat16,), x.device)
    if hidden is not None:
        _out(hidden, "hidden", (M, R), (torch.bfloat16,), x.device)
    lib = load_library()
    ws, wsb = _workspace(lib.trellis_mlp_decode_workspace_bytes(R, C, C_out, M, k_gu, k_down, L, T), x.device,
                         workspace)
    _check(lib.trellis_mlp_decode(_ptr(gcodes), _ptr(gscales), _ptr(ucodes), _ptr(uscales), _ptr(dcodes_t),
                                  _ptr(dscales), _ptr(x), _ptr(hidden), _ptr(out),
                                  R, C, C_out, M, k_gu, k_down, L, T, _ptr(ws), wsb, _stream(x.device)))
    return out


def expand_bf16(codes, scales, k, L=12, T=256, out=None):
    """bf16 [R, C] decode of the stored matrix (stored orientation); codes
    [R, C*k/32], or for k = 3 the block-interleaved axis-0 layout [C/512, R, 48]."""
    _need(codes, "codes", _CODES, codes.dim() if codes.dim() == 3 else 2)
    _need(scales, "scales", (torch.float16,), 1)
    R, C, il = _axis0_geometry(codes, k)
    _rows(scales, R)
    out = _out(out, "out", (R, C), (torch.bfloat16,), codes.device)
    lib = load_library()
    fn = lib.trellis_expand_bf16_il if il else lib.trellis_expand_bf16
    _check(fn(_ptr(codes), _ptr(scales), _ptr(out), R, C, k, L, T, _stream(codes.device)))
    return out


def prefill(codes, scales, x, k, L=12, T=256, algo=PREFILL_FUSED, out=None, workspace=None, tune=False):
    """bf16 [M, R] = x [M, C] times the bf16 expansion of the axis-1 codes.
    tune=True runs trellis_prefill_tune (expand + GEMM after timing the GEMM
    candidates; synchronises the host) instead of trellis_prefill."""
    _need(codes, "codes", _CODES, 2)
    _need(scales, "scales", (torch.float16,), 1)
    _need(x, "x", (torch.bfloat16,), 2)
    R, C = _geometry(codes, k)
    _rows(scales, R)
    M = x.shape[0]
    if x.shape[1] != C:
        raise ValueError(f"x has {x.shape[1]} features, codes encode {C}")
    out = _out(out, "out", (M, R), (torch.bfloat16,), x.device)
    lib = load_library()
    if tune:
        algo = PREFILL_EXPAND_GEMM
    ws, wsb = _workspace(lib.trellis_prefill_workspace_bytes(R, C, M, k, L, T, algo), x.device,
                         workspace)
    if tune:
        _check(lib.trellis_prefill_tune(_ptr(codes), _ptr(scales), _ptr(x), _ptr(out), R, C, M, k, L, T,
                                        _ptr(ws), wsb, _stream(x.device)))
    else:
        _check(lib.trellis_prefill(_ptr(codes), _ptr(scales), _ptr(x), _ptr(out), R, C, M, k, L, T, algo,
                                   _ptr(ws), wsb, _stream(x.device)))
    return out


def prefill_axis0(codes_t, scales, x, k, L=12, T=256, algo=PREFILL_EXPAND_GEMM, out=None, workspace=None,
                  tune=False):
    """out[m, c] = bf16(sum_r wb(r, c) x[m, r]) for a matrix stored transposed
    (axis 0): codes_t [R_in, C_out*k/32] (or for k = 3 the block-interleaved
    [C_out/512, R_in, 48]), x bf16 [M, R_in]; expand + GEMM, or the fused
    decode-to-LDS MFMA kernel (R_in a multiple of 128).  tune=True runs
    trellis_prefill_axis0_tune (row-major codes; synchronises the host)."""
    _need(codes_t, "codes", _CODES, codes_t.dim() if codes_t.dim() == 3 else 2)
    _need(scales, "scales", (torch.float16,), 1)
    _need(x, "x", (torch.bfloat16,), 2)
    R, C, il = _axis0_geometry(codes_t, k)
    _rows(scales, R)
    M = x.shape[0]
    if x.shape[1] != R:
        raise ValueError(f"x has {x.shape[1]} features, stored rows are {R}")
    out = _out(out, "out", (M, C), (torch.bfloat16,), x.device)
    lib = load_library()
    if tune:
        if il:
            raise ValueError("tune takes row-major codes (the GEMM it tunes is the same for both layouts)")
        algo = PREFILL_EXPAND_GEMM
    ws, wsb = _workspace(lib.trellis_prefill_axis0_workspace_bytes(R, C, M, k, L, T, algo), x.device, workspace)
    if tune:
        _check(lib.trellis_prefill_axis0_tune(_ptr(codes_t), _ptr(scales), _ptr(x), _ptr(out), R, C, M, k, L, T,
                                              _ptr(ws), wsb, _stream(x.device)))
        return out
    fn = lib.trellis_prefill_axis0_il if il else lib.trellis_prefill_axis0
    _check(fn(_ptr(codes_t), _ptr(scales), _ptr(x), _ptr(out), R, C, M, k, L, T, algo, _ptr(ws), wsb,
              _stream(x.device)))
    return out


def prefill_workspace_bytes(R, C, M, k, algo, L=12, T=256) -> int:
    return int(load_library().trellis_prefill_workspace_bytes(R, C, M, k, L, T, algo))


def decode_states(codes, k, L=12, T=256):
    """(states int16-bits [R, C], y int16 [R, C], value f32 [R, C]) from the GPU decoder."""
    _need(codes, "codes", _CODES, 2)
    R, C = _geometry(codes, k)
    dev = codes.device
    st = torch.empty((R, C), dtype=torch.int16, device=dev)
    ys = torch.empty((R, C), dtype=torch.int16, device=dev)
    vals = torch.empty((R, C), dtype=torch.float32, device=dev)
    _check(load_library().trellis_decode_states(_ptr(codes), R, C, k, L, T, _ptr(st), _ptr(ys),
                                                _ptr(vals), _stream(dev)))
    return st, ys, vals


PROBE_THREADS = 512


def probe_decode_only(runs, k, iters, blocks=None):
    """Measurement probe: decode the runs held in `runs` (int32/uint32
    [blocks * 512, k + 1]) `iters` times each; returns the per-wave sums
    (f32 [blocks * 8], 16 times the sum of the codes each wave decoded)."""
    _need(runs, "runs", _CODES, 2)
    n, words = runs.shape
    if words != k + 1 or n % PROBE_THREADS:
        raise ValueError(f"runs must be [blocks * {PROBE_THREADS}, k + 1], got {tuple(runs.shape)}")
    blocks = n // PROBE_THREADS if blocks is None else blocks
    out = torch.empty(blocks * PROBE_THREADS // 64, dtype=torch.float32, device=runs.device)
    _check(load_library().trellis_probe_decode_only(_ptr(runs), _ptr(out), blocks, iters, k, _stream(runs.device)))
    return out


def probe_gateup_decode_free(gcodes, gscales, ucodes, uscales, x, k, L=12, T=256, out=None):
    """Measurement probe: the gate/up kernel with no decode (timing floor; the
    output values are meaningless)."""
    R, C = _geometry(gcodes, k)
    M = x.shape[0]
    out = _out(out, "out", (M, R), (torch.bfloat16,), x.device)
    _check(load_library().trellis_probe_gateup_decode_free(_ptr(gcodes), _ptr(gscales), _ptr(ucodes), _ptr(uscales),
                                                           _ptr(x), _ptr(out), R, C, M, k, L, T, _stream(x.device)))
    return out


# ---- attention between the projections ------------------------------------
# These calls run many times a decode step on little data, so their checks are
# kept to one pass of plain comparisons per tensor, and pointers go to the
# library as integers.

_KV = {torch.bfloat16: KV_BF16, torch.float16: KV_F16}
_byref = ctypes.byref


def _tensor(t, name, dtype, shape, index):
    """Check a contiguous device tensor (shape entries of None: any size); its address."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    got = t.shape
    if got != shape and (len(got) != len(shape) or any(w is not None and w != g for w, g in zip(shape, got))):
        raise ValueError(f"{name}: shape {tuple(got)} of {t.numel()} entries, expected "
                         f"{tuple('any' if w is None else w for w in shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != index:
        raise ValueError(f"{name} must be a device tensor on the device of the call, is on {t.device}")
    return t.data_ptr()


def _c_int(v, name):
    """A number that the library takes as a C int; ctypes would drop the bits above."""
    if not -0x80000000 <= v <= 0x7FFFFFFF:
        raise ValueError(f"{name}={v} outside 32 bits")
    return v


def _index(t, name):
    """Device number of the tensor that a call runs by."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.get_device()


def _result(t, name, shape, dtype, device, index):
    """A caller's output buffer or a new one, and its address."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    return t, _tensor(t, name, dtype, shape, index)


def _scratch(nbytes, device, workspace):
    """(tensor to keep alive, address, bytes) of a call's workspace."""
    if nbytes == 0:
        return None, None, 0
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), nbytes
    if not (isinstance(workspace, torch.Tensor) and workspace.device == device and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous device tensor on the device of the call")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _call(fn, index, *args):
    """fn(*args, current stream) with the device of the call current."""
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch.cuda.current_device() == index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status != OK:
        _check(status)


def _kv_cache(k_cache, v_cache, layered):
    """(KvCache of the two pools after checking that they are one cache, device number)."""
    index = _index(k_cache, "k_cache")
    shape, dtype = k_cache.shape, k_cache.dtype
    if dtype not in _KV:
        raise TypeError(f"k_cache: dtype {dtype} not in {tuple(_KV)}")
    n = len(shape)
    if n != 5 and not (layered and n == 6):
        raise ValueError(f"k_cache: expected {'[layers, ' if layered else 'one layer ['}pages, heads, D/8, P, 8], got "
                         f"shape {tuple(shape)}")
    if n == 6:
        layers, pages, heads, blocks, page_size, eight = shape
        want = (layers, pages, heads, page_size // 8, blocks * 8, 8)
    else:
        layers = 1
        pages, heads, blocks, page_size, eight = shape
        want = (pages, heads, page_size // 8, blocks * 8, 8)
    if not isinstance(v_cache, torch.Tensor) or eight != 8 or v_cache.shape != want:
        raise ValueError(f"k_cache {tuple(shape)} and v_cache {tuple(getattr(v_cache, 'shape', ()))} are not one "
                         f"cache: keys [pages, heads, D/8, P, 8], values [pages, heads, P/8, D, 8]")
    k = _tensor(k_cache, "k_cache", dtype, shape, index)
    return KvCache(k, _tensor(v_cache, "v_cache", dtype, want, index), pages, layers, heads, blocks * 8, page_size,
                   _KV[dtype]), index


# a torch without these types serves every other call
_E4M3, _E8M0 = (getattr(torch, name, None) for name in ("float8_e4m3fn", "float8_e8m0fnu"))


def _need_8_bit_types():
    if _E4M3 is None or _E8M0 is None:
        raise TypeError("the cache in 8 bits needs torch.float8_e4m3fn and torch.float8_e8m0fnu, which this torch lacks")


def _type_of(q):
    """The 16-bit type of a call over an 8-bit cache: that of its queries."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if q.dtype not in _KV:
        raise TypeError(f"q: dtype {q.dtype} not in {tuple(_KV)}")
    return q.dtype


def _kv8_cache(k_cache, v_cache, k_scale, v_scale, dtype, layered):
    """(Kv8Cache of the pools and scales after checking that they are one cache, device number)."""
    _need_8_bit_types()
    index = _index(k_cache, "k_cache")
    shape = k_cache.shape
    n = len(shape)
    if n != 5 and not (layered and n == 6) or shape[-1] != 16:
        raise ValueError(f"k_cache: expected {'[layers, ' if layered else 'one layer ['}pages, heads, D/16, P, 16], got "
                         f"shape {tuple(shape)}")
    lead = tuple(shape[:-3])                                   # (layers,) pages, heads
    blocks, page_size = shape[-3], shape[-2]
    k = _tensor(k_cache, "k_cache", _E4M3, shape, index)
    v = _tensor(v_cache, "v_cache", _E4M3, lead + (page_size // 16, blocks * 16, 16), index)
    ks = _tensor(k_scale, "k_scale", _E8M0, lead + (page_size // 16,), index)
    vs = _tensor(v_scale, "v_scale", _E8M0, lead + (page_size // 16,), index)
    return Kv8Cache(k, v, ks, vs, lead[-2], lead[0] if n == 6 else 1, lead[-1], blocks * 16, page_size,
                    _KV[dtype]), index


def _kv_state(table, lengths, refs, pages, index):
    t = _tensor(table, "table", torch.int32, (None, None), index)
    seqs, width = table.shape
    return KvState(t, _tensor(lengths, "lengths", torch.int32, (seqs,), index),
                   None if refs is None else _tensor(refs, "refs", torch.int32, (pages,), index), seqs, width)


def _head_rows(t, name, heads, head_dim, dtype, index):
    """Address and row stride of [tokens, heads, D] whose rows may be a view of a wider tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, the cache holds {dtype}")
    shape = t.shape
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or shape[2] != head_dim:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [tokens, {heads or 'heads'}, {head_dim}]")
    if t.get_device() != index:
        raise ValueError(f"{name} must be a device tensor on the device of the call, is on {t.device}")
    n, h, _ = shape
    row, along, one = t.stride()
    if n and h and (one != 1 or (h > 1 and along != head_dim)):
        raise ValueError(f"{name}: the heads of a row must be contiguous, got strides {t.stride()}")
    return t.data_ptr(), row if n > 1 else h * head_dim


def _append(fn, cache, dev, dt, q, k, v, q_weight, k_weight, positions, inv_freq, slots, eps, interleaved, out):
    """What the two appends share; dt is the 16-bit type of the call."""
    D, i32 = cache.head_dim, torch.int32
    qp, qs = _head_rows(q, "q", None, D, dt, dev)
    kp, ks = _head_rows(k, "k", cache.heads, D, dt, dev)
    vp, vs = _head_rows(v, "v", cache.heads, D, dt, dev)
    N, hq = q.shape[0], q.shape[1]
    if k.shape[0] != N or v.shape[0] != N:
        raise ValueError(f"q, k and v have {N}, {k.shape[0]} and {v.shape[0]} tokens")
    wq = _tensor(q_weight, "q_weight", dt, (D,), dev)
    wk = _tensor(k_weight, "k_weight", dt, (D,), dev)
    inv = _tensor(inv_freq, "inv_freq", torch.float32, (None,), dev)
    pos = _tensor(positions, "positions", i32, (N,), dev)
    at = _tensor(slots, "slots", i32, (N,), dev)
    out, op = _result(out, "out", (N, hq, D), dt, q.device, dev)
    _call(fn, dev, qp, qs, kp, ks, vp, vs, wq, wk, pos, inv, 2 * inv_freq.shape[0], interleaved, eps, at, op,
          _byref(cache), N, hq)
    return out


def qk_norm_rope(q, k, v, q_weight, k_weight, positions, inv_freq, slots, k_cache, v_cache, eps=1e-6,
                 interleaved=False, out=None):
    """RMS norm of every head of q [N, Hq, D] and k [N, Hkv, D], rotation of the
    first 2 * len(inv_freq) dimensions by positions * inv_freq, and the append
    of k and v to the cache at `slots` (int32 [N], -1: not cached).  q, k and v
    may be views of one projection output.  Returns the queries [N, Hq, D]."""
    cache, dev = _kv_cache(k_cache, v_cache, False)
    return _append(load_library().trellis_qk_norm_rope, cache, dev, k_cache.dtype, q, k, v, q_weight, k_weight,
                   positions, inv_freq, slots, eps, interleaved, out)


def qk_norm_rope_kv8(q, k, v, q_weight, k_weight, positions, inv_freq, slots, k_cache, v_cache, k_scale, v_scale,
                     eps=1e-6, interleaved=False, out=None):
    """qk_norm_rope into a cache held in 8 bits.  Tokens whose slots lie in one
    block of 16 stand next to each other in the list, as cache_reserve gives
    them.  A block's scale grows with its tokens, and begins anew with its
    first slot."""
    dt = _type_of(q)
    cache, dev = _kv8_cache(k_cache, v_cache, k_scale, v_scale, dt, False)
    return _append(load_library().trellis_qk_norm_rope_kv8, cache, dev, dt, q, k, v, q_weight, k_weight, positions,
                   inv_freq, slots, eps, interleaved, out)


def _attention(q, cache, dev, dt, table, lengths, q_start, seq_ids, out):
    """What the attention calls share: (q's address and stride, state, addresses of seq_ids, q_start and out,
    entries, out)."""
    qp, stride = _head_rows(q, "q", None, cache.head_dim, dt, dev)
    state = _kv_state(table, lengths, None, cache.pages, dev)
    starts = _tensor(q_start, "q_start", torch.int32, (None,), dev)
    n = q_start.shape[0] - 1
    ids = None
    if seq_ids is not None:
        ids = _tensor(seq_ids, "seq_ids", torch.int32, (n,), dev)
    elif n > state.seqs:
        raise ValueError(f"q_start has {n} entries, the table {state.seqs} sequences")
    out, op = _result(out, "out", tuple(q.shape), dt, q.device, dev)
    return qp, stride, state, ids, starts, op, n, out


def _tree(fn, sizes, cache, dev, dt, q, table, lengths, q_start, ancestors, max_q, scale, seq_ids, out, workspace):
    qp, stride, state, ids, starts, op, n, out = _attention(q, cache, dev, dt, table, lengths, q_start, seq_ids, out)
    tokens, hq, D = q.shape
    anc = _tensor(ancestors, "ancestors", torch.int64, (tokens,), dev)
    c, s = _byref(cache), _byref(state)
    _keep, ws, wsb = _scratch(sizes(c, s, n, tokens, hq, max_q), q.device, workspace)
    _call(fn, dev, qp, stride, c, s, ids, n, starts, anc, tokens, hq, max_q, D ** -0.5 if scale is None else scale, op,
          ws, wsb)
    return out


def _window_numbers(max_q, window, sinks):
    for name, v in (("max_q", max_q), ("window", window), ("sinks", sinks)):
        _c_int(v, name)


def _window(fn, sizes, cache, dev, dt, q, table, lengths, q_start, max_q, window, sinks, scale, seq_ids, out,
            workspace):
    qp, stride, state, ids, starts, op, n, out = _attention(q, cache, dev, dt, table, lengths, q_start, seq_ids, out)
    tokens, hq, D = q.shape
    c, s = _byref(cache), _byref(state)
    _keep, ws, wsb = _scratch(sizes(c, s, n, tokens, hq, max_q, window, sinks), q.device, workspace)
    _call(fn, dev, qp, stride, c, s, ids, n, starts, tokens, hq, max_q, window, sinks,
          D ** -0.5 if scale is None else scale, op, ws, wsb)
    return out


def tree_attention(q, k_cache, v_cache, table, lengths, q_start, ancestors, max_q, scale=None, seq_ids=None, out=None,
                   workspace=None):
    """Attention of drafted tokens over the cache and their ancestors.  q [N, Hq,
    D]; entry e is sequence e (or seq_ids[e]) with rows q_start[e] ..
    q_start[e+1]-1, at most max_q (<= 64) of them, cached behind `lengths`.
    ancestors int64 [N]: bit m set if the row sees the entry's token m.  scale
    defaults to D ** -0.5.  Returns [N, Hq, D]."""
    _c_int(max_q, "max_q")
    cache, dev = _kv_cache(k_cache, v_cache, False)
    lib = load_library()
    return _tree(lib.trellis_tree_attention, lib.trellis_tree_attention_workspace_bytes, cache, dev, k_cache.dtype, q,
                 table, lengths, q_start, ancestors, max_q, scale, seq_ids, out, workspace)


def window_attention(q, k_cache, v_cache, table, lengths, q_start, max_q, window=0, sinks=0, scale=None, seq_ids=None,
                     out=None, workspace=None):
    """Causal attention of new tokens over the cache: the token at position p
    sees the keys j <= p with p - j < window (0: no limit) or j < sinks.
    Arguments otherwise as tree_attention; max_q has no upper bound."""
    _window_numbers(max_q, window, sinks)
    cache, dev = _kv_cache(k_cache, v_cache, False)
    lib = load_library()
    return _window(lib.trellis_window_attention, lib.trellis_window_attention_workspace_bytes, cache, dev,
                   k_cache.dtype, q, table, lengths, q_start, max_q, window, sinks, scale, seq_ids, out, workspace)


def tree_attention_kv8(q, k_cache, v_cache, k_scale, v_scale, table, lengths, q_start, ancestors, max_q, scale=None,
                       seq_ids=None, out=None, workspace=None):
    """tree_attention over a cache held in 8 bits; q and the result are bf16 or fp16."""
    _c_int(max_q, "max_q")
    dt = _type_of(q)
    cache, dev = _kv8_cache(k_cache, v_cache, k_scale, v_scale, dt, False)
    lib = load_library()
    return _tree(lib.trellis_tree_attention_kv8, lib.trellis_tree_attention_kv8_workspace_bytes, cache, dev, dt, q,
                 table, lengths, q_start, ancestors, max_q, scale, seq_ids, out, workspace)


def window_attention_kv8(q, k_cache, v_cache, k_scale, v_scale, table, lengths, q_start, max_q, window=0, sinks=0,
                         scale=None, seq_ids=None, out=None, workspace=None):
    """window_attention over a cache held in 8 bits; q and the result are bf16 or fp16."""
    _window_numbers(max_q, window, sinks)
    dt = _type_of(q)
    cache, dev = _kv8_cache(k_cache, v_cache, k_scale, v_scale, dt, False)
    lib = load_library()
    return _window(lib.trellis_window_attention_kv8, lib.trellis_window_attention_kv8_workspace_bytes, cache, dev, dt,
                   q, table, lengths, q_start, max_q, window, sinks, scale, seq_ids, out, workspace)


def kv_cache(layers, pages, heads, head_dim, page_size, dtype=torch.bfloat16, device="cuda"):
    """Empty pools (k_cache, v_cache) of `layers` layers; k_cache[i], v_cache[i] are one layer."""
    k = torch.zeros((layers, pages, heads, head_dim // 8, page_size, 8), dtype=dtype, device=device)
    return k, torch.zeros((layers, pages, heads, page_size // 8, head_dim, 8), dtype=dtype, device=device)


def kv8_cache(layers, pages, heads, head_dim, page_size, device="cuda"):
    """Empty pools and scales (k_cache, v_cache, k_scale, v_scale) of `layers` layers in 8 bits; [i] is one layer."""
    _need_8_bit_types()

    def zeros(dtype, *shape):
        return torch.zeros((layers, pages, heads) + shape, dtype=torch.uint8, device=device).view(dtype)

    return (zeros(_E4M3, head_dim // 16, page_size, 16), zeros(_E4M3, page_size // 16, head_dim, 16),
            zeros(_E8M0, page_size // 16), zeros(_E8M0, page_size // 16))


def kv_state(seqs, width, pages, device="cuda"):
    """Empty (table, lengths, refs): `seqs` sequences of at most `width` pages."""
    return (torch.full((seqs, width), -1, dtype=torch.int32, device=device),
            torch.zeros(seqs, dtype=torch.int32, device=device), torch.zeros(pages, dtype=torch.int32, device=device))


def _state_only(table, lengths, refs, page_size):
    """(cache without pools, state, device number) of the calls that touch no keys or values"""
    _c_int(page_size, "page_size")
    dev = _index(refs, "refs")
    if refs.dim() != 1:
        raise ValueError(f"refs: expected [pages], got shape {tuple(refs.shape)}")
    pages = refs.shape[0]
    return KvCache(None, None, pages, 1, 1, 64, page_size, KV_BF16), _kv_state(table, lengths, refs, pages, dev), dev


def cache_reserve(table, lengths, refs, page_size, seq_ids, q_start, tokens, slots=None, granted=None, workspace=None):
    """Slots for new tokens: entry b wants q_start[b+1] - q_start[b] tokens behind
    sequence seq_ids[b]; `tokens` in all.  Missing pages are taken from the free
    ones, lowest first.  Returns (slots int32 [tokens], -1 where refused,
    granted int32 [n])."""
    cache, state, dev = _state_only(table, lengths, refs, page_size)
    i32, device = torch.int32, refs.device
    ids = _tensor(seq_ids, "seq_ids", i32, (None,), dev)
    n = seq_ids.shape[0]
    starts = _tensor(q_start, "q_start", i32, (n + 1,), dev)
    slots, sp = _result(slots, "slots", (tokens,), i32, device, dev)
    granted, gp = _result(granted, "granted", (n,), i32, device, dev)
    lib, c, s = load_library(), _byref(cache), _byref(state)
    _keep, ws, wsb = _scratch(lib.trellis_cache_reserve_workspace_bytes(c, s, n), device, workspace)
    _call(lib.trellis_cache_reserve, dev, c, s, ids, n, starts, tokens, sp, gp, ws, wsb)
    return slots, granted


def _fork(fn, sizes, cache, dev, device, table, lengths, refs, parents, children, granted, workspace):
    state = _kv_state(table, lengths, refs, cache.pages, dev)
    par = _tensor(parents, "parents", torch.int32, (None,), dev)
    n = parents.shape[0]
    kid = _tensor(children, "children", torch.int32, (n,), dev)
    granted, gp = _result(granted, "granted", (n,), torch.int32, device, dev)
    c, s = _byref(cache), _byref(state)
    _keep, ws, wsb = _scratch(sizes(c, s, n), device, workspace)
    _call(fn, dev, c, s, par, kid, n, gp, ws, wsb)
    return granted


def cache_fork(k_cache, v_cache, table, lengths, refs, parents, children, granted=None, workspace=None):
    """children[b] becomes a copy of parents[b]: full pages shared, the last
    partial page copied in every layer.  Returns granted int32 [n]."""
    cache, dev = _kv_cache(k_cache, v_cache, True)
    lib = load_library()
    return _fork(lib.trellis_cache_fork, lib.trellis_cache_fork_workspace_bytes, cache, dev, k_cache.device, table,
                 lengths, refs, parents, children, granted, workspace)


def cache_fork_kv8(k_cache, v_cache, k_scale, v_scale, table, lengths, refs, parents, children, granted=None,
                   workspace=None):
    """cache_fork of a cache held in 8 bits."""
    cache, dev = _kv8_cache(k_cache, v_cache, k_scale, v_scale, torch.bfloat16, True)
    lib = load_library()
    return _fork(lib.trellis_cache_fork_kv8, lib.trellis_cache_fork_kv8_workspace_bytes, cache, dev, k_cache.device,
                 table, lengths, refs, parents, children, granted, workspace)


def _accept(fn, cache, dev, table, lengths, seq_ids, path, counts, new_lengths):
    state, i32 = _kv_state(table, lengths, None, cache.pages, dev), torch.int32
    ids = _tensor(seq_ids, "seq_ids", i32, (None,), dev)
    n = seq_ids.shape[0]
    pp = _tensor(path, "path", i32, (n, None), dev)
    cp = _tensor(counts, "counts", i32, (n,), dev)
    if new_lengths is None:
        new_lengths = lengths
    to = _tensor(new_lengths, "new_lengths", i32, (state.seqs,), dev)
    _call(fn, dev, _byref(cache), _byref(state), ids, n, pp, path.shape[1], cp, to)
    return new_lengths


def cache_accept(k_cache, v_cache, table, lengths, seq_ids, path, counts, new_lengths=None):
    """Drafted rows path[b][: counts[b]] of sequence seq_ids[b] move up behind its
    cached tokens in every layer; lengths grows by counts (in place, or into
    new_lengths).  Returns the new lengths."""
    cache, dev = _kv_cache(k_cache, v_cache, True)
    return _accept(load_library().trellis_cache_accept, cache, dev, table, lengths, seq_ids, path, counts, new_lengths)


def cache_accept_kv8(k_cache, v_cache, k_scale, v_scale, table, lengths, seq_ids, path, counts, new_lengths=None):
    """cache_accept in a cache held in 8 bits.  Blocks that rows move into take the
    largest scale of what they hold; their rows are rounded again under it."""
    cache, dev = _kv8_cache(k_cache, v_cache, k_scale, v_scale, torch.bfloat16, True)
    return _accept(load_library().trellis_cache_accept_kv8, cache, dev, table, lengths, seq_ids, path, counts,
                   new_lengths)


def cache_free(table, lengths, refs, seq_ids):
    """The pages of the listed sequences are returned; their rows become empty."""
    cache, state, dev = _state_only(table, lengths, refs, 16)
    ids = _tensor(seq_ids, "seq_ids", torch.int32, (None,), dev)
    _call(load_library().trellis_cache_free, dev, _byref(cache), _byref(state), ids, seq_ids.shape[0])


# ---- low-rank adapters -----------------------------------------------------
# As above, checks are one pass of plain comparisons: a call of three matrices
# has fifteen tensors.

_NAMES = {n: tuple(f"{n}[{k}]" for k in range(LORA_MAX)) for n in ("a", "b", "ys", "outs")}
_BF = torch.bfloat16


def _matrix_rows(t, name, rows, n, dtype, index):
    """Address and row stride of [rows, n] (None: any size) whose rows may lie in a wider tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    shape = t.shape
    if len(shape) != 2 or (rows is not None and (shape[0] != rows or shape[1] != n)):
        raise ValueError(f"{name}: shape {tuple(shape)}, expected "
                         f"{('any', 'any') if rows is None else (rows, n)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be a device tensor on the device of the call, is on {t.device}")
    row, one = t.stride()
    if one != 1 and shape[0] and shape[1] > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous, got strides {t.stride()}")
    return t.data_ptr(), row if shape[0] > 1 else shape[1]


def _lora(x, a, b, ys, starts, adapters, scales, ranks):
    """Checks what the two adapter calls share: (device number, x's address, stride, rows and columns, for every
    target the addresses of a, b and y with its outputs and stride, rank, pool, addresses of starts, adapters,
    scales and ranks, entries, the type of ys)."""
    dev, i32 = _index(x, "x"), torch.int32
    xp, xs = _matrix_rows(x, "x", None, None, _BF, dev)
    M, C = x.shape
    if not isinstance(a[0], torch.Tensor) or a[0].dim() != 3:
        raise ValueError("a: expected [pool, rank, in]")
    pool, rank, _ = a[0].shape
    dt = ys[0].dtype if isinstance(ys[0], torch.Tensor) else None
    if dt not in _F:
        raise TypeError(f"y: dtype {dt} not in {_F}")
    targets = []
    for k, y in enumerate(ys):
        bk = b[k]
        ap = _tensor(a[k], _NAMES["a"][k], _BF, (pool, rank, C), dev)
        bp = _tensor(bk, _NAMES["b"][k], _BF, (pool, None, rank), dev)
        R = bk.shape[1]
        yp, stride = _matrix_rows(y, _NAMES["ys"][k], M, R, dt, dev)
        targets.append((ap, bp, yp, R, stride))
    st = _tensor(starts, "starts", i32, (None,), dev)
    n = starts.shape[0] - 1
    ad = _tensor(adapters, "adapters", i32, (n,), dev)
    sc = _tensor(scales, "scales", torch.float32, (pool,), dev)
    rk = None if ranks is None else _tensor(ranks, "ranks", i32, (pool,), dev)
    return dev, xp, xs, M, C, targets, rank, pool, st, ad, sc, rk, n, dt


def lora_add(x, a, b, ys, starts, adapters, scales, ranks=None, outs=None, workspace=None):
    """outs[k] = ys[k] + scales[i] * B_i (A_i x) for every row, i the adapter of the
    row's entry: entry e has the rows starts[e] .. starts[e+1]-1 of x bf16 [M, C]
    and adapter adapters[e] (-1: none, outs = ys).  a and b are lists of the
    factors bf16 [pool, r, C] and [pool, R_k, r] of 1..4 projections of x, ys
    their outputs [M, R_k] (bf16 or f32; views of a wider tensor may be given).
    ranks int32 [pool]: adapters whose own rank is below r.  outs may be ys (in
    place); rows of no entry are not written.  Returns outs."""
    count = len(ys)
    if not 1 <= count <= LORA_MAX or len(a) != count or len(b) != count:
        raise ValueError(f"{len(a)} and {len(b)} factors for {count} projections (1..{LORA_MAX})")
    dev, xp, xs, M, C, targets, rank, pool, st, ad, sc, rk, n, dt = _lora(x, a, b, ys, starts, adapters, scales, ranks)
    if outs is None:
        outs = [torch.empty_like(y) if y.is_contiguous() else torch.empty(y.shape, dtype=dt, device=y.device) for y in ys]
        to = [(o.data_ptr(), t[3]) for o, t in zip(outs, targets)]
    elif len(outs) != count:
        raise ValueError(f"{len(outs)} outputs for {count} projections")
    else:
        to = [_matrix_rows(o, name, M, t[3], dt, dev) for o, name, t in zip(outs, _NAMES["outs"], targets)]
    packed = (LoraTarget * count)(*[(ap, bp, yp, op, R, stride, out_stride)
                                    for (ap, bp, yp, R, stride), (op, out_stride) in zip(targets, to)])
    lib = load_library()
    _keep, ws, wsb = _scratch(lib.trellis_lora_workspace_bytes(M, C, n, count, rank), x.device, workspace)
    _call(lib.trellis_lora_add, dev, xp, xs, packed, count, OUT_F32 if dt is torch.float32 else OUT_BF16, st, ad, n, sc,
          rk, pool, rank, M, C, ws, wsb)
    return outs


def lora_swiglu(x, a_gate, b_gate, a_up, b_up, gate, up, starts, adapters, scales, ranks=None, out=None,
                workspace=None):
    """bf16 silu(g) * u with g = gate + its adapter's part and u = up + its: gate and
    up [M, R] (bf16 or f32, such as gate_f32 and up_f32 of gateup_swiglu); the
    other arguments as lora_add.  Returns out [M, R]."""
    dev, xp, xs, M, C, targets, rank, pool, st, ad, sc, rk, n, dt = _lora(x, (a_gate, a_up), (b_gate, b_up), (gate, up),
                                                                          starts, adapters, scales, ranks)
    gate_t, up_t = (LoraTarget(ap, bp, yp, None, R, stride, 0) for ap, bp, yp, R, stride in targets)
    if out is None:
        out = torch.empty((M, gate_t.R), dtype=_BF, device=x.device)
    op, out_stride = _matrix_rows(out, "out", M, gate_t.R, _BF, dev)
    lib = load_library()
    _keep, ws, wsb = _scratch(lib.trellis_lora_workspace_bytes(M, C, n, 2, rank), x.device, workspace)
    _call(lib.trellis_lora_swiglu, dev, xp, xs, _byref(gate_t), _byref(up_t), op, out_stride,
          OUT_F32 if dt is torch.float32 else OUT_BF16, st, ad, n, sc, rk, pool, rank, M, C, ws, wsb)
    return out
