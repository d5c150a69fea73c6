"""ctypes binding over libqlinear's C ABI (``include/qlinear.h``).

Argument marshalling only: every step of the product runs in the HIP library.
Device arguments are torch CUDA tensors (PyTorch supplies device memory and the
stream); host helpers take numpy arrays. Each function has the name of the C
entry point it calls. A non-zero status raises ``QLinearError``. The library is
loaded on first use; if it is not built the call fails loudly (there is no
fallback of any kind).
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlinear.so")

QL_OK, QL_EINVAL, QL_EALIGN, QL_EUNSUPPORTED, QL_EWORKSPACE, QL_EHIP, QL_ERANGE = 0, -1, -2, -3, -4, -5, -6
QL_OUT_F32, QL_OUT_BF16 = 0, 1
QL_PATH_AUTO, QL_PATH_SKINNY, QL_PATH_GEMM, QL_PATH_SPLITK = 0, 1, 2, 3
QL_LAYOUT_CANONICAL, QL_LAYOUT_TILED = 0, 1
QL_MODE_AUTO, QL_MODE_EXACT, QL_MODE_FAST, QL_MODE_SPLIT = 0, 1, 2, 3
QL_EPI_NONE, QL_EPI_SWIGLU, QL_EPI_GATE_RESIDUAL = 0, 1, 2
QL_NORM_NONE, QL_NORM_RMS, QL_NORM_LAYER = 0, 1, 2
QL_ADAPTER_BF16, QL_ADAPTER_F16 = 0, 1

EXPORTED = (
    "qlinear_forward", "qlinear_forward_ex", "qlinear_workspace_bytes", "qlinear_packed_words",
    "qlinear_pack_host", "qlinear_unpack_host", "qlinear_quantize_rtn_host", "qlinear_quantize_rtn",
    "qlinear_dequantize", "qlinear_status_string", "qlinear_last_path", "qlinear_version",
    "qlinear_group_sums", "qlinear_group_sums_ld", "qlinear_tiled_words", "qlinear_tiled_sb_words",
    "qlinear_repack", "qlinear_unrepack", "qlinear_fast_activations", "qlinear_fast_activations_adaln",
    "qlinear_repack_glu",
    "qlinear_unrepack_glu", "qlinear_quantize_imatrix", "qlinear_forward_workspace_bytes",
    "qlinear_forward_noalloc", "qlinear_forward_noalloc_max_scratch",
    "qlinear_block_norm", "qlinear_adapters", "qlinear_adapters_workspace_bytes",
)


class QLinearError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({qlinear_status_string(status)})")


class ql_forward_args(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("packed_q", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("biases", ctypes.c_void_p),
        ("bits", ctypes.c_int),
        ("group", ctypes.c_int),
        ("M", ctypes.c_int64),
        ("N", ctypes.c_int64),
        ("K", ctypes.c_int64),
        ("out", ctypes.c_void_p),
        ("out_dtype", ctypes.c_int),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("path", ctypes.c_int),
        ("split_k", ctypes.c_int),
        ("tile", ctypes.c_int),
        ("xsum", ctypes.c_void_p),
        ("ld_xsum", ctypes.c_int64),
        ("layout", ctypes.c_int),
        ("mode", ctypes.c_int),
        ("x16", ctypes.c_void_p),
        ("rowscale", ctypes.c_void_p),
        ("epilogue", ctypes.c_int),
        ("residual", ctypes.c_void_p),
        ("gate", ctypes.c_void_p),
        ("gate_rows", ctypes.c_int64),
    ]


class ql_block_norm_args(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int64),
        ("D", ctypes.c_int64),
        ("residual", ctypes.c_void_p),
        ("residual_dtype", ctypes.c_int),
        ("residual_scale", ctypes.c_float),
        ("y", ctypes.c_void_p),
        ("y_dtype", ctypes.c_int),
        ("post_norm", ctypes.c_int),
        ("post_eps", ctypes.c_float),
        ("post_weight", ctypes.c_void_p),
        ("post_bias", ctypes.c_void_p),
        ("gate", ctypes.c_void_p),
        ("gate_ld", ctypes.c_int64),
        ("residual_out", ctypes.c_void_p),
        ("pre_norm", ctypes.c_int),
        ("pre_eps", ctypes.c_float),
        ("pre_weight", ctypes.c_void_p),
        ("pre_bias", ctypes.c_void_p),
        ("scale", ctypes.c_void_p),
        ("scale_ld", ctypes.c_int64),
        ("shift", ctypes.c_void_p),
        ("shift_ld", ctypes.c_int64),
        ("mod_rows", ctypes.c_int64),
        ("row_sample", ctypes.c_void_p),
        ("samples", ctypes.c_int64),
        ("h", ctypes.c_void_p),
        ("x16", ctypes.c_void_p),
        ("rowscale", ctypes.c_void_p),
    ]


class ql_adapter_args(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("a", ctypes.c_void_p),
        ("b", ctypes.c_void_p),
        ("ab_dtype", ctypes.c_int),
        ("M", ctypes.c_int64),
        ("N", ctypes.c_int64),
        ("K", ctypes.c_int64),
        ("adapters", ctypes.c_int64),
        ("rank", ctypes.c_int64),
        ("row_adapter", ctypes.c_void_p),
        ("ranks", ctypes.c_void_p),
        ("scaling", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("y_dtype", ctypes.c_int),
        ("out", ctypes.c_void_p),
        ("out_dtype", ctypes.c_int),
        ("epilogue", ctypes.c_int),
        ("residual", ctypes.c_void_p),
        ("gate", ctypes.c_void_p),
        ("gate_rows", ctypes.c_int64),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load (once) and return libqlinear with argument types declared."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"libqlinear.so not found at {path}; build it with "
            "`python -m group_wise_affine_qlinear_amd.build` (hipcc, gfx950)")
    # torch ships its own HIP runtime; loading it first makes the library bind
    # to that same runtime, so device pointers and streams from torch are valid
    # in the library's calls (a second runtime instance would not know them)
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    lib = ctypes.CDLL(path)
    i64, vp, i32, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    sig = {
        "qlinear_forward": ([vp, vp, vp, vp, i32, i32, i64, i64, i64, vp], i32),
        "qlinear_forward_ex": ([ctypes.POINTER(ql_forward_args), vp], i32),
        "qlinear_workspace_bytes": ([i32, i64, i64, i64], sz),
        "qlinear_forward_workspace_bytes": ([ctypes.POINTER(ql_forward_args)], sz),
        "qlinear_forward_noalloc": ([ctypes.POINTER(ql_forward_args), vp], i32),
        "qlinear_forward_noalloc_max_scratch": ([], sz),
        "qlinear_packed_words": ([i32, i64, i64], sz),
        "qlinear_pack_host": ([vp, i32, i64, i64, vp], i32),
        "qlinear_unpack_host": ([vp, i32, i64, i64, vp], i32),
        "qlinear_quantize_rtn_host": ([vp, i32, i32, i64, i64, vp, vp, vp], i32),
        "qlinear_quantize_rtn": ([vp, i32, i32, i64, i64, vp, vp, vp, vp, vp], i32),
        "qlinear_quantize_imatrix": ([vp, vp, i32, i32, i64, i64, vp, vp, vp, vp, vp], i32),
        "qlinear_dequantize": ([vp, vp, vp, i32, i32, i64, i64, vp, vp], i32),
        "qlinear_status_string": ([i32], ctypes.c_char_p),
        "qlinear_last_path": ([ctypes.c_char_p, sz], i32),
        "qlinear_version": ([], i32),
        "qlinear_group_sums": ([vp, i64, i64, vp, i64, vp], i32),
        "qlinear_group_sums_ld": ([i64], i64),
        "qlinear_fast_activations": ([vp, i64, i64, vp, vp, vp], i32),
        "qlinear_fast_activations_adaln": ([vp, vp, i64, i64, i64, vp, vp, vp], i32),
        "qlinear_tiled_words": ([i32, i64, i64], sz),
        "qlinear_tiled_sb_words": ([i64, i64], sz),
        "qlinear_repack": ([vp, vp, vp, i32, i32, i64, i64, vp, vp, vp], i32),
        "qlinear_unrepack": ([vp, vp, i32, i32, i64, i64, vp, vp, vp, vp], i32),
        "qlinear_repack_glu": ([vp, vp, vp, i32, i32, i64, i64, vp, vp, vp], i32),
        "qlinear_unrepack_glu": ([vp, vp, i32, i32, i64, i64, vp, vp, vp, vp], i32),
        "qlinear_block_norm": ([ctypes.POINTER(ql_block_norm_args), vp], i32),
        "qlinear_adapters": ([ctypes.POINTER(ql_adapter_args), vp], i32),
        "qlinear_adapters_workspace_bytes": ([i64, i64, i64, i64, i64], sz),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != QL_OK:
        raise QLinearError(status, where)


# ------------------------------------------------------------------ torch helpers

def _torch():
    import torch
    return torch


def _dev_ptr(t, name, dtypes, shape=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _stream_handle(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _u16(torch):
    return (torch.int16, torch.uint16, torch.float16, torch.bfloat16)


def _empty(torch, shape, dtype, device, stream):
    """Memory of a call on ``stream`` (None: the current one) from torch's caching allocator. Taken under the
    call's own stream: the allocator orders the users of a block by the stream it was taken on alone, so a block of
    the current stream may still be in use there when a call on another stream begins to write it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _result(torch, shape, dtype, device, stream):
    """Memory of a call on ``stream`` that is returned to the caller, who may go on with it on the current stream:
    kept from reuse until what is queued there when it is freed has run."""
    t = _empty(torch, shape, dtype, device, stream)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(device))
    return t


# ------------------------------------------------------------------ device entry points

def qlinear_forward(x, packed_q, scales, biases, bits, group, M, N, K, out):
    """C ``qlinear_forward``: out[M, N] fp32 = x[M, K] (bf16) @ W_hat^T, default stream."""
    torch = _torch()
    u16 = _u16(torch)
    lib = load_library()
    G = K // group if group else 0
    st = lib.qlinear_forward(
        _dev_ptr(x, "x", u16, (M, K)),
        _dev_ptr(packed_q, "packed_q", (torch.int32, torch.uint32), (N, K * bits // 32)),
        _dev_ptr(scales, "scales", u16, (N, G)),
        _dev_ptr(biases, "biases", u16, (N, G)),
        bits, group, M, N, K,
        _dev_ptr(out, "out", (torch.float32,), (M, N)))
    _check(st, "qlinear_forward")
    return out


# Default of ``qlinear_forward_ex(workspace=...)``: a workspace of
# ``qlinear_workspace_bytes`` taken from torch's caching allocator for the call.
TORCH_WORKSPACE = "torch"


def qlinear_forward_ex(x, packed_q, scales, biases, bits, M, N, K, out, *, group=64,
                       workspace=TORCH_WORKSPACE, stream=None, path=QL_PATH_AUTO, split_k=0, tile=0,
                       xsum=None, layout=QL_LAYOUT_CANONICAL, mode=QL_MODE_AUTO, x16=None,
                       rowscale=None, epilogue=QL_EPI_NONE, residual=None, gate=None, gate_rows=0):
    """C ``qlinear_forward_ex``: explicit stream, workspace, out dtype, layout, numerics mode
    and forced path.

    With ``layout=QL_LAYOUT_TILED``, ``packed_q`` and ``scales`` are the outputs of
    ``qlinear_repack`` (tiled codes, tiled scale|bias words) and ``biases`` is ignored.
    ``mode`` is a ``ql_mode`` (AUTO: FAST for the large-M path; with no workspace and no
    ``x16`` the GEMM converts x to fp16 itself). ``workspace`` is a device tensor the library may use
    as scratch, ``None`` (the call keeps to plans that need none, as the C call with a NULL
    workspace), or by default a tensor of ``qlinear_workspace_bytes`` bytes that torch's caching
    allocator provides on the call's stream (the library itself never allocates);
    ``x16``/``rowscale`` are optional FAST-mode activations from ``qlinear_fast_activations``.
    ``epilogue=QL_EPI_SWIGLU`` takes GLU-ordered tiled weights (``qlinear_repack_glu``) and
    writes ``out`` [M, N/2] = silu(gate) * up. ``epilogue=QL_EPI_GATE_RESIDUAL`` writes
    ``out`` = ``residual`` + ``gate``[m // ``gate_rows``] * y (``residual`` [M, N] of out's
    dtype, may be ``out``; ``gate`` fp32 [ceil(M / gate_rows), N]).
    """
    torch = _torch()
    u16 = _u16(torch)
    lib = load_library()
    G = K // group if group else 0
    a = ql_forward_args()
    a.x = _dev_ptr(x, "x", u16, (M, K))
    a.layout = layout
    if layout == QL_LAYOUT_TILED:
        a.packed_q = _dev_ptr(packed_q, "packed_q", (torch.int32, torch.uint32), (qlinear_tiled_words(bits, N, K),))
        a.scales = _dev_ptr(scales, "scales", (torch.int32, torch.uint32), (qlinear_tiled_sb_words(N, K),))
        a.biases = None
    else:
        a.packed_q = _dev_ptr(packed_q, "packed_q", (torch.int32, torch.uint32), (N, K * bits // 32))
        a.scales = _dev_ptr(scales, "scales", u16, (N, G))
        a.biases = _dev_ptr(biases, "biases", u16, (N, G))
    a.bits, a.group, a.M, a.N, a.K = bits, group, M, N, K
    if out.dtype == torch.float32:
        a.out_dtype = QL_OUT_F32
    elif out.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        a.out_dtype = QL_OUT_BF16
    else:
        raise TypeError("out must be float32 or bfloat16")
    a.epilogue = epilogue
    a.out = _dev_ptr(out, "out", (out.dtype,), (M, N // 2 if epilogue == QL_EPI_SWIGLU else N))
    if isinstance(workspace, str):
        if workspace != TORCH_WORKSPACE:
            raise ValueError(f"workspace must be a device tensor, None or {TORCH_WORKSPACE!r}")
        workspace = None
        nbytes = -1   # sized below, once every field of the call is set
    else:
        nbytes = None
    a.path, a.split_k, a.tile, a.mode = path, split_k, tile, mode
    if xsum is not None:
        a.xsum = _dev_ptr(xsum, "xsum", (torch.float32,))
        a.ld_xsum = xsum.shape[1]
        if xsum.dim() != 2 or xsum.shape[0] != K // group:
            raise ValueError("xsum must be [K/64, ld_xsum]")
    if epilogue == QL_EPI_GATE_RESIDUAL:
        a.gate_rows = gate_rows
        if residual is not None:
            a.residual = _dev_ptr(residual, "residual", (out.dtype,), (M, N))
        if gate is not None and gate_rows >= 1:
            a.gate = _dev_ptr(gate, "gate", (torch.float32,), (-(-M // gate_rows), N))
    if x16 is not None:
        a.x16 = _dev_ptr(x16, "x16", (torch.float16, torch.int16), (M, K))
        a.rowscale = _dev_ptr(rowscale, "rowscale", (torch.float32,), (M,))
    if nbytes == -1:
        nbytes = int(lib.qlinear_forward_workspace_bytes(ctypes.byref(a)))
        if nbytes > 0:
            workspace = _empty(torch, nbytes, torch.uint8, x.device, stream)
    if workspace is not None:
        a.workspace = _dev_ptr(workspace, "workspace", (workspace.dtype,))
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    st = lib.qlinear_forward_ex(ctypes.byref(a), _stream_handle(stream))
    _check(st, "qlinear_forward_ex")
    return out


def qlinear_group_sums_ld(M) -> int:
    return int(load_library().qlinear_group_sums_ld(M))


def qlinear_group_sums(x, M, K, xsum=None, stream=None):
    """C ``qlinear_group_sums``: per-group row sums of x, [K/64, ld] fp32 (allocated if None)."""
    torch = _torch()
    lib = load_library()
    ld = qlinear_group_sums_ld(M)
    if xsum is None:
        xsum = _result(torch, (K // 64, ld), torch.float32, x.device, stream)
    st = lib.qlinear_group_sums(_dev_ptr(x, "x", _u16(torch), (M, K)), M, K,
                                _dev_ptr(xsum, "xsum", (torch.float32,)), xsum.shape[1],
                                _stream_handle(stream))
    _check(st, "qlinear_group_sums")
    return xsum


def qlinear_fast_activations(x, M, K, x16=None, rowscale=None, stream=None):
    """C ``qlinear_fast_activations``: fp16 x with per-row power-of-two scales (FAST mode)."""
    torch = _torch()
    lib = load_library()
    if x16 is None:
        x16 = _result(torch, (M, K), torch.float16, x.device, stream)
    if rowscale is None:
        rowscale = _result(torch, (M,), torch.float32, x.device, stream)
    st = lib.qlinear_fast_activations(_dev_ptr(x, "x", _u16(torch), (M, K)), M, K,
                                      _dev_ptr(x16, "x16", (torch.float16, torch.int16), (M, K)),
                                      _dev_ptr(rowscale, "rowscale", (torch.float32,), (M,)),
                                      _stream_handle(stream))
    _check(st, "qlinear_fast_activations")
    return x16, rowscale


def qlinear_fast_activations_adaln(x, scale, scale_rows, M, K, x16=None, rowscale=None, stream=None):
    """C ``qlinear_fast_activations_adaln``: FAST-mode activations of x * (1 + scale[m // scale_rows])."""
    torch = _torch()
    lib = load_library()
    if x16 is None:
        x16 = _result(torch, (M, K), torch.float16, x.device, stream)
    if rowscale is None:
        rowscale = _result(torch, (M,), torch.float32, x.device, stream)
    samples = -(-M // scale_rows) if scale_rows > 0 else 0
    st = lib.qlinear_fast_activations_adaln(_dev_ptr(x, "x", _u16(torch), (M, K)),
                                            _dev_ptr(scale, "scale", (torch.float32,), (samples, K)),
                                            scale_rows, M, K,
                                            _dev_ptr(x16, "x16", (torch.float16, torch.int16), (M, K)),
                                            _dev_ptr(rowscale, "rowscale", (torch.float32,), (M,)),
                                            _stream_handle(stream))
    _check(st, "qlinear_fast_activations_adaln")
    return x16, rowscale


def qlinear_tiled_words(bits, N, K) -> int:
    return int(load_library().qlinear_tiled_words(bits, N, K))


def qlinear_tiled_sb_words(N, K) -> int:
    return int(load_library().qlinear_tiled_sb_words(N, K))


def qlinear_repack(packed_q, scales, biases, bits, group, N, K, tiled_q=None, tiled_sb=None, stream=None):
    """C ``qlinear_repack``: canonical -> tiled; returns (tiled_q, tiled_sb) int32 tensors."""
    torch = _torch()
    u16 = _u16(torch)
    lib = load_library()
    dev = packed_q.device
    if tiled_q is None:
        tiled_q = _result(torch, (qlinear_tiled_words(bits, N, K),), torch.int32, dev, stream)
    if tiled_sb is None:
        tiled_sb = _result(torch, (qlinear_tiled_sb_words(N, K),), torch.int32, dev, stream)
    st = lib.qlinear_repack(
        _dev_ptr(packed_q, "packed_q", (torch.int32, torch.uint32), (N, K * bits // 32)),
        _dev_ptr(scales, "scales", u16, (N, K // group)),
        _dev_ptr(biases, "biases", u16, (N, K // group)), bits, group, N, K,
        _dev_ptr(tiled_q, "tiled_q", (torch.int32, torch.uint32), (qlinear_tiled_words(bits, N, K),)),
        _dev_ptr(tiled_sb, "tiled_sb", (torch.int32, torch.uint32), (qlinear_tiled_sb_words(N, K),)),
        _stream_handle(stream))
    _check(st, "qlinear_repack")
    return tiled_q, tiled_sb


def qlinear_repack_glu(packed_q, scales, biases, bits, group, N, K, tiled_q=None, tiled_sb=None, stream=None):
    """C ``qlinear_repack_glu``: stacked [gate; up] canonical weight -> tiled GLU order."""
    torch = _torch()
    u16 = _u16(torch)
    lib = load_library()
    dev = packed_q.device
    if tiled_q is None:
        tiled_q = _result(torch, (qlinear_tiled_words(bits, N, K),), torch.int32, dev, stream)
    if tiled_sb is None:
        tiled_sb = _result(torch, (qlinear_tiled_sb_words(N, K),), torch.int32, dev, stream)
    st = lib.qlinear_repack_glu(
        _dev_ptr(packed_q, "packed_q", (torch.int32, torch.uint32), (N, K * bits // 32)),
        _dev_ptr(scales, "scales", u16, (N, K // group)),
        _dev_ptr(biases, "biases", u16, (N, K // group)), bits, group, N, K,
        _dev_ptr(tiled_q, "tiled_q", (torch.int32, torch.uint32), (qlinear_tiled_words(bits, N, K),)),
        _dev_ptr(tiled_sb, "tiled_sb", (torch.int32, torch.uint32), (qlinear_tiled_sb_words(N, K),)),
        _stream_handle(stream))
    _check(st, "qlinear_repack_glu")
    return tiled_q, tiled_sb


def qlinear_unrepack_glu(tiled_q, tiled_sb, bits, group, N, K, packed_q, scales, biases, stream=None):
    """C ``qlinear_unrepack_glu``: tiled GLU order -> stacked [gate; up] canonical, into the given tensors."""
    torch = _torch()
    u16 = _u16(torch)
    lib = load_library()
    st = lib.qlinear_unrepack_glu(
        _dev_ptr(tiled_q, "tiled_q", (torch.int32, torch.uint32), (qlinear_tiled_words(bits, N, K),)),
        _dev_ptr(tiled_sb, "tiled_sb", (torch.int32, torch.uint32), (qlinear_tiled_sb_words(N, K),)),
        bits, group, N, K,
        _dev_ptr(packed_q, "packed_q", (torch.int32, torch.uint32), (N, K * bits // 32)),
        _dev_ptr(scales, "scales", u16, (N, K // group)),
        _dev_ptr(biases, "biases", u16, (N, K // group)), _stream_handle(stream))
    _check(st, "qlinear_unrepack_glu")


def qlinear_unrepack(tiled_q, tiled_sb, bits, group, N, K, packed_q, scales, biases, stream=None):
    """C ``qlinear_unrepack``: tiled -> canonical into the given tensors."""
    torch = _torch()
    u16 = _u16(torch)
    lib = load_library()
    st = lib.qlinear_unrepack(
        _dev_ptr(tiled_q, "tiled_q", (torch.int32, torch.uint32), (qlinear_tiled_words(bits, N, K),)),
        _dev_ptr(tiled_sb, "tiled_sb", (torch.int32, torch.uint32), (qlinear_tiled_sb_words(N, K),)),
        bits, group, N, K,
        _dev_ptr(packed_q, "packed_q", (torch.int32, torch.uint32), (N, K * bits // 32)),
        _dev_ptr(scales, "scales", u16, (N, K // group)),
        _dev_ptr(biases, "biases", u16, (N, K // group)),
        _stream_handle(stream))
    _check(st, "qlinear_unrepack")


def qlinear_quantize_rtn(w, bits, group, N, K, packed_q, scales, biases, status=None, stream=None):
    """C ``qlinear_quantize_rtn``: device load-time RTN fit + pack."""
    torch = _torch()
    u16 = _u16(torch)
    lib = load_library()
    st = lib.qlinear_quantize_rtn(
        _dev_ptr(w, "w", (torch.float32,), (N, K)), bits, group, N, K,
        _dev_ptr(packed_q, "packed_q", (torch.int32, torch.uint32), (N, K * bits // 32)),
        _dev_ptr(scales, "scales", u16, (N, K // group)),
        _dev_ptr(biases, "biases", u16, (N, K // group)),
        _dev_ptr(status, "status", (torch.int32,)) if status is not None else None,
        _stream_handle(stream))
    _check(st, "qlinear_quantize_rtn")


def qlinear_quantize_imatrix(w, importance, bits, group, N, K, packed_q, scales, biases, status=None, stream=None):
    """C ``qlinear_quantize_imatrix``: device importance-weighted fit + pack (importance fp32 [K])."""
    torch = _torch()
    u16 = _u16(torch)
    lib = load_library()
    st = lib.qlinear_quantize_imatrix(
        _dev_ptr(w, "w", (torch.float32,), (N, K)),
        _dev_ptr(importance, "importance", (torch.float32,), (K,)), bits, group, N, K,
        _dev_ptr(packed_q, "packed_q", (torch.int32, torch.uint32), (N, K * bits // 32)),
        _dev_ptr(scales, "scales", u16, (N, K // group)),
        _dev_ptr(biases, "biases", u16, (N, K // group)),
        _dev_ptr(status, "status", (torch.int32,)) if status is not None else None,
        _stream_handle(stream))
    _check(st, "qlinear_quantize_imatrix")


def qlinear_dequantize(packed_q, scales, biases, bits, group, N, K, w_out, stream=None):
    """C ``qlinear_dequantize``: W_hat fp32 [N, K]."""
    torch = _torch()
    u16 = _u16(torch)
    lib = load_library()
    st = lib.qlinear_dequantize(
        _dev_ptr(packed_q, "packed_q", (torch.int32, torch.uint32), (N, K * bits // 32)),
        _dev_ptr(scales, "scales", u16, (N, K // group)),
        _dev_ptr(biases, "biases", u16, (N, K // group)),
        bits, group, N, K,
        _dev_ptr(w_out, "w_out", (torch.float32,), (N, K)),
        _stream_handle(stream))
    _check(st, "qlinear_dequantize")
    return w_out


# ------------------------------------------------------------------ around a projection

def _operand(t, name, dtypes, shape, device):
    """Data pointer of a contiguous tensor of one of the dtypes, of this shape, on this device."""
    if getattr(t, "device", None) == device and t.dtype in dtypes and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _dev_ptr(t, name, dtypes, shape)
    raise ValueError(f"{name} is on {t.device}, expected {device}")


def _value_dtype(torch, t, name):
    """ql_out_dtype of a stream of values."""
    dtype = t.dtype
    if dtype is torch.float32:
        return QL_OUT_F32
    if dtype is torch.bfloat16:
        return QL_OUT_BF16
    raise TypeError(f"{name} must be float32 or bfloat16")


def _modulation(torch, t, name, rows, D, device):
    """(pointer, row pitch) of a [samples, D] fp32 tensor whose rows may be slices of longer ones."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32:
        raise TypeError(f"{name} must be a float32 tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    shape = t.shape
    if len(shape) != 2 or shape[1] != D or shape[0] < rows:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected [>= {rows}, {D}]")
    pitch, step = t.stride()
    if (D > 1 and step != 1) or (shape[0] > 1 and pitch < D):
        raise ValueError(f"{name} must have rows of consecutive values that do not overlap")
    return t.data_ptr(), pitch if pitch > D else D


def _launch(torch, fn, where, args, device, stream):
    """Calls a C entry point on `stream` (default: the current stream of the tensors' device) with that device current."""
    if stream is None:
        # the handle alone: a torch Stream object costs as much as the rest of a small call's checks
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        handle = raw(device.index) if raw else torch.cuda.current_stream(device).cuda_stream
    elif isinstance(stream, int):
        handle = stream
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, expected {device}")
    else:
        handle = stream.cuda_stream
    if torch.cuda.current_device() == device.index:
        st = fn(ctypes.byref(args), handle)
    else:
        with torch.cuda.device(device):
            st = fn(ctypes.byref(args), handle)
    if st != QL_OK:
        raise QLinearError(st, where)


def qlinear_block_norm(residual, M, D, *, y=None, residual_scale=1.0, post_norm=QL_NORM_NONE, post_eps=1e-6,
                       post_weight=None, post_bias=None, gate=None, residual_out=None, pre_norm=QL_NORM_NONE,
                       pre_eps=1e-6, pre_weight=None, pre_bias=None, scale=None, shift=None, mod_rows=0,
                       row_sample=None, samples=None, h=None, x16=None, rowscale=None, stream=None):
    """C ``qlinear_block_norm``: the norms before and after a block with modulation, gate and residual.

    ``z = N_post(y) * post_weight + post_bias``; ``r = residual_scale * residual + gate[s] * z`` goes to
    ``residual_out`` (may be ``residual``); ``h = (N_pre(r) * pre_weight + pre_bias) * (1 + scale[s]) + shift[s]``
    goes to ``h`` (bf16) and/or ``x16``/``rowscale`` (FAST activations). ``residual``, ``residual_out`` and ``y``
    are fp32 or bf16 [M, D]; ``gate``, ``scale`` and ``shift`` fp32 [samples, D], slices of a wider modulation
    output included. The sample of row m is ``m // mod_rows`` (``mod_rows`` 0: one sample) or ``row_sample[m]``
    (int32); a row whose sample is outside [0, samples) is left as it is. ``samples`` defaults to the rows of
    the modulation arrays given with ``row_sample``.
    """
    torch = _torch()
    lib = load_library()
    if not isinstance(residual, torch.Tensor):
        raise TypeError("residual must be a torch tensor")
    dev = residual.device
    shape = (M, D)
    f32, stream_types = (torch.float32,), (torch.float32, torch.bfloat16)
    a = ql_block_norm_args()
    a.M, a.D, a.residual_scale = M, D, residual_scale
    a.residual = _operand(residual, "residual", stream_types, shape, dev)
    a.residual_dtype = _value_dtype(torch, residual, "residual")
    if dev.type != "cuda":
        raise ValueError("residual must be a device tensor")
    if y is not None:
        a.y = _operand(y, "y", stream_types, shape, dev)
        a.y_dtype = _value_dtype(torch, y, "y")
    a.post_norm, a.post_eps, a.pre_norm, a.pre_eps = post_norm, post_eps, pre_norm, pre_eps
    if post_weight is not None:
        a.post_weight = _operand(post_weight, "post_weight", f32, (D,), dev)
    if post_bias is not None:
        a.post_bias = _operand(post_bias, "post_bias", f32, (D,), dev)
    if pre_weight is not None:
        a.pre_weight = _operand(pre_weight, "pre_weight", f32, (D,), dev)
    if pre_bias is not None:
        a.pre_bias = _operand(pre_bias, "pre_bias", f32, (D,), dev)
    if row_sample is not None:
        a.row_sample = _operand(row_sample, "row_sample", (torch.int32,), (M,), dev)
        if samples is None:
            given = [t for t in (gate, scale, shift) if t is not None]
            if not given:
                raise ValueError("row_sample without gate, scale or shift needs samples")
            if not all(isinstance(t, torch.Tensor) and t.dim() == 2 for t in given):
                raise TypeError(f"gate, scale and shift must be float32 tensors [samples, {D}]")
            samples = min(t.shape[0] for t in given)
        a.samples = need = samples
    else:
        a.mod_rows = mod_rows
        need = -(-M // mod_rows) if mod_rows > 0 else 1
    if gate is not None:
        a.gate, a.gate_ld = _modulation(torch, gate, "gate", need, D, dev)
    if scale is not None:
        a.scale, a.scale_ld = _modulation(torch, scale, "scale", need, D, dev)
    if shift is not None:
        a.shift, a.shift_ld = _modulation(torch, shift, "shift", need, D, dev)
    if residual_out is not None:
        a.residual_out = _operand(residual_out, "residual_out", (residual.dtype,), shape, dev)
    if h is not None:
        a.h = _operand(h, "h", (torch.bfloat16,), shape, dev)
    if x16 is not None:
        a.x16 = _operand(x16, "x16", (torch.float16,), shape, dev)
    if rowscale is not None:
        a.rowscale = _operand(rowscale, "rowscale", f32, (M,), dev)
    _launch(torch, lib.qlinear_block_norm, "qlinear_block_norm", a, dev, stream)


def qlinear_adapters_workspace_bytes(M, N, K, rank, adapters) -> int:
    return int(load_library().qlinear_adapters_workspace_bytes(M, N, K, rank, adapters))


def qlinear_adapters(x, a, b, row_adapter, M, N, K, out, *, y=None, ranks=None, scaling=None, epilogue=QL_EPI_NONE,
                     residual=None, gate=None, gate_rows=0, workspace=TORCH_WORKSPACE, stream=None):
    """C ``qlinear_adapters``: low-rank adapters of many requests beside a projection they share.

    ``t[m] = y[m] + scaling[id] * b[id] @ (a[id] @ x[m])`` with ``id = row_adapter[m]`` (int32; outside the
    table: no adapter), then ``out = t`` or an epilogue of it. ``x`` bf16 [M, K] (``x`` and ``b`` may be None
    where nothing of them is read: an empty table, or for ``x`` K = 0); ``a`` [adapters, rank, K] and
    ``b`` [adapters, N, rank], both bf16 or both fp16; ``ranks`` int32 and ``scaling`` fp32 [adapters]; ``y``
    [M, N] and ``out`` fp32 or bf16 (``out`` may be ``y``). ``epilogue=QL_EPI_SWIGLU`` writes ``out`` [M, N/2]
    = silu(t[:, :N/2]) * t[:, N/2:]; ``epilogue=QL_EPI_GATE_RESIDUAL`` writes ``residual`` +
    ``gate``[m // ``gate_rows``] * t. ``workspace`` is a device tensor of
    ``qlinear_adapters_workspace_bytes`` bytes, by default one from torch's caching allocator on the call's stream.
    """
    torch = _torch()
    lib = load_library()
    for t, name in ((a, "a"), (out, "out")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
    if a.dim() != 3:
        raise ValueError("a must be a tensor [adapters, rank, K]")
    dev = out.device
    if dev.type != "cuda":
        raise ValueError("out must be a device tensor")
    n, rank = a.shape[0], a.shape[1]
    f = ql_adapter_args()
    f.M, f.N, f.K, f.adapters, f.rank = M, N, K, n, rank
    if a.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("a must be bfloat16 or float16")
    f.ab_dtype = QL_ADAPTER_F16 if a.dtype == torch.float16 else QL_ADAPTER_BF16
    if x is not None or (n > 0 and K > 0):  # not read otherwise
        f.x = _operand(x, "x", (torch.bfloat16, torch.int16, torch.uint16), (M, K), dev)
    f.a = _operand(a, "a", (a.dtype,), (n, rank, K), dev)
    if b is not None or n > 0:
        f.b = _operand(b, "b", (a.dtype,), (n, N, rank), dev)
    f.row_adapter = _operand(row_adapter, "row_adapter", (torch.int32,), (M,), dev)
    if ranks is not None:
        f.ranks = _operand(ranks, "ranks", (torch.int32,), (n,), dev)
    if scaling is not None:
        f.scaling = _operand(scaling, "scaling", (torch.float32,), (n,), dev)
    if y is not None:
        f.y = _operand(y, "y", (torch.float32, torch.bfloat16), (M, N), dev)
        f.y_dtype = _value_dtype(torch, y, "y")
    f.out_dtype = _value_dtype(torch, out, "out")
    f.out = _operand(out, "out", (out.dtype,), (M, N // 2 if epilogue == QL_EPI_SWIGLU else N), dev)
    f.epilogue = epilogue
    if epilogue == QL_EPI_GATE_RESIDUAL:
        f.gate_rows = gate_rows
        if residual is not None:
            f.residual = _operand(residual, "residual", (out.dtype,), (M, N), dev)
        if gate is not None and gate_rows >= 1:
            f.gate = _operand(gate, "gate", (torch.float32,), (-(-M // gate_rows), N), dev)
    if isinstance(workspace, str):
        if workspace != TORCH_WORKSPACE:
            raise ValueError(f"workspace must be a device tensor, None or {TORCH_WORKSPACE!r}")
        nbytes = lib.qlinear_adapters_workspace_bytes(M, N, K, rank, n)
        workspace = _empty(torch, nbytes, torch.uint8, dev, stream) if nbytes else None
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor):
            raise TypeError(f"workspace must be a device tensor, None or {TORCH_WORKSPACE!r}")
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        f.workspace = workspace.data_ptr()
        f.workspace_bytes = workspace.numel() * workspace.element_size()
    _launch(torch, lib.qlinear_adapters, "qlinear_adapters", f, dev, stream)
    return out


# ------------------------------------------------------------------ host entry points

def qlinear_packed_words(bits, N, K) -> int:
    return int(load_library().qlinear_packed_words(bits, N, K))


def qlinear_workspace_bytes(bits, M, N, K) -> int:
    return int(load_library().qlinear_workspace_bytes(bits, M, N, K))


def qlinear_pack_host(q: np.ndarray, bits: int) -> np.ndarray:
    q = np.ascontiguousarray(q, dtype=np.uint8)
    n, k = q.shape
    out = np.empty((n, k * bits // 32), dtype=np.uint32)
    _check(load_library().qlinear_pack_host(q.ctypes.data, bits, n, k, out.ctypes.data), "qlinear_pack_host")
    return out


def qlinear_unpack_host(packed: np.ndarray, bits: int, K: int) -> np.ndarray:
    packed = np.ascontiguousarray(packed, dtype=np.uint32)
    n = packed.shape[0]
    out = np.empty((n, K), dtype=np.uint8)
    _check(load_library().qlinear_unpack_host(packed.ctypes.data, bits, n, K, out.ctypes.data),
           "qlinear_unpack_host")
    return out


def qlinear_quantize_rtn_host(w: np.ndarray, bits: int, group: int = 64):
    w = np.ascontiguousarray(w, dtype=np.float32)
    n, k = w.shape
    q = np.empty((n, k), dtype=np.uint8)
    g = k // group if group else 0
    s = np.empty((n, g), dtype=np.uint16)
    b = np.empty((n, g), dtype=np.uint16)
    _check(load_library().qlinear_quantize_rtn_host(w.ctypes.data, bits, group, n, k, q.ctypes.data,
                                                    s.ctypes.data, b.ctypes.data), "qlinear_quantize_rtn_host")
    return q, s, b


def qlinear_status_string(status: int) -> str:
    return load_library().qlinear_status_string(status).decode()


def qlinear_last_path() -> str:
    buf = ctypes.create_string_buffer(160)
    _check(load_library().qlinear_last_path(buf, 160), "qlinear_last_path")
    return buf.value.decode()


def qlinear_version() -> int:
    return int(load_library().qlinear_version())
