"""Python binding of ``libgl.so`` (see ``include/gl.h``).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of the library.  PyTorch supplies device memory and the current
stream.  The entry points keep the C names: :func:`gl_offsets`,
:func:`gl_fwd`, :func:`gl_dgrad`, :func:`gl_wgrad` and
:func:`group_quantize_mxfp8`.  There is no fallback: if the library has not
been built, the first call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence, Union

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgl.so")
_lib = None

GL_OK, GL_ERR_INVALID, GL_ERR_UNSUPPORTED, GL_ERR_CUDA = 0, 1, 2, 3
GL_DEV_NEG_SPLIT, GL_DEV_SUM_MISMATCH, GL_DEV_OUT_OVERFLOW, GL_DEV_TIMEOUT = 1, 2, 4, 8
GL_DEV_BAD_INDEX = 16
GL_STACKED, GL_PER_GROUP = 0, 1
GL_SCALES_ROWMAJOR, GL_SCALES_MMA = 0, 1
(GL_ACT_NONE, GL_ACT_RELU, GL_ACT_RELU2, GL_ACT_GELU, GL_ACT_SILU, GL_ACT_SWIGLU, GL_ACT_GEGLU) = range(7)
ACTS = {"none": GL_ACT_NONE, "relu": GL_ACT_RELU, "relu2": GL_ACT_RELU2, "gelu": GL_ACT_GELU, "silu": GL_ACT_SILU,
        "swiglu": GL_ACT_SWIGLU, "geglu": GL_ACT_GEGLU}
GL_MOE_MAX_TOKENS, GL_MOE_MAX_EXPERTS, GL_MOE_MAX_TOP_K, GL_MOE_RENORM = 128, 256, 16, 1

EXPORTED = ("gl_version", "gl_status_string", "gl_offsets", "gl_fwd", "gl_dgrad", "gl_wgrad",
            "gl_dbias", "group_quantize_mxfp8", "gl_mxfp8_scale_bytes", "gl_dbias_workspace_bytes",
            "group_quantize_mxfp8_dbias", "gl_fwd_mxfp8", "gl_dgrad_mxfp8", "gl_wgrad_mxfp8",
            "gl_fwd_act", "gl_dgrad_act", "gl_rmsnorm", "gl_rmsnorm_bwd", "gl_rmsnorm_bwd_workspace_bytes",
            "gl_moe_tokens", "gl_moe_workspace_bytes")


class GlGrouped(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int), ("base", ctypes.c_void_p),
                ("ptrs", ctypes.POINTER(ctypes.c_void_p))]


GL_TILES_PAIR, GL_TILES_SINGLE, GL_TILES_BY_SIZE = 0, 1, 2


GL_OPT_HOLD_LOADS = 1


class GlGemmOpts(ctypes.Structure):
    _fields_ = [("tiles", ctypes.c_int), ("wait_limit_us", ctypes.c_uint32), ("flags", ctypes.c_uint32)]


class GlError(RuntimeError):
    pass


def lib_path() -> str:
    return _LIB_PATH


def load() -> ctypes.CDLL:
    """Load libgl.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise GlError(f"{_LIB_PATH} is missing: build it with `python -m grouped_gemm_splits_b200.build`")
    L = ctypes.CDLL(_LIB_PATH)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    L.gl_version.restype = i32
    L.gl_status_string.restype = ctypes.c_char_p
    L.gl_status_string.argtypes = [i32]
    L.gl_offsets.restype = i32
    L.gl_offsets.argtypes = [vp, i32, i64, i64, vp, vp, vp]
    L.gl_fwd.restype = i32
    op = ctypes.POINTER(GlGemmOpts)
    L.gl_fwd.argtypes = [vp, GlGrouped, ctypes.POINTER(GlGrouped), vp, vp, i32, i64, i32, i32, vp, i64, op, vp]
    L.gl_dgrad.restype = i32
    L.gl_dgrad.argtypes = [vp, GlGrouped, vp, vp, i32, i64, i32, i32, vp, i64, op, vp]
    L.gl_wgrad.restype = i32
    L.gl_wgrad.argtypes = [vp, vp, vp, vp, i32, i64, i32, i32, GlGrouped, i32, op, vp]
    L.gl_dbias.restype = i32
    L.gl_dbias.argtypes = [vp, vp, vp, i32, i64, i32, GlGrouped, vp]
    L.group_quantize_mxfp8.restype = i32
    L.group_quantize_mxfp8.argtypes = [vp, i64, i32, vp, i32, vp, vp, vp, vp, vp, i32, vp]
    L.gl_mxfp8_scale_bytes.restype = ctypes.c_size_t
    L.gl_mxfp8_scale_bytes.argtypes = [i64, i32, i32, i32, i32]
    L.gl_dbias_workspace_bytes.restype = ctypes.c_size_t
    L.gl_dbias_workspace_bytes.argtypes = [i64, i32, i32]
    L.group_quantize_mxfp8_dbias.restype = i32
    L.group_quantize_mxfp8_dbias.argtypes = [vp, i64, i32, vp, i32, vp, vp, vp, vp, vp, i32, GlGrouped, vp,
                                             ctypes.c_size_t, vp]
    L.gl_fwd_mxfp8.restype = i32
    L.gl_fwd_mxfp8.argtypes = [vp, vp, GlGrouped, GlGrouped, ctypes.POINTER(GlGrouped), vp, vp, i32, i64, i32,
                               i32, vp, i64, op, vp]
    L.gl_dgrad_mxfp8.restype = i32
    L.gl_dgrad_mxfp8.argtypes = [vp, vp, GlGrouped, GlGrouped, vp, vp, i32, i64, i32, i32, vp, i64, op, vp]
    L.gl_wgrad_mxfp8.restype = i32
    L.gl_wgrad_mxfp8.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, GlGrouped, i32, op, vp]
    L.gl_fwd_act.restype = i32
    L.gl_fwd_act.argtypes = [vp, GlGrouped, ctypes.POINTER(GlGrouped), vp, i32, vp, vp, i32, i64, i32, i32, vp, vp, i64,
                             op, vp]
    L.gl_dgrad_act.restype = i32
    L.gl_dgrad_act.argtypes = [vp, GlGrouped, vp, i32, vp, vp, i32, i64, i32, i32, vp, i64, op, vp]
    L.gl_rmsnorm.restype = i32
    L.gl_rmsnorm.argtypes = [vp, vp, vp, ctypes.c_float, i64, i32, vp, vp, vp, vp, vp, i32, vp]
    L.gl_rmsnorm_bwd.restype = i32
    L.gl_rmsnorm_bwd.argtypes = [vp, vp, vp, vp, vp, i64, i32, vp, vp, i32, vp, ctypes.c_size_t, vp]
    L.gl_rmsnorm_bwd_workspace_bytes.restype = ctypes.c_size_t
    L.gl_rmsnorm_bwd_workspace_bytes.argtypes = [i64, i32]
    L.gl_moe_tokens.restype = i32
    L.gl_moe_tokens.argtypes = [vp, vp, GlGrouped, GlGrouped, i32, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp,
                                ctypes.c_size_t, op, vp]
    L.gl_moe_workspace_bytes.restype = ctypes.c_size_t
    L.gl_moe_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    _lib = L
    return L


def _check(st: int, what: str) -> None:
    if st != GL_OK:
        raise GlError(f"{what}: {load().gl_status_string(st).decode()} ({st})")


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


TensorOrList = Union[torch.Tensor, Sequence[torch.Tensor]]


def _grouped(t: TensorOrList, G: int):
    """gl_grouped for a stacked tensor or a list of per-group tensors.

    Returns (struct, keepalive) -- keep the second value alive for the call.
    """
    if isinstance(t, torch.Tensor):
        assert t.is_contiguous() and t.shape[0] == G
        return GlGrouped(GL_STACKED, t.data_ptr(), None), None
    assert len(t) == G
    arr = (ctypes.c_void_p * G)(*[x.data_ptr() for x in t])
    return GlGrouped(GL_PER_GROUP, None, ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p))), arr


def _shape_nk(w: TensorOrList):
    return tuple((w if isinstance(w, torch.Tensor) else w[0]).shape[-2:])


def _opts(pair: bool, wait_limit_us: int, flags: int = 0):
    """Per-call GEMM options (``gl_gemm_opts``); None for the defaults."""
    if pair and not wait_limit_us and not flags:
        return None
    return ctypes.pointer(GlGemmOpts(GL_TILES_PAIR if pair else GL_TILES_SINGLE, wait_limit_us, flags))


def _opts_open(pair: Optional[bool], wait_limit_us: int, flags: int):
    """The same where None for ``pair`` leaves the tile shape to the library."""
    if pair is None and not wait_limit_us and not flags:
        return None
    tiles = GL_TILES_BY_SIZE if pair is None else GL_TILES_PAIR if pair else GL_TILES_SINGLE
    return ctypes.pointer(GlGemmOpts(tiles, wait_limit_us, flags))


def gl_offsets(m_splits: torch.Tensor, expect_rows: int, out_rows: Optional[int] = None,
               offsets: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None):
    """Device prefix scan of ``m_splits`` (int64[G]) -> (offsets int64[G+1], status int32[1])."""
    G = m_splits.numel()
    dev = m_splits.device
    if offsets is None:
        offsets = torch.empty(G + 1, dtype=torch.int64, device=dev)
    if status is None:
        status = torch.empty(1, dtype=torch.int32, device=dev)
    out_rows = expect_rows if out_rows is None else out_rows
    _check(load().gl_offsets(m_splits.data_ptr(), G, expect_rows, out_rows, offsets.data_ptr(),
                             status.data_ptr(), _stream()), "gl_offsets")
    return offsets, status


def gl_fwd(x: torch.Tensor, w: TensorOrList, bias: Optional[TensorOrList], offsets: torch.Tensor,
           status: torch.Tensor, y: Optional[torch.Tensor] = None, pair: bool = True, wait_limit_us: int = 0, opt_flags: int = 0) -> torch.Tensor:
    """y rows of group g = x rows of group g @ W_g^T (+ b_g).  ``y`` may be a
    caller buffer with more rows than x; only the valid rows are written."""
    G = offsets.numel() - 1
    M, K = x.shape
    N, K2 = _shape_nk(w)
    assert K2 == K
    if y is None:
        y = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    wg, keep_w = _grouped(w, G)
    bptr = None
    keep_b = None
    if bias is not None:
        bg, keep_b = _grouped(bias, G)
        bptr = ctypes.pointer(bg)
    _check(load().gl_fwd(x.data_ptr(), wg, bptr, offsets.data_ptr(), status.data_ptr(), G, M, N, K,
                         y.data_ptr(), y.shape[0], _opts(pair, wait_limit_us, opt_flags), _stream()), "gl_fwd")
    del keep_w, keep_b
    return y


def gl_dgrad(dy: torch.Tensor, w: TensorOrList, offsets: torch.Tensor, status: torch.Tensor,
             dx: Optional[torch.Tensor] = None, pair: bool = True, wait_limit_us: int = 0, opt_flags: int = 0) -> torch.Tensor:
    """dx rows of group g = dy rows of group g @ W_g."""
    G = offsets.numel() - 1
    M, N = dy.shape
    N2, K = _shape_nk(w)
    assert N2 == N
    if dx is None:
        dx = torch.empty(M, K, dtype=torch.bfloat16, device=dy.device)
    wg, keep_w = _grouped(w, G)
    _check(load().gl_dgrad(dy.data_ptr(), wg, offsets.data_ptr(), status.data_ptr(), G, M, N, K,
                           dx.data_ptr(), dx.shape[0], _opts(pair, wait_limit_us, opt_flags), _stream()), "gl_dgrad")
    del keep_w
    return dx


def gl_wgrad(x: torch.Tensor, dy: torch.Tensor, offsets: torch.Tensor, status: torch.Tensor,
             main_grad: TensorOrList, accumulate: bool = True, pair: bool = True, wait_limit_us: int = 0, opt_flags: int = 0) -> TensorOrList:
    """main_grad[g] (+)= dy_g^T @ x_g (fp32)."""
    G = offsets.numel() - 1
    M, K = x.shape
    N = dy.shape[1]
    mg, keep = _grouped(main_grad, G)
    _check(load().gl_wgrad(x.data_ptr(), dy.data_ptr(), offsets.data_ptr(), status.data_ptr(), G,
                           M, N, K, mg, 1 if accumulate else 0, _opts(pair, wait_limit_us, opt_flags), _stream()), "gl_wgrad")
    del keep
    return main_grad


def gl_dbias(dy: torch.Tensor, offsets: torch.Tensor, status: torch.Tensor,
             dbias: Optional[TensorOrList] = None) -> TensorOrList:
    """Bias gradient: per group, the column sums of its rows of dy (bf16 out).
    ``dbias`` may be a [G, N] tensor or a list of G [N] tensors."""
    G = offsets.numel() - 1
    M, N = dy.shape
    if dbias is None:
        dbias = torch.empty(G, N, dtype=torch.bfloat16, device=dy.device)
    db, keep = _grouped(dbias, G)
    _check(load().gl_dbias(dy.data_ptr() if M > 0 else None, offsets.data_ptr(), status.data_ptr(), G, M, N, db,
                           _stream()), "gl_dbias")
    del keep
    return dbias


def mxfp8_scale_bytes(rows: int, cols: int, G: int, colwise: bool, mma: bool) -> int:
    """Bytes to allocate for a scale array (``gl_mxfp8_scale_bytes``)."""
    n = load().gl_mxfp8_scale_bytes(rows, cols, G, 1 if colwise else 0, GL_SCALES_MMA if mma else GL_SCALES_ROWMAJOR)
    if n == 0:
        raise GlError(f"gl_mxfp8_scale_bytes: invalid arguments ({rows}, {cols}, {G})")
    return n


def group_quantize_mxfp8(src: torch.Tensor, row_offsets: Optional[torch.Tensor] = None, G: int = 1,
                         rowwise: bool = True, colwise: bool = False,
                         status: Optional[torch.Tensor] = None, out: Optional[dict] = None,
                         mma_scales: bool = False) -> dict:
    """MXFP8 cast of a bf16 [rows, cols] tensor (rows in G groups).

    Returns a dict with ``codes_r``/``scales_r`` (blocks along each row) and/or
    ``codes_c``/``scales_c`` (blocks of 32 rows inside each group).  Scales are
    [rows, cols/32] and [ceil(rows/32) + G, cols] arrays, or with
    ``mma_scales`` flat byte arrays in the tcgen05 scale-factor layout that the
    MXFP8 GEMMs read (``GL_SCALES_MMA``).
    """
    src2, rows, cols, G = _cast_shape(src, row_offsets, G)
    out = _cast_outputs(src2, G, rowwise, colwise, out, mma_scales)
    _check(load().group_quantize_mxfp8(
        src2.data_ptr(), rows, cols, _ptr(row_offsets), G, _ptr(status),
        _ptr(out.get("codes_r")) if rowwise else None, _ptr(out.get("scales_r")) if rowwise else None,
        _ptr(out.get("codes_c")) if colwise else None, _ptr(out.get("scales_c")) if colwise else None,
        GL_SCALES_MMA if mma_scales else GL_SCALES_ROWMAJOR, _stream()), "group_quantize_mxfp8")
    return out


def _cast_shape(src: torch.Tensor, row_offsets: Optional[torch.Tensor], G: int):
    if src.dim() == 3:
        G = src.shape[0]
        src2 = src.reshape(-1, src.shape[-1])
    else:
        src2 = src
    if row_offsets is not None:
        G = row_offsets.numel() - 1
    rows, cols = src2.shape
    return src2, rows, cols, G


def _cast_outputs(src2: torch.Tensor, G: int, rowwise: bool, colwise: bool, out: Optional[dict],
                  mma_scales: bool) -> dict:
    rows, cols = src2.shape
    dev = src2.device
    out = {} if out is None else out

    def need(key, make):
        if key not in out:  # allocate only what the caller did not supply
            out[key] = make()

    if rowwise:
        need("codes_r", lambda: torch.empty(rows, cols, dtype=torch.uint8, device=dev))
        if mma_scales:
            need("scales_r", lambda: torch.empty(mxfp8_scale_bytes(rows, cols, G, False, True), dtype=torch.uint8,
                                                 device=dev))
        else:
            need("scales_r", lambda: torch.empty(rows, cols // 32, dtype=torch.uint8, device=dev))
    if colwise:
        need("codes_c", lambda: torch.empty(rows, cols, dtype=torch.uint8, device=dev))
        if mma_scales:
            need("scales_c", lambda: torch.empty(mxfp8_scale_bytes(rows, cols, G, True, True), dtype=torch.uint8,
                                                 device=dev))
        else:
            need("scales_c", lambda: torch.empty((rows + 31) // 32 + G, cols, dtype=torch.uint8, device=dev))
    return out


def dbias_workspace_bytes(rows: int, cols: int, G: int) -> int:
    """Workspace bytes of :func:`group_quantize_mxfp8_dbias` (``gl_dbias_workspace_bytes``)."""
    n = load().gl_dbias_workspace_bytes(rows, cols, G)
    if n == 0:
        raise GlError(f"gl_dbias_workspace_bytes: invalid arguments ({rows}, {cols}, {G})")
    return n


def group_quantize_mxfp8_dbias(dy: torch.Tensor, row_offsets: torch.Tensor, status: torch.Tensor,
                               rowwise: bool = True, colwise: bool = True, out: Optional[dict] = None,
                               mma_scales: bool = False, dbias: Optional[TensorOrList] = None,
                               workspace: Optional[torch.Tensor] = None):
    """:func:`group_quantize_mxfp8` of a ragged dy that also returns its bias
    gradient (per group, the column sums of its rows; bf16 [G, cols] or a list
    of G [cols] tensors) from the same pass.  ``workspace`` (uint8, at least
    :func:`dbias_workspace_bytes`, 256-byte aligned) is allocated when absent.
    Returns (codes/scales dict, dbias)."""
    src2, rows, cols, G = _cast_shape(dy, row_offsets, 1)
    out = _cast_outputs(src2, G, rowwise, colwise, out, mma_scales)
    if dbias is None:
        dbias = torch.empty(G, cols, dtype=torch.bfloat16, device=dy.device)
    nbytes = dbias_workspace_bytes(rows, cols, G)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dy.device)
    db, keep = _grouped(dbias, G)
    _check(load().group_quantize_mxfp8_dbias(
        src2.data_ptr(), rows, cols, row_offsets.data_ptr(), G, status.data_ptr(),
        _ptr(out.get("codes_r")) if rowwise else None, _ptr(out.get("scales_r")) if rowwise else None,
        _ptr(out.get("codes_c")) if colwise else None, _ptr(out.get("scales_c")) if colwise else None,
        GL_SCALES_MMA if mma_scales else GL_SCALES_ROWMAJOR, db, workspace.data_ptr(), workspace.numel(),
        _stream()), "group_quantize_mxfp8_dbias")
    del keep
    return out, dbias


# ---------------------------------------------------------------- MXFP8 GEMMs

def _grouped_any(t: TensorOrList, G: int):
    """gl_grouped for a stacked tensor (any leading shape) or a list of G tensors."""
    if isinstance(t, torch.Tensor):
        assert t.is_contiguous()
        return GlGrouped(GL_STACKED, t.data_ptr(), None), None
    assert len(t) == G
    arr = (ctypes.c_void_p * G)(*[x.data_ptr() for x in t])
    return GlGrouped(GL_PER_GROUP, None, ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p))), arr


def gl_fwd_mxfp8(x_codes: torch.Tensor, x_scales: torch.Tensor, w_codes: TensorOrList, w_scales: TensorOrList,
                 bias: Optional[TensorOrList], offsets: torch.Tensor, status: torch.Tensor,
                 y: Optional[torch.Tensor] = None, pair: bool = True, wait_limit_us: int = 0, opt_flags: int = 0) -> torch.Tensor:
    """fprop on MXFP8 operands: x rowwise codes [M,K] + scale atoms; W rowwise
    codes [G,N,K] (or G x [N,K]) + scale atoms (all scales ``mma_scales``)."""
    G = offsets.numel() - 1
    M, K = x_codes.shape
    N = (w_codes if isinstance(w_codes, torch.Tensor) else w_codes[0]).shape[-2]
    if y is None:
        y = torch.empty(M, N, dtype=torch.bfloat16, device=x_codes.device)
    wc, k1 = _grouped_any(w_codes, G)
    ws, k2 = _grouped_any(w_scales, G)
    bptr, k3 = None, None
    if bias is not None:
        bg, k3 = _grouped(bias, G)
        bptr = ctypes.pointer(bg)
    _check(load().gl_fwd_mxfp8(x_codes.data_ptr(), x_scales.data_ptr(), wc, ws, bptr, offsets.data_ptr(),
                               status.data_ptr(), G, M, N, K, y.data_ptr(), y.shape[0], _opts(pair, wait_limit_us, opt_flags), _stream()),
           "gl_fwd_mxfp8")
    del k1, k2, k3
    return y


def gl_dgrad_mxfp8(dy_codes: torch.Tensor, dy_scales: torch.Tensor, w_codes_c: TensorOrList,
                   w_scales_c: TensorOrList, offsets: torch.Tensor, status: torch.Tensor,
                   dx: Optional[torch.Tensor] = None, pair: bool = True, wait_limit_us: int = 0, opt_flags: int = 0) -> torch.Tensor:
    """dgrad on MXFP8 operands: dy rowwise codes [M,N] + scale atoms; W
    columnwise codes [G,N,K] + columnwise scale atoms."""
    G = offsets.numel() - 1
    M, N = dy_codes.shape
    K = (w_codes_c if isinstance(w_codes_c, torch.Tensor) else w_codes_c[0]).shape[-1]
    if dx is None:
        dx = torch.empty(M, K, dtype=torch.bfloat16, device=dy_codes.device)
    wc, k1 = _grouped_any(w_codes_c, G)
    ws, k2 = _grouped_any(w_scales_c, G)
    _check(load().gl_dgrad_mxfp8(dy_codes.data_ptr(), dy_scales.data_ptr(), wc, ws, offsets.data_ptr(),
                                 status.data_ptr(), G, M, N, K, dx.data_ptr(), dx.shape[0], _opts(pair, wait_limit_us, opt_flags), _stream()),
           "gl_dgrad_mxfp8")
    del k1, k2
    return dx


def gl_wgrad_mxfp8(x_codes_c: torch.Tensor, x_scales_c: torch.Tensor, dy_codes_c: torch.Tensor,
                   dy_scales_c: torch.Tensor, offsets: torch.Tensor, status: torch.Tensor,
                   main_grad: TensorOrList, accumulate: bool = True, pair: bool = True, wait_limit_us: int = 0, opt_flags: int = 0) -> TensorOrList:
    """wgrad on MXFP8 operands: x and dy columnwise codes + columnwise scale atoms."""
    G = offsets.numel() - 1
    M, K = x_codes_c.shape
    N = dy_codes_c.shape[1]
    mg, keep = _grouped(main_grad, G)
    _check(load().gl_wgrad_mxfp8(x_codes_c.data_ptr(), x_scales_c.data_ptr(), dy_codes_c.data_ptr(),
                                 dy_scales_c.data_ptr(), offsets.data_ptr(), status.data_ptr(), G, M, N, K, mg,
                                 1 if accumulate else 0, _opts(pair, wait_limit_us, opt_flags), _stream()), "gl_wgrad_mxfp8")
    del keep
    return main_grad


# ------------------------------------------------------------------- RMS norm

def _refuse(what: str, why: str) -> None:
    raise GlError(f"{what}: {why}")


def _tensor(what: str, name: str, t, dtype, shape) -> None:
    """Refuse anything but a contiguous tensor of this dtype and shape."""
    if isinstance(t, torch.Tensor):
        if t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return
        if t.dtype is not dtype:
            _refuse(what, f"{name} must be {dtype}, not {t.dtype}")
        if t.shape != shape:
            _refuse(what, f"{name} must be {tuple(shape)}, not {tuple(t.shape)}")
        _refuse(what, f"{name} must be contiguous")
    _refuse(what, f"{name} must be a tensor")


def _matrix(what: str, name: str, t) -> torch.Size:
    """The shape of a contiguous bf16 [rows, cols] tensor."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        _refuse(what, f"{name} must be a matrix")
    shape = t.shape
    _tensor(what, name, t, torch.bfloat16, shape)
    return shape


def _status_word(what: str, t) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.numel() != 1:
        _refuse(what, "status must be one int32")


def _device(what: str, first: torch.Tensor, *others) -> int:
    """The CUDA device that all of a call's tensors are on."""
    dev = first.get_device()
    for t in others:
        if t is not None:
            if not isinstance(t, torch.Tensor):
                _refuse(what, f"{t!r} is not a tensor")
            if t.get_device() != dev:
                _refuse(what, f"tensors on {first.device} and {t.device}")
    if dev < 0:
        _refuse(what, f"tensors must be on a CUDA device, not {first.device}")
    return dev


def _scratch(what: str, t) -> None:
    """Refuse a workspace whose elements are not all there in a row."""
    if not isinstance(t, torch.Tensor) or not t.is_contiguous():
        _refuse(what, "workspace must be a contiguous tensor")


# the current device, and the handle of a device's current stream (what
# torch.cuda.current_stream() wraps in an object; absent from a torch without CUDA)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def gl_rmsnorm(x: torch.Tensor, gamma: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
               y: bool = True, mxfp8: bool = False, mma_scales: bool = False, out: Optional[dict] = None) -> dict:
    """RMS norm of ``x`` (+ ``residual``), bf16 [rows, cols].

    Returns a dict: ``rstd`` (fp32 [rows]); ``sum`` (bf16, the new residual
    stream) where there is a residual; ``y`` (bf16) if asked for; with
    ``mxfp8`` the rowwise ``codes_r`` / ``scales_r`` of the fp32 result, as
    :func:`group_quantize_mxfp8` lays them out (``mma_scales``: the layout the
    MXFP8 products read).  Tensors given in ``out`` are written instead of new
    ones; ``out["sum"]`` and ``out["y"]`` may be ``x`` or ``residual``.
    """
    what = "gl_rmsnorm"
    bf = torch.bfloat16
    shape = _matrix(what, "x", x)
    rows, cols = shape
    _tensor(what, "gamma", gamma, bf, (cols,))
    if residual is not None:
        _tensor(what, "residual", residual, bf, shape)
    if not (y or mxfp8):
        _refuse(what, "at least one of y and mxfp8 is required")
    if mxfp8 and cols % (128 if mma_scales else 32):
        _refuse(what, f"cols = {cols} does not fit the scale layout")
    out = {} if out is None else dict(out)
    dev = _device(what, x, gamma, residual, *out.values())
    if dev != _current_device():
        with torch.cuda.device(dev):
            return gl_rmsnorm(x, gamma, eps, residual, y, mxfp8, mma_scales, out)
    rstd = out.get("rstd")
    if rstd is None:
        rstd = out["rstd"] = torch.empty(rows, dtype=torch.float32, device=x.device)
    else:
        _tensor(what, "rstd", rstd, torch.float32, (rows,))
    s = out.get("sum")
    if s is not None:
        _tensor(what, "sum", s, bf, shape)
    elif residual is not None:
        s = out["sum"] = torch.empty_like(x)
    yt = out.get("y")
    if yt is not None:
        _tensor(what, "y", yt, bf, shape)
    elif y:
        yt = out["y"] = torch.empty_like(x)
    codes, scales = out.get("codes_r"), out.get("scales_r")
    if mxfp8:
        if codes is None:
            codes = out["codes_r"] = torch.empty_like(x, dtype=torch.uint8)
        else:
            _tensor(what, "codes_r", codes, torch.uint8, shape)
        size = ((rows + 127) // 128 * (cols // 128) * 512,) if mma_scales else (rows, cols // 32)
        if scales is None:
            scales = out["scales_r"] = torch.empty(size, dtype=torch.uint8, device=x.device)
        elif mma_scales:
            _tensor(what, "scales_r", scales, torch.uint8, size)
        else:  # [rows, cols / 32], or the same bytes in a row
            _tensor(what, "scales_r", scales, torch.uint8, size if scales.dim() == 2 else (rows * (cols // 32),))
    known = 1 + (s is not None) + y + 2 * mxfp8
    if len(out) != known:
        _refuse(what, f"out has {sorted(out)}: more than this call's outputs")
    _check(load().gl_rmsnorm(x.data_ptr(), _ptr(residual), gamma.data_ptr(), eps, rows, cols, _ptr(s), _ptr(yt),
                             rstd.data_ptr(), _ptr(codes), _ptr(scales),
                             GL_SCALES_MMA if mma_scales else GL_SCALES_ROWMAJOR, _current_stream(dev)), what)
    return out


def rmsnorm_bwd_workspace_bytes(rows: int, cols: int) -> int:
    """Workspace bytes of :func:`gl_rmsnorm_bwd` on the current device."""
    n = load().gl_rmsnorm_bwd_workspace_bytes(rows, cols)
    if n == 0:
        raise GlError(f"gl_rmsnorm_bwd_workspace_bytes: invalid arguments ({rows}, {cols})")
    return n


def gl_rmsnorm_bwd(dy: torch.Tensor, sum: torch.Tensor, gamma: torch.Tensor, rstd: torch.Tensor,
                   dsum: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                   dgamma: Optional[torch.Tensor] = None, accumulate: bool = False,
                   workspace: Optional[torch.Tensor] = None):
    """Gradients of :func:`gl_rmsnorm`: (dx bf16 [rows, cols], dgamma fp32 [cols]).

    ``dx`` is the gradient of x and of the residual alike; ``dsum`` is what
    reaches the sum along the residual stream.  ``accumulate`` adds to the
    given ``dgamma``.
    """
    what = "gl_rmsnorm_bwd"
    bf = torch.bfloat16
    rows, cols = _matrix(what, "dy", dy)
    _tensor(what, "sum", sum, bf, (rows, cols))
    _tensor(what, "gamma", gamma, bf, (cols,))
    _tensor(what, "rstd", rstd, torch.float32, (rows,))
    if dsum is not None:
        _tensor(what, "dsum", dsum, bf, (rows, cols))
    if dx is not None:
        _tensor(what, "dx", dx, bf, (rows, cols))
    if dgamma is not None:
        _tensor(what, "dgamma", dgamma, torch.float32, (cols,))
    if accumulate and dgamma is None:
        _refuse(what, "accumulate needs a dgamma")
    if workspace is not None:
        _scratch(what, workspace)
    dev = _device(what, dy, sum, gamma, rstd, dsum, dx, dgamma, workspace)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return gl_rmsnorm_bwd(dy, sum, gamma, rstd, dsum, dx, dgamma, accumulate, workspace)
    if dx is None:
        dx = torch.empty_like(dy)
    if dgamma is None:
        dgamma = torch.empty(cols, dtype=torch.float32, device=dy.device)
    if workspace is None:
        workspace = torch.empty(rmsnorm_bwd_workspace_bytes(rows, cols), dtype=torch.uint8, device=dy.device)
    _check(load().gl_rmsnorm_bwd(dy.data_ptr(), sum.data_ptr(), gamma.data_ptr(), rstd.data_ptr(), _ptr(dsum),
                                 rows, cols, dx.data_ptr(), dgamma.data_ptr(), 1 if accumulate else 0,
                                 workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                 _current_stream(dev)), what)
    return dx, dgamma


# ------------------------------------- products with an activation in the epilogue

def _gated(act: int) -> bool:
    return act in (GL_ACT_SWIGLU, GL_ACT_GEGLU)


def _weight_dims(what: str, name: str, w: TensorOrList):
    """Rows and columns of a group's weight."""
    t = w if isinstance(w, torch.Tensor) else w[0] if len(w) else None
    if not isinstance(t, torch.Tensor) or t.dim() < 2:
        _refuse(what, f"{name} must be a [groups, rows, cols] tensor or a list of matrices")
    return t.shape[-2], t.shape[-1]


def _weights(what: str, name: str, w: TensorOrList, G: int, shape) -> torch.Tensor:
    """Check a stacked tensor or a list of G tensors of the given per-group shape; returns one of them."""
    if isinstance(w, torch.Tensor):
        _tensor(what, name, w, torch.bfloat16, (G, *shape))
        return w
    if len(w) != G:
        _refuse(what, f"{name} must have {G} tensors, not {len(w)}")
    for t in w:
        _tensor(what, name, t, torch.bfloat16, shape)
        if t.device != w[0].device:
            _refuse(what, f"{name} on {w[0].device} and {t.device}")
    return w[0]


def _plan(what: str, offsets: torch.Tensor, status: torch.Tensor) -> int:
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() < 2:
        _refuse(what, "offsets must be the [G + 1] tensor of gl_offsets")
    _tensor(what, "offsets", offsets, torch.int64, offsets.shape)
    _status_word(what, status)
    return offsets.numel() - 1


def _rows_at_least(what: str, name: str, t: torch.Tensor, rows: int, cols: int) -> None:
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.shape[0] < rows:
        _refuse(what, f"{name} must have at least {rows} rows")
    _tensor(what, name, t, torch.bfloat16, (t.shape[0], cols))


def gl_fwd_act(x: torch.Tensor, w: TensorOrList, bias: Optional[TensorOrList], offsets: torch.Tensor,
               status: torch.Tensor, act: int, residual: Optional[torch.Tensor] = None, save_z: bool = False,
               z: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, pair: Optional[bool] = None,
               wait_limit_us: int = 0, opt_flags: int = 0):
    """:func:`gl_fwd` with an activation (``GL_ACT_*``) and a residual in its
    epilogue: y = act(x W^T + b) + residual, or, gated, act(u0) * u1 + residual
    on the halves of u = x W^T + b.  Returns (y, z): z is u (bf16 [M, N]), what
    :func:`gl_dgrad_act` reads, if ``save_z`` is set or a ``z`` is given, else
    None.  ``y`` may have more rows than x; only the valid ones are written.
    ``pair`` picks the tile shape (None: by size).
    """
    what = "gl_fwd_act"
    G = _plan(what, offsets, status)
    M, K = _matrix(what, "x", x)
    if not GL_ACT_NONE <= act <= GL_ACT_GEGLU:
        _refuse(what, f"unknown activation {act}")
    N = _weight_dims(what, "w", w)[0]
    if _gated(act) and N % 2:
        _refuse(what, f"a gated activation halves {N} columns")
    w0 = _weights(what, "w", w, G, (N, K))
    b0 = _weights(what, "bias", bias, G, (N,)) if bias is not None else None
    Nout = N // 2 if _gated(act) else N
    if residual is not None:
        _tensor(what, "residual", residual, torch.bfloat16, (M, Nout))
    if z is not None:
        _tensor(what, "z", z, torch.bfloat16, (M, N))
    if y is not None:
        _rows_at_least(what, "y", y, M, Nout)
    dev = _device(what, x, w0, b0, residual, offsets, status, z, y)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return gl_fwd_act(x, w, bias, offsets, status, act, residual, save_z, z, y, pair, wait_limit_us, opt_flags)
    if y is None:
        y = torch.empty(M, Nout, dtype=torch.bfloat16, device=x.device)
    if z is None and save_z:
        z = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    wg, keep_w = _grouped(w, G)
    bptr, keep_b = None, None
    if bias is not None:
        bg, keep_b = _grouped(bias, G)
        bptr = ctypes.byref(bg)
    _check(load().gl_fwd_act(x.data_ptr(), wg, bptr, _ptr(residual), act, offsets.data_ptr(), status.data_ptr(),
                             G, M, N, K, _ptr(z), y.data_ptr(), y.shape[0], _opts_open(pair, wait_limit_us, opt_flags),
                             _current_stream(dev)), what)
    del keep_w, keep_b
    return y, z


def gl_dgrad_act(dy: torch.Tensor, w: TensorOrList, z: torch.Tensor, offsets: torch.Tensor, status: torch.Tensor,
                 act: int, dz: Optional[torch.Tensor] = None, pair: Optional[bool] = None, wait_limit_us: int = 0,
                 opt_flags: int = 0) -> torch.Tensor:
    """:func:`gl_dgrad` that goes on through the activation in front of the
    product: dz = (dy W) * act'(z), with z from the :func:`gl_fwd_act` before
    ([M, K], or [M, 2K] for a gated activation, whose dz has both factors'
    gradients)."""
    what = "gl_dgrad_act"
    G = _plan(what, offsets, status)
    M, N = _matrix(what, "dy", dy)
    if not GL_ACT_NONE < act <= GL_ACT_GEGLU:
        _refuse(what, f"activation {act} has no slope to apply")
    K = _weight_dims(what, "w", w)[1]
    w0 = _weights(what, "w", w, G, (N, K))
    width = 2 * K if _gated(act) else K
    _tensor(what, "z", z, torch.bfloat16, (M, width))
    if dz is not None:
        _rows_at_least(what, "dz", dz, M, width)
    dev = _device(what, dy, w0, z, offsets, status, dz)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return gl_dgrad_act(dy, w, z, offsets, status, act, dz, pair, wait_limit_us, opt_flags)
    if dz is None:
        dz = torch.empty(M, width, dtype=torch.bfloat16, device=dy.device)
    wg, keep = _grouped(w, G)
    _check(load().gl_dgrad_act(dy.data_ptr(), wg, z.data_ptr(), act, offsets.data_ptr(), status.data_ptr(), G, M,
                               N, K, dz.data_ptr(), dz.shape[0], _opts_open(pair, wait_limit_us, opt_flags), _current_stream(dev)),
           what)
    del keep
    return dz


# -------------------------------------------- a mixture-of-experts layer for a few tokens

def moe_workspace_bytes(T: int, E: int, top_k: int, H: int, F: int) -> int:
    """Workspace bytes of :func:`gl_moe_tokens` on the current device."""
    n = load().gl_moe_workspace_bytes(T, E, top_k, H, F)
    if n == 0:
        raise GlError(f"gl_moe_workspace_bytes: outside the layer's limits ({T}, {E}, {top_k}, {H}, {F})")
    return n


def gl_moe_tokens(x: torch.Tensor, w1: TensorOrList, w2: TensorOrList, top_k: int, status: torch.Tensor,
                  router_w: Optional[torch.Tensor] = None, topk_idx: Optional[torch.Tensor] = None,
                  topk_w: Optional[torch.Tensor] = None, act: int = GL_ACT_SWIGLU, renorm: bool = True,
                  y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  wait_limit_us: int = 0, opt_flags: int = 0):
    """A mixture-of-experts layer for up to 128 tokens: y = sum over each
    token's experts of w * ((act(x W1a^T) * (x W1b^T)) W2^T), W1 = [W1a; W1b].

    With ``router_w`` ([E, H]) the experts are the ``top_k`` largest of
    softmax(x router_w^T), their weights divided by their sum if ``renorm``;
    without it ``topk_idx`` (int32 [T, top_k], -1: none) and ``topk_w`` (fp32)
    are the routing.  ``workspace`` (uint8, at least
    :func:`moe_workspace_bytes`) is allocated when absent; calls that overlap
    need one each.  Returns (y, topk_idx, topk_w).
    """
    what = "gl_moe_tokens"
    bf = torch.bfloat16
    T, H = _matrix(what, "x", x)
    _status_word(what, status)
    _weight_dims(what, "w1", w1)
    E, F = len(w1), _weight_dims(what, "w2", w2)[1]
    a = _weights(what, "w1", w1, E, (2 * F, H))
    b = _weights(what, "w2", w2, E, (H, F))
    if T > GL_MOE_MAX_TOKENS:
        _refuse(what, f"{T} tokens: at most {GL_MOE_MAX_TOKENS}")
    if router_w is not None:
        _tensor(what, "router_w", router_w, bf, (E, H))
    elif topk_idx is None or topk_w is None:
        _refuse(what, "router_w, or topk_idx and topk_w, are required")
    if topk_idx is not None:
        _tensor(what, "topk_idx", topk_idx, torch.int32, (T, top_k))
    if topk_w is not None:
        _tensor(what, "topk_w", topk_w, torch.float32, (T, top_k))
    if y is not None:
        _tensor(what, "y", y, bf, (T, H))
    if workspace is not None:
        _scratch(what, workspace)
    dev = _device(what, x, a, b, router_w, status, topk_idx, topk_w, y, workspace)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return gl_moe_tokens(x, w1, w2, top_k, status, router_w, topk_idx, topk_w, act, renorm, y, workspace,
                                 wait_limit_us, opt_flags)
    if topk_idx is None:
        topk_idx = torch.empty(T, top_k, dtype=torch.int32, device=x.device)
    if topk_w is None:
        topk_w = torch.empty(T, top_k, dtype=torch.float32, device=x.device)
    if y is None:
        y = torch.empty_like(x)
    if workspace is None:
        workspace = torch.empty(moe_workspace_bytes(T, E, top_k, H, F), dtype=torch.uint8, device=x.device)
    g1, keep1 = _grouped(w1, E)
    g2, keep2 = _grouped(w2, E)
    _check(load().gl_moe_tokens(x.data_ptr(), _ptr(router_w), g1, g2, act, GL_MOE_RENORM if renorm else 0, T, E,
                                top_k, H, F, topk_idx.data_ptr(), topk_w.data_ptr(), y.data_ptr(),
                                status.data_ptr(), workspace.data_ptr(),
                                workspace.numel() * workspace.element_size(), _opts(True, wait_limit_us, opt_flags),
                                _current_stream(dev)), what)
    del keep1, keep2
    return y, topk_idx, topk_w
