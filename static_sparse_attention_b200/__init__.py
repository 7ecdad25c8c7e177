"""Python binding of libradattn.so (the C ABI in include/radattn.h).

Argument marshalling only: every step of the computation runs in the library's
CUDA kernels.  The C entry points are exposed under their own names
(ra_build_mask, ra_attention_fwd, ...) taking plain integers / pointers, plus a
thin torch-facing layer (Mask, build_mask, attention_fwd, attention_fwd_host, ...)
that passes tensor addresses and the current CUDA stream.  The operators whose
calls last microseconds (norm and rotation, the 8-bit ring) have that layer in a
CPython extension, _torch_binding.so.

There is no CPU fallback: importing this package fails loudly when the
compiled library is missing (build it with
`python static_sparse_attention_b200/build.py`), and so does the first call of an
operator whose extension is; the C entry points need neither it nor torch.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
from typing import NamedTuple

_PKG = os.path.dirname(os.path.abspath(__file__))
# RA_LIBRARY_VARIANT=debug selects the build with device-side bounds checks
# (libradattn_debug.so, `build.py --debug`); the default is the release build.
VARIANT = os.environ.get("RA_LIBRARY_VARIANT", "release")
if VARIANT not in ("release", "debug"):
    raise ImportError(f"RA_LIBRARY_VARIANT must be 'release' or 'debug', not {VARIANT!r}")
LIB_PATH = os.path.join(_PKG, "libradattn_debug.so" if VARIANT == "debug" else "libradattn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{os.path.basename(LIB_PATH)} is not built ({LIB_PATH}); run "
                      f"`python static_sparse_attention_b200/build.py{' --debug' if VARIANT == 'debug' else ''}`")

_lib = ctypes.CDLL(LIB_PATH)

# ------------------------------------------------------------------ constants
RA_MASK_DENSE, RA_MASK_RADIAL, RA_MASK_WINDOW3D, RA_MASK_SWC = 0, 1, 2, 3
RA_MODE_TOKEN_EXACT, RA_MODE_BLOCK = 0, 1
RA_TILE_PARTIAL, RA_TILE_FULL = 0, 1
(RA_OK, RA_ERR_INVALID_ARG, RA_ERR_UNSUPPORTED, RA_ERR_CUDA, RA_ERR_OUT_OF_MEMORY, RA_ERR_DEVICE_TIMEOUT,
 RA_ERR_DEVICE_BOUNDS) = range(7)
RA_TILE = 128
RA_PV_AUTO, RA_PV_BF16, RA_PV_SPLIT = 0, 1, 2
RA_CACHE8_ROWS, RA_CACHE8_ROWS_AHEAD, RA_CACHE8_ONE_TILE, RA_CACHE8_TWO_TILES = range(4)
FAMILIES = {"dense": RA_MASK_DENSE, "radial": RA_MASK_RADIAL, "window3d": RA_MASK_WINDOW3D, "swc": RA_MASK_SWC}
MODES = {"token_exact": RA_MODE_TOKEN_EXACT, "block": RA_MODE_BLOCK}


class ra_mask_params(ctypes.Structure):
    _fields_ = [("grid_h", ctypes.c_int), ("grid_w", ctypes.c_int), ("r_t", ctypes.c_int), ("r_s", ctypes.c_int),
                ("window_frames", ctypes.c_int), ("sink_tokens", ctypes.c_int)]


class ra_mask_info_t(ctypes.Structure):
    _fields_ = [("family", ctypes.c_int), ("f", ctypes.c_int), ("s", ctypes.c_int), ("nb", ctypes.c_int),
                ("n", ctypes.c_longlong), ("nnz", ctypes.c_longlong), ("full_tiles", ctypes.c_longlong),
                ("kept_pairs", ctypes.c_longlong), ("block_pairs", ctypes.c_longlong),
                ("row_min", ctypes.c_int), ("row_max", ctypes.c_int)]


class ra_rope(ctypes.Structure):
    _fields_ = [("t", ctypes.c_void_p), ("h", ctypes.c_void_p), ("w", ctypes.c_void_p),
                ("frames", ctypes.c_int), ("grid_h", ctypes.c_int), ("grid_w", ctypes.c_int),
                ("t_pairs", ctypes.c_int), ("h_pairs", ctypes.c_int), ("w_pairs", ctypes.c_int)]


class ra_head_rows(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("stride_b", ctypes.c_longlong), ("stride_n", ctypes.c_longlong),
                ("stride_h", ctypes.c_longlong), ("heads", ctypes.c_int), ("weight_fp32", ctypes.c_int),
                ("weight", ctypes.c_void_p)]


class ra_head_grads(ctypes.Structure):
    _fields_ = [("dy", ctypes.c_void_p), ("dx", ctypes.c_void_p), ("stride_b", ctypes.c_longlong),
                ("stride_n", ctypes.c_longlong), ("stride_h", ctypes.c_longlong), ("dweight", ctypes.c_void_p)]


_vp, _i, _ll, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
_MaskP = ctypes.c_void_p
_SIGS = {
    "ra_build_mask": ([_i, _i, _i, ctypes.POINTER(ra_mask_params), _vp, ctypes.POINTER(_MaskP)], _i),
    "ra_mask_info": ([_MaskP, ctypes.POINTER(ra_mask_info_t)], _i),
    "ra_build_mask_noalloc": ([_i, _i, _i, ctypes.POINTER(ra_mask_params), _vp, _vp, _vp, _vp, _ll,
                               ctypes.POINTER(ra_mask_info_t), _vp], _i),
    "ra_mask_copy_to_host": ([_MaskP, _vp, _vp, _vp, _vp], _i),
    "ra_mask_device_arrays": ([_MaskP, ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                               ctypes.POINTER(_vp)], _i),
    "ra_mask_free": ([_MaskP], None),
    "ra_mask_copy_transpose_to_host": ([_MaskP, _vp, _vp, _vp], _i),
    "ra_attention_fwd": ([_vp, _vp, _vp, _vp, _i, _i, _i, _MaskP, _f, _i, _vp, _vp], _i),
    "ra_attention_fwd_host": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _MaskP, _f, _i, _vp], _i),
    "ra_attention_bwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _MaskP, _f, _i, _vp], _i),
    "ra_swc_cache_create": ([_i, _i, _i, _i, _i, ctypes.POINTER(_vp)], _i),
    "ra_swc_cache_step": ([_vp, _vp, _vp, _vp, _vp, _f, _vp, _vp], _i),
    "ra_swc_cache_info": ([_vp, ctypes.POINTER(_ll), ctypes.POINTER(_i)], _i),
    "ra_swc_cache_copy_rings_to_host": ([_vp, _vp, _vp], _i),
    "ra_swc_cache_reset": ([_vp], _i),
    "ra_swc_cache_free": ([_vp], None),
    "ra_rope_table": ([_vp, _i, _i, _i, ctypes.c_double, _vp], _i),
    "ra_qk_norm_rope": ([_vp, _vp, _vp, _vp, _i, _i, _i, _vp, _i, _f, _vp], _i),
    "ra_qk_norm_rope_bwd_workspace_bytes": ([_i], ctypes.c_size_t),
    "ra_qk_norm_rope_bwd": ([_vp, _vp, _vp, _vp, _i, _i, _i, _vp, _i, _f, _vp, ctypes.c_size_t, _vp], _i),
    "ra_cache8_append": ([_vp, _vp, _i, _i, _i, _i, _i, _ll, _vp, _f, _vp, _vp, _vp, _vp, _vp], _i),
    "ra_cache8_attention_workspace_bytes": ([_i, _i, _i, _i, _i, _i, _i, ctypes.POINTER(ctypes.c_size_t)], _i),
    "ra_cache8_attention": ([_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _f, _vp, _vp,
                             ctypes.c_size_t, _vp], _i),
    "ra_cache8_attention_plan": ([_i, _i, _i, _i, _i, _i, _i, ctypes.POINTER(_i), ctypes.POINTER(_i)], _i),
    "ra_cache8_attention_check": ([_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _f, _vp, _vp,
                                   ctypes.c_size_t], _i),
    "ra_get_device_status": ([_vp], _i),
    "ra_get_device_error_site": ([ctypes.POINTER(_i), ctypes.POINTER(_i)], _i),
    "ra_selftest_wait_timeout": ([_ll, _vp], _i),
    "ra_selftest_bounds": ([_vp], _i),
    "ra_set_wait_timeout_ns": ([_ll], _i),
    "ra_set_pv_precision": ([_i], _i),
    "ra_status_string": ([_i], ctypes.c_char_p),
    "ra_last_error": ([], ctypes.c_char_p),
    "ra_version": ([], _i),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res
    globals()[_name] = _fn


class RaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = (ra_last_error() or b"").decode(errors="replace")
        super().__init__(f"{where}: {ra_status_string(status).decode()} ({status}): {detail}")


def check(status: int, where: str) -> None:
    if status != RA_OK:
        raise RaError(status, where)


def _stream_handle(stream) -> int | None:
    import torch
    if stream is None:  # the current stream's handle, without making a Stream object for it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_NO_CONTEXT = contextlib.nullcontext()


def _allocating_on(stream, handle: int):
    """Torch work inside is on `stream` (the current one when None): memory that a
    call allocates and drops again is reused only behind the call's own work."""
    if stream is None:
        return _NO_CONTEXT
    import torch
    if handle == torch.cuda.current_stream().cuda_stream:
        return _NO_CONTEXT
    return torch.cuda.stream(torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream())


def _refuse_capture(stream) -> None:
    import torch
    with _allocating_on(stream, 0 if stream is None else _stream_handle(stream)):
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the cache's frame number is host state: a captured step would repeat it")


# ------------------------------------------------------------------- masks
class Mask:
    """A block-CSR mask built on the current CUDA device (owns the C handle)."""

    def __init__(self, family, f: int, s: int, grid_h: int = 0, grid_w: int = 0, r_t: int = 0, r_s: int = 0,
                 window_frames: int = 0, sink_tokens: int = 0, stream=None):
        fam = FAMILIES[family] if isinstance(family, str) else int(family)
        params = ra_mask_params(grid_h, grid_w, r_t, r_s, window_frames, sink_tokens)
        handle = _MaskP()
        check(ra_build_mask(fam, f, s, ctypes.byref(params), _stream_handle(stream), ctypes.byref(handle)),
              "ra_build_mask")
        self._h = handle
        info = ra_mask_info_t()
        check(ra_mask_info(self._h, ctypes.byref(info)), "ra_mask_info")
        self.info = {k: getattr(info, k) for k, _ in ra_mask_info_t._fields_}

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("mask has been freed")
        return self._h

    @property
    def n(self) -> int:
        return self.info["n"]

    def to_host(self) -> dict:
        import numpy as np
        nb, nnz = self.info["nb"], self.info["nnz"]
        row_ptr = np.empty(nb + 1, dtype=np.int32)
        col_idx = np.empty(nnz, dtype=np.int32)
        count = np.empty(nnz, dtype=np.int32)
        flag = np.empty(nnz, dtype=np.uint8)
        check(ra_mask_copy_to_host(self.handle, row_ptr.ctypes.data, col_idx.ctypes.data, count.ctypes.data,
                                   flag.ctypes.data), "ra_mask_copy_to_host")
        return dict(row_ptr=row_ptr, col_idx=col_idx, count=count, flag=flag, nnz=nnz)

    def transpose_to_host(self) -> dict:
        """The transposed block-CSR: col_ptr, row_idx, tflag."""
        import numpy as np
        nb, nnz = self.info["nb"], self.info["nnz"]
        col_ptr = np.empty(nb + 1, dtype=np.int32)
        row_idx = np.empty(nnz, dtype=np.int32)
        tflag = np.empty(nnz, dtype=np.uint8)
        check(ra_mask_copy_transpose_to_host(self.handle, col_ptr.ctypes.data, row_idx.ctypes.data,
                                             tflag.ctypes.data), "ra_mask_copy_transpose_to_host")
        return dict(col_ptr=col_ptr, row_idx=row_idx, tflag=tflag)

    def free(self) -> None:
        if getattr(self, "_h", None) is not None:
            ra_mask_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def build_mask(mask: dict, f: int, s: int, grid=(0, 0), stream=None) -> Mask:
    """Mask from a dict {family, r_t, r_s, window_frames, sink_tokens} (grid used by window3d)."""
    return Mask(mask["family"], f, s, grid[0], grid[1], mask.get("r_t", 0), mask.get("r_s", 0),
                mask.get("window_frames", 0), mask.get("sink_tokens", 0), stream=stream)


# --------------------------------------------------------------- attention
def _check_bf16_cuda(name, t):
    import torch
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")


def attention_fwd(q, k, v, mask: Mask, scale: float | None = None, mode="block", out=None, lse=None, stream=None):
    """O = softmax(scale * q k^T + M) v over the mask's kept tiles; q, k, v bf16 [B, H, n, d]."""
    import torch
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_bf16_cuda(name, t)
    B, H, n, d = q.shape
    if k.shape != q.shape or v.shape != q.shape or n != mask.n:
        raise ValueError("q, k, v must share shape [B, H, n, d] with n equal to the mask's n")
    if out is None:
        out = torch.empty_like(q)
    _check_bf16_cuda("out", out)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, n) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous fp32 tensor [B, H, n]")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    mode = MODES[mode] if isinstance(mode, str) else int(mode)
    check(ra_attention_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, d, mask.handle, scale,
                           mode, None if lse is None else lse.data_ptr(), _stream_handle(stream)),
          "ra_attention_fwd")
    return out


def attention_fwd_host(q_host, k_host, v_host, o_host, q_dev, k_dev, v_dev, o_dev, mask: Mask,
                       scale: float | None = None, mode="block", stream=None):
    """Same call with host inputs / output: enqueues H2D copies, the kernel and the D2H copy."""
    B, H, n, d = q_host.shape
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    mode = MODES[mode] if isinstance(mode, str) else int(mode)
    check(ra_attention_fwd_host(q_host.data_ptr(), k_host.data_ptr(), v_host.data_ptr(), o_host.data_ptr(),
                                q_dev.data_ptr(), k_dev.data_ptr(), v_dev.data_ptr(), o_dev.data_ptr(), B, H, d,
                                mask.handle, scale, mode, _stream_handle(stream)), "ra_attention_fwd_host")
    return o_host


def attention_bwd(q, k, v, out, dout, lse, mask: Mask, scale: float | None = None, mode="block",
                  dq=None, dk=None, dv=None, workspace=None, stream=None):
    """dQ, dK, dV of attention_fwd given its output `out`, its fp32 `lse` and the
    output gradient `dout` (all bf16 [B, H, n, d] except lse [B, H, n])."""
    import torch
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out), ("dout", dout)):
        _check_bf16_cuda(name, t)
    B, H, n, d = q.shape
    if any(t.shape != q.shape for t in (k, v, out, dout)) or n != mask.n:
        raise ValueError("q, k, v, out, dout must share shape [B, H, n, d] with n equal to the mask's n")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, n) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 tensor [B, H, n]")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _check_bf16_cuda(name, t)
        if t.shape != q.shape:
            raise ValueError(f"{name} must have shape [B, H, n, d]")
    if workspace is None:
        workspace = torch.empty((B, H, n), dtype=torch.float32, device=q.device)
    if workspace.dtype != torch.float32 or workspace.numel() < B * H * n or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous fp32 tensor of at least B * H * n elements")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    mode = MODES[mode] if isinstance(mode, str) else int(mode)
    check(ra_attention_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), dout.data_ptr(),
                           lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(),
                           B, H, d, mask.handle, scale, mode, _stream_handle(stream)), "ra_attention_bwd")
    return dq, dk, dv


class SwcCache:
    """Streaming sliding-window causal attention with a key/value ring cache of
    `window_frames` frames of `s` tokens for B x H heads of d channels."""

    def __init__(self, B: int, H: int, d: int, s: int, window_frames: int):
        h = ctypes.c_void_p()
        check(ra_swc_cache_create(B, H, d, s, window_frames, ctypes.byref(h)), "ra_swc_cache_create")
        self._h = h
        self.B, self.H, self.d, self.s, self.W = B, H, d, s, window_frames

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("cache was freed")
        return self._h

    def step(self, q, k, v, out=None, lse=None, scale: float | None = None, stream=None):
        """Feed the next frame (q, k, v bf16 [B, H, s, d]); returns its output."""
        import torch
        for name, t in (("q", q), ("k", k), ("v", v)):
            _check_bf16_cuda(name, t)
            if tuple(t.shape) != (self.B, self.H, self.s, self.d):
                raise ValueError(f"{name} must have shape [B, H, s, d]")
        if out is None:
            out = torch.empty_like(q)
        _check_bf16_cuda("out", out)
        if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (self.B, self.H, self.s)
                                or not lse.is_contiguous()):
            raise ValueError("lse must be a contiguous fp32 tensor [B, H, s]")
        scale = 1.0 / math.sqrt(self.d) if scale is None else float(scale)
        check(ra_swc_cache_step(self.handle, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), scale,
                                None if lse is None else lse.data_ptr(), _stream_handle(stream)), "ra_swc_cache_step")
        return out

    @property
    def info(self) -> dict:
        seen, held = ctypes.c_longlong(), ctypes.c_int()
        check(ra_swc_cache_info(self.handle, ctypes.byref(seen), ctypes.byref(held)), "ra_swc_cache_info")
        return dict(frames_seen=seen.value, frames_held=held.value)

    def rings_to_host(self):
        """(K ring, V ring) as uint16 bf16 bit patterns [B, H, W * s, d]; frame i in slot i mod W."""
        import numpy as np
        shape = (self.B, self.H, self.W * self.s, self.d)
        k, v = np.empty(shape, dtype=np.uint16), np.empty(shape, dtype=np.uint16)
        check(ra_swc_cache_copy_rings_to_host(self.handle, k.ctypes.data, v.ctypes.data),
              "ra_swc_cache_copy_rings_to_host")
        return k, v

    def reset(self) -> None:
        check(ra_swc_cache_reset(self.handle), "ra_swc_cache_reset")

    def free(self) -> None:
        if getattr(self, "_h", None) is not None:
            ra_swc_cache_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


# ------------------------------------------- norm and rotation of Q and K
class Rope3D(NamedTuple):
    """Position tables of the time, height and width axes: contiguous fp32 CUDA
    tensors [frames | grid_h | grid_w, pairs, 2] of (cos, sin).  Any tuple of
    three such tensors does in its place."""
    t: object
    h: object
    w: object


def rope_axes(d: int) -> tuple:
    """Channels of the time, height and width axes of a head of d channels when
    none are named: height and width 2 * (d // 6) each, time the rest."""
    return d - 4 * (d // 6), 2 * (d // 6), 2 * (d // 6)


def rope3d(frames: int, grid_h: int, grid_w: int, d: int, axes=None, base: float = 10000.0, stream=None) -> Rope3D:
    """Tables for `frames` frames of grid_h x grid_w tokens: pair i of an axis of
    c channels turns by position * base^(-2 i / c).  axes: channels of each axis
    (even, at most d together)."""
    import torch
    axes = rope_axes(d) if axes is None else tuple(axes)
    if len(axes) != 3 or any(c < 0 or c % 2 for c in axes) or not 0 < sum(axes) <= d:
        raise ValueError("axes must be three even numbers of channels, at most d together")
    handle = _stream_handle(stream)
    tables = []
    for length, c in zip((frames, grid_h, grid_w), axes):
        if length < 1:
            raise ValueError("frames, grid_h and grid_w must be >= 1")
        with _allocating_on(stream, handle):
            table = torch.empty((length, c // 2, 2), dtype=torch.float32, device="cuda")
        if c:
            check(ra_rope_table(table.data_ptr(), 0, length, c // 2, float(base), handle), "ra_rope_table")
        tables.append(table)
    return Rope3D(*tables)


_binding = None


def _load_binding():
    """The extension that checks and allocates the tensors of the operators below, bound to the loaded library."""
    global _binding
    if _binding is None:
        import torch  # noqa: F401  (its libraries have to be loaded first)

        if not os.path.exists(os.path.join(_PKG, "_torch_binding.so")):
            raise ImportError("_torch_binding.so is not built; run `python static_sparse_attention_b200/build.py`")
        from . import _torch_binding as module
        module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in
                      (ra_qk_norm_rope, ra_qk_norm_rope_bwd_workspace_bytes, ra_qk_norm_rope_bwd, ra_cache8_append,
                       ra_cache8_attention_workspace_bytes, ra_cache8_attention, ra_cache8_attention_check)))
        _binding = module
    return _binding


def qk_norm_rope(q, k=None, q_weight=None, k_weight=None, rope=None, frame0: int = 0, eps: float = 1e-6, q_out=None,
                 k_out=None, stream=None):
    """Per-head RMS norm and 3-axis rotation of the projections q and k (bf16
    [B, n, H, d], any strides with contiguous channels, such as slices of a fused
    projection): returns (q, k) as bf16 [B, H, n, d], ready for attention_fwd.

    A weight (bf16 or fp32 [d]) turns the norm of its tensor on; rope (rope3d, or
    a tuple of three tables) the rotation, the first token being the first of frame
    `frame0`.  k may be left out (None is returned in its place)."""
    r = (_binding or _load_binding()).qk_norm_rope(q, k, q_weight, k_weight, rope, frame0, eps, q_out, k_out,
                                                    None if stream is None else _stream_handle(stream))
    if type(r) is int:
        check(r, "ra_qk_norm_rope")
    return r


def qk_norm_rope_bwd(q, k, dq_out, dk_out, q_weight=None, k_weight=None, rope=None, frame0: int = 0, eps: float = 1e-6,
                     dq=None, dk=None, dq_weight=None, dk_weight=None, workspace=None, stream=None):
    """Gradient of qk_norm_rope: from dq_out, dk_out (bf16 [B, H, n, d], as
    attention_bwd returns them) to (dq, dk, dq_weight, dk_weight): dq, dk bf16
    [B, n, H, d] (given ones may be strided, such as slices of one packed gradient)
    and fp32 [d] for each weight (None without one).  q, k, the weights, rope,
    frame0 and eps as in the forward call; k and dk_out may both be None."""
    r = (_binding or _load_binding()).qk_norm_rope_bwd(q, k, dq_out, dk_out, q_weight, k_weight, rope, frame0, eps, dq,
                                                        dk, dq_weight, dk_weight, workspace,
                                                        None if stream is None else _stream_handle(stream))
    if type(r) is int:
        check(r, "ra_qk_norm_rope_bwd")
    return r


# ------------------------------------------------------- 8-bit key/value ring
CACHE8_BLOCK = 64  # tokens of a frame that share a scale


def cache8_append(k, v, k8, v8, k_scale, v_scale, frame: int, k_weight=None, rope=None, eps: float = 1e-6,
                  stream=None) -> None:
    """New frames into an 8-bit key/value ring of W frames of s tokens (k8, v8:
    float8_e4m3fn [B, H, W * s, d]; k_scale, v_scale: fp32 [B, H, W, ceil(s / 64)]),
    the first one being frame number `frame` of the stream, in slot frame mod W.

    k, v: bf16 [B, frames * s, H, d], any strides with contiguous channels.  A
    k_weight (bf16 or fp32 [d]) norms the keys, rope (tables whose grid is one
    frame's) rotates them on the way."""
    check((_binding or _load_binding()).cache8_append(k, v, k8, v8, k_scale, v_scale, frame, k_weight, rope, eps,
                                                       None if stream is None else _stream_handle(stream)),
          "ra_cache8_append")


def cache8_attention(q, k8, v8, k_scale, v_scale, held: int, key_counts=None, scale: float | None = None, out=None,
                     lse=None, workspace=None, stream=None):
    """Attention of q (bf16 [B, H, nq, d], nq >= 1) over the frames in slots 0 ..
    held - 1 of an 8-bit ring (see cache8_append).  key_counts (int32 [B]) limits
    each batch element to its first rows; a query without keys gets 0 (lse -inf)."""
    r = (_binding or _load_binding()).cache8_attention(q, k8, v8, k_scale, v_scale, held, key_counts, scale, out, lse,
                                                        workspace, None if stream is None else _stream_handle(stream))
    if type(r) is int:
        check(r, "ra_cache8_attention")
    return r


class SwcCache8:
    """Streaming sliding-window causal attention over an 8-bit key/value ring: the
    window of SwcCache in half its memory, fed with the projections' rows, which
    are normed and rotated on the way.

    k8, v8, k_scale and v_scale are the ring's buffers (see cache8_append).  Creation
    is synchronous.  Steps must be ordered on one stream (any one; the buffers' memory
    is reused behind its work), and are refused while it is being captured into a CUDA
    graph (a replay would repeat one frame number): capture cache8_append and
    cache8_attention there instead."""

    def __init__(self, B: int, H: int, d: int, s: int, window_frames: int):
        import torch
        if min(B, H, s, window_frames) < 1:
            raise ValueError("B, H, s and window_frames must be >= 1")
        if d not in (64, 128):
            raise ValueError(f"head dim {d} is not supported (64 or 128)")
        self.B, self.H, self.d, self.s, self.W = B, H, d, s, window_frames
        # zeros: slots not yet filled hold numbers too
        self.k8, self.v8 = (torch.zeros((B, H, window_frames * s, d), dtype=torch.uint8, device="cuda")
                            .view(torch.float8_e4m3fn) for _ in range(2))
        self.k_scale, self.v_scale = (torch.ones((B, H, window_frames, -(-s // CACHE8_BLOCK)), device="cuda")
                                      for _ in range(2))
        # the fills are on the current stream, the steps on whatever stream they are given
        self._streams = {_stream_handle(None)}
        torch.cuda.current_stream().synchronize()
        self.frames_seen = 0

    def _used_on(self, stream) -> None:
        """Have the allocator reuse the ring's memory only behind the work of `stream`."""
        handle = _stream_handle(stream)
        if handle not in self._streams:
            import torch
            other = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
            for t in self._ring:
                t.record_stream(other)
            self._streams.add(handle)

    @property
    def frames_held(self) -> int:
        return min(self.frames_seen, self.W)

    @property
    def info(self) -> dict:
        return dict(frames_seen=self.frames_seen, frames_held=self.frames_held)

    @property
    def _ring(self):
        return self.k8, self.v8, self.k_scale, self.v_scale

    def append(self, k, v, k_weight=None, rope=None, eps: float = 1e-6, stream=None) -> None:
        """One or more new frames (k, v: bf16 [B, frames * s, H, d]); of more than W
        the last W are kept."""
        _refuse_capture(stream)
        self._used_on(stream)
        self._append(k, v, k_weight, rope, eps, stream)

    def _append(self, k, v, k_weight, rope, eps, stream) -> None:
        if k.dim() != 4 or v.shape != k.shape or k.shape[1] < self.s or k.shape[1] % self.s:
            raise ValueError(f"k and v must have shape [{self.B}, frames * {self.s}, {self.H}, {self.d}]")
        frames = k.shape[1] // self.s
        if frames > self.W:
            skip = frames - self.W
            k, v = k[:, skip * self.s:], v[:, skip * self.s:]
        else:
            skip = 0
        cache8_append(k, v, *self._ring, self.frames_seen + skip, k_weight, rope, eps, stream)
        self.frames_seen += frames

    def attend(self, q, out=None, lse=None, scale: float | None = None, workspace=None, stream=None):
        """Attention of q (bf16 [B, H, nq, d]) over every token of the frames held."""
        self._used_on(stream)
        return cache8_attention(q, *self._ring, self.frames_held, None, scale, out, lse, workspace, stream)

    def step(self, q, k, v, q_weight=None, k_weight=None, rope=None, eps: float = 1e-6, out=None, lse=None,
             scale: float | None = None, stream=None):
        """Feed the next frame (q, k, v: bf16 [B, s, H, d], the projections' rows);
        returns its output, bf16 [B, H, s, d].  A step that raises feeds nothing: the
        attention's arguments are checked and its buffers allocated before the append."""
        _refuse_capture(stream)
        if tuple(q.shape) != (self.B, self.s, self.H, self.d) or q.shape != k.shape:
            raise ValueError(f"q, k and v must have shape [{self.B}, {self.s}, {self.H}, {self.d}]")
        self._used_on(stream)
        if q_weight is None and rope is None:
            with _allocating_on(stream, _stream_handle(stream)):
                q = q.transpose(1, 2).contiguous()
        else:
            q, _ = qk_norm_rope(q, None, q_weight, None, rope, self.frames_seen, eps, stream=stream)
        r = (_binding or _load_binding()).cache8_attention_prepare(
            q, *self._ring, min(self.frames_seen + 1, self.W), None, scale, out, lse, None,
            None if stream is None else _stream_handle(stream))
        if type(r) is int:
            check(r, "ra_cache8_attention")
        out, workspace = r
        self._append(k, v, k_weight, rope, eps, stream)
        try:
            return cache8_attention(q, *self._ring, self.frames_held, None, scale, out, lse, workspace, stream)
        except Exception:
            self.frames_seen -= 1  # the launch failed: the next step takes the same slot
            raise

    def reset(self) -> None:
        """Forget every frame (the next one is frame 0)."""
        self.frames_seen = 0


class DenseFirstPolicy:
    """Which mask a denoising step uses in each attention block: dense for the
    first `dense_steps` steps (warm-up) and, at every step, for the first
    `dense_blocks` blocks; the sparse mask elsewhere ("Radial Attention",
    sec. 6: the first 2 DiT blocks and the first 12 denoising steps stay dense)."""

    def __init__(self, sparse: Mask, dense: Mask, dense_steps: int = 12, dense_blocks: int = 2):
        if dense_steps < 0 or dense_blocks < 0:
            raise ValueError("dense_steps and dense_blocks must be >= 0")
        if sparse.n != dense.n:
            raise ValueError("both masks must cover the same tokens")
        self.sparse, self.dense = sparse, dense
        self.dense_steps, self.dense_blocks = dense_steps, dense_blocks

    def is_dense(self, step: int, block: int) -> bool:
        return step < self.dense_steps or block < self.dense_blocks

    def mask(self, step: int, block: int) -> Mask:
        return self.dense if self.is_dense(step, block) else self.sparse

    def dense_calls(self, steps: int, blocks: int) -> int:
        """Dense calls in a schedule of `steps` x `blocks` attention calls."""
        warm = min(self.dense_steps, steps)
        return warm * blocks + (steps - warm) * min(self.dense_blocks, blocks)


def device_status(stream=None) -> int:
    """Synchronise and read (then clear) the device error word; returns the status code."""
    return ra_get_device_status(_stream_handle(stream))
