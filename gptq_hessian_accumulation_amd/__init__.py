"""Calibration-Hessian accumulation on AMD Instinct MI355X (gfx950).

Python binding of ``libhess.so`` (C ABI in ``include/hess.h``).  The binding
only marshals arguments: every step runs in the library's HIP kernels.
PyTorch supplies device memory and the current HIP stream.

    H = (2/N) * sum_t x_t x_t^T         (GPTQModel PR 2979, What Changed)

``Hessian.add_batch`` accumulates one calibration batch in place,
``Hessian.materialize`` scales by 2/N, neutralizes dead columns and adds
``damp_percent * mean(diag)`` to the diagonal (GPTQModel wiki "QQQ",
Concepts > Quadratic error compensation), ``local_blocks`` builds the 16 x 16
per-block Gram matrices and ``add_batch_grouped`` updates many routed-expert
Hessians in one launch (Model-Optimizer PR 3002 page, "What does this PR do?").

There is no CPU fallback: without the built library every call raises.
"""

from __future__ import annotations

import ctypes
import os
import re
from typing import NamedTuple

import torch
import torch.autograd.forward_ad as _forward_ad

__all__ = [
    "Hessian",
    "HessError",
    "local_blocks",
    "add_batch_grouped",
    "reset_grouped",
    "materialize_grouped",
    "chol_inverse_upper",
    "gptq_quantize",
    "gated_ffn",
    "gated_ffn_forward",
    "gated_ffn_backward",
    "distill_topk",
    "distill_topk_forward",
    "distill_topk_backward",
    "distill_topk_step",
    "Int8Rows",
    "quantize_int8",
    "dequantize_int8",
    "int8_matmul",
    "int8_linear",
    "int8_linear_forward",
    "int8_linear_backward",
    "set_tile_override",
    "set_ffn_schedule",
    "set_staging",
    "library_path",
    "exported_symbols",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libhess.so")
_HEADER = os.path.join(os.path.dirname(_PKG), "include", "hess.h")

HESS_BF16 = 0
HESS_F32 = 1
HESS_F16 = 2
HESS_NO_NEUTRALIZE = 1

_STATUS = {0: "HESS_OK", -1: "HESS_EINVAL", -2: "HESS_ENOMEM", -3: "HESS_EHIP", -4: "HESS_ESTATE",
           -5: "HESS_EALIGN", -6: "HESS_ENOTPD"}


class HessError(RuntimeError):
    """A libhess call returned an error status."""

    def __init__(self, code: int, message: str):
        super().__init__(f"{_STATUS.get(code, code)}: {message}")
        self.code = code


_lib = None


def library_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"libhess.so is not built ({_LIB_PATH}); run `python gptq_hessian_accumulation_amd/build.py` "
            "(or __graft_entry__.build()).  There is no CPU fallback.")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i64, c_int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    sig = {
        "hess_abi_version": (c_int, []),
        "hess_strerror": (ctypes.c_char_p, [c_int]),
        "hess_last_error": (ctypes.c_char_p, []),
        "hess_create": (vp, [i64, c_int]),
        "hess_create_ex": (vp, [i64, c_int, i64]),
        "hess_destroy": (c_int, [vp]),
        "hess_add_batch": (c_int, [vp, vp, i64, i64, vp]),
        "hess_add_batch_cast": (c_int, [vp, vp, c_int, i64, i64, vp]),
        "hess_materialize": (c_int, [vp, ctypes.c_float, vp]),
        "hess_materialize_ex": (c_int, [vp, ctypes.c_float, ctypes.c_uint, vp, vp, vp, vp]),
        "hess_reset": (c_int, [vp, vp]),
        "hess_token_count": (c_int, [vp, ctypes.POINTER(i64)]),
        "hess_set_tile_override": (c_int, [c_int]),
        "hess_set_ffn_schedule": (c_int, [c_int, c_int, c_int]),
        "hess_set_staging": (c_int, [c_int]),
        "hess_set_async_flush": (c_int, [c_int]),
        "hess_set_group_chunk": (c_int, [i64]),
        "hess_flush": (c_int, [vp, vp]),
        "hess_set_timing": (c_int, [vp, c_int]),
        "hess_timing": (c_int, [vp, ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.POINTER(ctypes.c_double)]),
        "hess_info": (c_int, [vp, ctypes.POINTER(i64), ctypes.POINTER(c_int)]),
        "hess_state_buffer": (c_int, [vp, ctypes.POINTER(vp)]),
        "hess_local_blocks": (c_int, [vp, i64, i64, c_int, vp]),
        "hess_local_blocks_ex": (c_int, [vp, c_int, i64, i64, i64, c_int, vp, c_int, vp]),
        "hess_local_blocks_noalloc": (c_int, [vp, c_int, i64, i64, i64, c_int, vp, c_int, vp]),
        "hess_add_batch_grouped": (c_int, [ctypes.POINTER(vp), c_int, vp, i64, vp, ctypes.POINTER(i64), vp]),
        "hess_add_batch_grouped_ex": (c_int, [ctypes.POINTER(vp), c_int, vp, i64, i64, vp, ctypes.POINTER(i64), vp]),
        "hess_set_group_direct": (c_int, [c_int]),
        "hess_adopt": (c_int, [vp, vp, vp]),
        "hess_reset_grouped": (c_int, [ctypes.POINTER(vp), c_int, vp]),
        "hess_materialize_grouped": (c_int, [ctypes.POINTER(vp), c_int, ctypes.c_float, ctypes.c_uint,
                                             ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp), vp]),
        "hess_chol_inverse_workspace": (i64, [i64]),
        "hess_gptq_quantize_workspace": (i64, [i64, i64]),
        "hess_gptq_quantize": (c_int, [vp, i64, i64, i64, vp, i64, vp, c_int, vp, i64, vp, i64, vp, vp, i64, vp,
                                       i64, vp]),
        "hess_chol_inverse_upper": (c_int, [vp, i64, i64, vp, i64, vp, i64, vp, vp]),
        "hess_gated_ffn_workspace": (i64, [i64, i64, i64, c_int, c_int]),
        "hess_gated_ffn_preact_cols": (i64, [i64]),
        "hess_gated_ffn_forward": (c_int, [vp, i64, vp, i64, vp, i64, c_int, c_int, i64, i64, i64, vp, i64, vp, vp,
                                           i64, vp]),
        "hess_gated_ffn_backward": (c_int, [vp, i64, vp, i64, vp, i64, vp, i64, vp, c_int, c_int, i64, i64, i64, vp,
                                            i64, vp, i64, vp, i64, vp, i64, vp]),
        "hess_distill_topk_workspace": (i64, [i64, i64, c_int]),
        "hess_distill_topk": (c_int, [vp, i64, c_int, i64, i64, vp, c_int, i64, vp, c_int, i64, c_int, vp,
                                      ctypes.c_float, vp, vp, vp, i64, vp, i64, vp]),
        "hess_distill_topk_backward": (c_int, [vp, vp, i64, c_int, i64, i64, vp, c_int, i64, vp, c_int, i64, c_int,
                                               vp, ctypes.c_float, vp, vp, i64, vp]),
        "hess_gated_ffn_preact_i8_cols": (i64, [i64]),
        "hess_gated_ffn_i8_workspace": (i64, [i64, i64, i64, c_int]),
        "hess_gated_ffn_backward_x8": (c_int, [vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, c_int, c_int, i64, i64, i64,
                                               vp, i64, vp, i64, vp, i64, vp, i64, vp]),
        "hess_int8_quantize": (c_int, [vp, i64, c_int, i64, i64, c_int, vp, i64, i64, vp, vp]),
        "hess_int8_dequantize": (c_int, [vp, i64, vp, i64, i64, c_int, vp, i64, c_int, vp]),
        "hess_int8_matmul_workspace": (i64, [i64, i64, i64]),
        "hess_int8_matmul": (c_int, [vp, i64, vp, vp, i64, vp, i64, i64, i64, vp, i64, c_int, vp, i64, vp]),
        "hess_int8_linear_workspace": (i64, [i64, i64, i64, c_int, c_int]),
        "hess_int8_linear_forward": (c_int, [vp, i64, c_int, vp, i64, vp, i64, i64, i64, vp, i64, vp, i64, vp, vp, i64,
                                             vp]),
        "hess_int8_linear_backward": (c_int, [vp, i64, c_int, vp, i64, vp, vp, i64, vp, i64, i64, i64, vp, i64, vp,
                                              i64, vp, i64, vp]),
        "hess_imatrix_create": (vp, [i64, c_int]),
        "hess_imatrix_destroy": (c_int, [vp]),
        "hess_imatrix_add_batch": (c_int, [vp, vp, i64, i64, vp]),
        "hess_imatrix_read": (c_int, [vp, vp, ctypes.POINTER(i64), vp]),
        "hess_imatrix_reset": (c_int, [vp, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(code: int) -> None:
    if code != 0:
        lib = _load()
        raise HessError(code, lib.hess_last_error().decode(errors="replace"))


def exported_symbols() -> list:
    """Names of the functions declared in include/hess.h."""
    with open(_HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(hess_[a-z0-9_]+)\s*\(", text)))


# The current stream's raw handle without building a Stream object (about 2.5 us
# per call saved, which matters at one call per short calibration batch).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream=None, device=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device() if device is None else device)
    return torch.cuda.current_stream(device).cuda_stream


def _dtype_code(dtype) -> int:
    if dtype == torch.bfloat16:
        return HESS_BF16
    if dtype == torch.float32:
        return HESS_F32
    raise TypeError(f"unsupported activation dtype {dtype}; use torch.bfloat16 or torch.float32")


def _act_code(dtype) -> int:
    if dtype == torch.float16:
        return HESS_F16
    return _dtype_code(dtype)


def _as_rows(x: torch.Tensor, d: int):
    """(tokens, d) view of x whose rows are d contiguous elements at a stride ld >= d.

    Returns (tensor, n, ld).  A view whose rows overlap or repeat (a broadcast
    row, stride 0, or a sliding window, stride < d) or whose features are not
    contiguous is copied first, so the library never reads past the storage.
    """
    if x.shape[-1] != d:
        raise ValueError(f"last dimension {x.shape[-1]} != d = {d}")
    x2 = x.reshape(-1, d) if x.dim() != 2 else x
    n = x2.shape[0]
    if n > 0 and d > 1 and x2.stride(1) != 1:
        x2 = x2.contiguous()
    if n > 1 and x2.stride(0) < d:
        x2 = x2.contiguous()
    ld = x2.stride(0) if n > 1 else d
    return x2, n, ld


def set_staging(enable: bool) -> None:
    """Enable (default) or disable the staging of short batches; process-wide."""
    _check(_load().hess_set_staging(1 if enable else 0))


def set_async_flush(enable: bool) -> None:
    """Enable (default) or disable asynchronous staging flushes for Hessians created afterwards; process-wide."""
    _check(_load().hess_set_async_flush(1 if enable else 0))


def set_group_chunk(nbytes: int) -> None:
    """Cap the rows gathered per 256-tile grouped launch (bytes; 0 = the whole buffer); process-wide."""
    _check(_load().hess_set_group_chunk(int(nbytes)))


def set_group_direct(enable: bool) -> None:
    """Grouped 256-tile updates read the routed rows in place (default) or gather them first; process-wide."""
    _check(_load().hess_set_group_direct(1 if enable else 0))


def set_tile_override(edge: int) -> None:
    """Force the SYRK tile edge (0 = automatic, 64, 128 or 256); process-wide."""
    _check(_load().hess_set_tile_override(int(edge)))


def set_ffn_schedule(edge: int = 0, whole: int = 0, parts: int = 1) -> None:
    """Force the feed-forward block's and the 8-bit product's tiles (edge 0 = automatic, 64, 128 or 256), the first
    ``whole`` done whole and the others in ``parts`` ranges of the sum; process-wide."""
    _check(_load().hess_set_ffn_schedule(int(edge), int(whole), int(parts)))


class Hessian:
    """One calibration-Hessian accumulator of width ``d`` on the current GPU.

    ``dtype`` is the staging dtype (``torch.bfloat16`` or ``torch.float32``):
    the type the products are formed in.  Batches of that type are read as
    they are; float16, bfloat16 or float32 batches of another type are
    converted on their way into the staging buffer (rounded to nearest even
    when narrowing).  The Hessian is always float32.  ``staging_bytes`` sizes
    the buffer that collects short batches (default: 1 GiB at
    d >= 1024, else 64 MiB; 0 disables staging and conversion).
    """

    def __init__(self, d: int, dtype=torch.bfloat16, staging_bytes: int | None = None):
        lib = _load()
        self.d = int(d)
        self.dtype = dtype
        self._code = _dtype_code(dtype)
        if staging_bytes is None:
            h = lib.hess_create(self.d, self._code)
        else:
            h = lib.hess_create_ex(self.d, self._code, int(staging_bytes))
        if not h:
            raise HessError(-1, lib.hess_last_error().decode(errors="replace"))
        self._h = ctypes.c_void_p(h)
        self._device = torch.cuda.current_device()
        self._add = lib.hess_add_batch

    # -- accumulation ----------------------------------------------------
    def add_batch(self, x: torch.Tensor, stream=None) -> None:
        """S += X^T X, N += tokens; leading dimensions of x are flattened to tokens."""
        if not x.is_cuda:
            raise ValueError("activations must be on the GPU")
        code = _act_code(x.dtype)
        x2, n, ld = _as_rows(x, self.d)
        ptr = x2.data_ptr() if n > 0 else None
        if code == self._code:
            rc = self._add(self._h, ptr, n, ld, _stream(stream))
        else:
            rc = _load().hess_add_batch_cast(self._h, ptr, code, n, ld, _stream(stream))
        if rc != 0:
            _check(rc)

    def materialize(self, damp_percent: float = 0.01, out: torch.Tensor | None = None, neutralize: bool = True,
                    stream=None):
        """Return ``(H, dead, damp)``: H float32 (d, d), dead bool (d,), damp float32 (1,), all on the GPU."""
        dev = torch.device("cuda", self._device)
        if out is None:
            out = torch.empty((self.d, self.d), dtype=torch.float32, device=dev)
        elif out.dtype != torch.float32 or tuple(out.shape) != (self.d, self.d) or not out.is_contiguous():
            raise ValueError("out must be a contiguous float32 (d, d) GPU tensor")
        dead = torch.empty(self.d, dtype=torch.uint8, device=dev)
        damp = torch.empty(1, dtype=torch.float32, device=dev)
        flags = 0 if neutralize else HESS_NO_NEUTRALIZE
        _check(_load().hess_materialize_ex(self._h, float(damp_percent), flags, out.data_ptr(), dead.data_ptr(),
                                           damp.data_ptr(), _stream(stream)))
        return out, dead.view(torch.bool), damp

    def materialize_in_place(self, damp_percent: float = 0.01, neutralize: bool = True, stream=None):
        """Materialize into the accumulator's own buffer; the handle then needs reset()."""
        dev = torch.device("cuda", self._device)
        dead = torch.empty(self.d, dtype=torch.uint8, device=dev)
        damp = torch.empty(1, dtype=torch.float32, device=dev)
        flags = 0 if neutralize else HESS_NO_NEUTRALIZE
        _check(_load().hess_materialize_ex(self._h, float(damp_percent), flags, None, dead.data_ptr(),
                                           damp.data_ptr(), _stream(stream)))
        return dead.view(torch.bool), damp

    def state_buffer_ptr(self) -> int:
        p = ctypes.c_void_p()
        _check(_load().hess_state_buffer(self._h, ctypes.byref(p)))
        return p.value

    def flush(self, stream=None) -> None:
        """Fold staged short batches into the Gram sum."""
        _check(_load().hess_flush(self._h, _stream(stream)))

    def state_tensor(self) -> torch.Tensor:
        """A (d, d) float32 view of the accumulator's device buffer (S, or H after an in-place materialize).

        Call flush() first when reading S, so that staged batches are included.
        """
        ptr, d = self.state_buffer_ptr(), self.d

        class _View:
            __cuda_array_interface__ = {"shape": (d, d), "typestr": "<f4", "data": (ptr, False), "version": 2,
                                        "strides": None}

        return torch.as_tensor(_View(), device=torch.device("cuda", self._device))

    def reset(self, stream=None) -> None:
        _check(_load().hess_reset(self._h, _stream(stream)))

    def adopt_from(self, leader: "Hessian", stream=None) -> None:
        """Replace this Hessian's statistics with a private copy of leader's (sum and token count)."""
        _check(_load().hess_adopt(self._h, leader._h, _stream(stream)))

    def set_timing(self, on: bool) -> None:
        """Bracket every SYRK launch of this handle with HIP events on its stream."""
        _check(_load().hess_set_timing(self._h, 1 if on else 0))

    def timing(self):
        """``(launches, tokens, ms)`` of the SYRK launches timed since the last read (waits for them)."""
        n, t, ms = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_double()
        _check(_load().hess_timing(self._h, ctypes.byref(n), ctypes.byref(t), ctypes.byref(ms)))
        return n.value, t.value, ms.value

    @property
    def nsamples(self) -> int:
        n = ctypes.c_int64()
        _check(_load().hess_token_count(self._h, ctypes.byref(n)))
        return n.value

    def close(self) -> None:
        if getattr(self, "_h", None) is not None and self._h.value:
            _check(_load().hess_destroy(self._h))
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def local_blocks(x: torch.Tensor, out: torch.Tensor | None = None, accumulate: bool = True, block: int = 16,
                 stream=None) -> torch.Tensor:
    """out[b] (+)= X_b^T X_b for every 16-feature block b; float32 (d/16, 16, 16)."""
    if not x.is_cuda:
        raise ValueError("activations must be on the GPU")
    d = x.shape[-1]
    x2, n, ld = _as_rows(x, d)
    if out is None:
        out = torch.zeros((d // block, block, block), dtype=torch.float32, device=x.device)
    elif out.dtype != torch.float32 or not out.is_contiguous() or out.numel() != (d // block) * block * block:
        raise ValueError("out must be a contiguous float32 (d/16, 16, 16) GPU tensor")
    ptr = x2.data_ptr() if n > 0 else None
    _check(_load().hess_local_blocks_ex(ptr, _dtype_code(x.dtype), n, d, ld, block, out.data_ptr(),
                                        1 if accumulate else 0, _stream(stream)))
    return out


def chol_inverse_upper(H: torch.Tensor, out: torch.Tensor | None = None, check: bool = True,
                       workspace: torch.Tensor | None = None, stream=None):
    """U (float32, upper triangular, positive diagonal) with U^T U = H^-1, for a damped Hessian H.

    Only H's upper triangle is read; ``out`` may be H itself.  With ``check``
    the call waits for the result and raises HessError(HESS_ENOTPD) when H
    is not positive definite; otherwise it returns ``(U, info)`` with info a
    device int32 tensor (0, or 1 + the failing column).
    """
    if not H.is_cuda or H.dtype != torch.float32 or H.dim() != 2 or H.shape[0] != H.shape[1]:
        raise ValueError("H must be a square float32 GPU tensor")
    if H.stride(1) != 1:
        raise ValueError("H must have unit column stride")
    lib = _load()
    d = H.shape[0]
    if out is None:
        out = torch.empty((d, d), dtype=torch.float32, device=H.device)
    elif out.dtype != torch.float32 or tuple(out.shape) != (d, d) or out.stride(1) != 1:
        raise ValueError("out must be a float32 (d, d) GPU tensor with unit column stride")
    need = int(lib.hess_chol_inverse_workspace(d))
    if need < 0:
        raise HessError(-1, f"width {d} not supported")
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=H.device)
    info = torch.empty(1, dtype=torch.int32, device=H.device)
    _check(lib.hess_chol_inverse_upper(H.data_ptr(), d, H.stride(0), out.data_ptr(), out.stride(0),
                                       workspace.data_ptr(), need, info.data_ptr(), _stream(stream)))
    if not check:
        return out, info
    bad = int(info.item())
    if bad:
        raise HessError(-6, f"the damped Hessian is not positive definite (pivot of column {bad - 1} failed)")
    return out


def gptq_quantize(W: torch.Tensor, U: torch.Tensor, group_size: int = -1, dead: torch.Tensor | None = None,
                  nsamples: int = 1, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                  stream=None):
    """4-bit error-propagating quantization of W (outputs x inputs, float32) with the factor U.

    Returns ``(Q, codes, scales, loss)``: dequantized float32 weights (``out`` may be W itself),
    uint8 codes 0..15, float32 steps (rows x groups) and a float64 device scalar loss.
    """
    for name, t in (("W", W), ("U", U)):
        if not t.is_cuda or t.dtype != torch.float32 or t.dim() != 2 or t.stride(1) != 1:
            raise ValueError(f"{name} must be a 2-D float32 GPU tensor with unit column stride")
    rows, cols = W.shape
    if tuple(U.shape) != (cols, cols):
        raise ValueError("U must be (cols, cols)")
    lib = _load()
    dev = W.device
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.float32, device=dev)
    codes = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    groups = 1 if group_size == -1 or group_size >= cols else -(-cols // group_size)
    scales = torch.empty((rows, groups), dtype=torch.float32, device=dev)
    loss = torch.empty(1, dtype=torch.float64, device=dev)
    need = int(lib.hess_gptq_quantize_workspace(rows, cols))
    if need < 0:
        raise HessError(-1, f"shape {rows} x {cols} not supported")
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    dptr = None
    if dead is not None:
        dead = dead.to(device=dev, dtype=torch.uint8).contiguous()
        if dead.numel() != cols:
            raise ValueError("dead must have one entry per column")
        dptr = dead.data_ptr()
    _check(lib.hess_gptq_quantize(W.data_ptr(), rows, cols, W.stride(0), U.data_ptr(), U.stride(0), dptr,
                                  int(group_size), out.data_ptr(), out.stride(0), codes.data_ptr(), codes.stride(0),
                                  scales.data_ptr(), loss.data_ptr(), int(nsamples), workspace.data_ptr(), need,
                                  _stream(stream)))
    return out, codes, scales, loss


class ImatrixStat:
    """Per-column float32 sums of squares of a layer's inputs (the imatrix statistic)."""

    def __init__(self, d: int, dtype=torch.bfloat16):
        self.d = int(d)
        self.dtype = dtype
        self._h = _load().hess_imatrix_create(self.d, _dtype_code(dtype))
        if not self._h:
            raise HessError(-1, _load().hess_last_error().decode(errors="replace"))

    def add_batch(self, x: torch.Tensor, stream=None) -> None:
        if not x.is_cuda:
            raise ValueError("activations must be on the GPU")
        if x.dtype != self.dtype:
            raise ValueError(f"expected {self.dtype} activations, got {x.dtype}")
        x2, n, ld = _as_rows(x, self.d)
        _check(_load().hess_imatrix_add_batch(self._h, x2.data_ptr() if n > 0 else None, n, ld, _stream(stream)))

    def read(self, out: torch.Tensor | None = None, stream=None):
        """(sums, tokens): the float32 per-column sums and the token count."""
        if out is None:
            out = torch.empty(self.d, dtype=torch.float32, device="cuda")
        n = ctypes.c_int64()
        _check(_load().hess_imatrix_read(self._h, out.data_ptr(), ctypes.byref(n), _stream(stream)))
        return out, int(n.value)

    def reset(self, stream=None) -> None:
        _check(_load().hess_imatrix_reset(self._h, _stream(stream)))

    def close(self) -> None:
        if getattr(self, "_h", None):
            _check(_load().hess_imatrix_destroy(self._h))
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def add_batch_grouped(hessians, x: torch.Tensor, offsets, row_idx: torch.Tensor | None = None, stream=None) -> None:
    """For each e: hessians[e] accumulates rows row_idx[offsets[e]:offsets[e+1]] of x, in one launch."""
    if not hessians:
        raise ValueError("need at least one Hessian")
    d = hessians[0].d
    for h in hessians:
        if h.dtype != x.dtype:
            raise TypeError("all Hessians must take the activation dtype")
    x2, n, ld = _as_rows(x, d)
    offs = [int(o) for o in (offsets.tolist() if hasattr(offsets, "tolist") else offsets)]
    if len(offs) != len(hessians) + 1:
        raise ValueError("offsets must have len(hessians) + 1 entries")
    if row_idx is not None:
        if row_idx.dtype != torch.int32 or not row_idx.is_cuda or not row_idx.is_contiguous():
            raise ValueError("row_idx must be a contiguous int32 GPU tensor")
        if row_idx.numel() < offs[-1]:
            raise ValueError("row_idx shorter than offsets[-1]")
    elif offs[-1] > n:
        raise ValueError("offsets exceed the number of rows of x")
    arr = (ctypes.c_void_p * len(hessians))(*[h._h.value for h in hessians])
    oarr = (ctypes.c_int64 * len(offs))(*offs)
    _check(_load().hess_add_batch_grouped_ex(arr, len(hessians), x2.data_ptr() if n > 0 else None, n, ld,
                                             row_idx.data_ptr() if row_idx is not None else None, oarr,
                                             _stream(stream)))


def reset_grouped(hessians, stream=None) -> None:
    """hessians[e].reset() for every e, in one launch per 64 Hessians of one width."""
    arr = (ctypes.c_void_p * len(hessians))(*[h._h.value for h in hessians])
    _check(_load().hess_reset_grouped(arr, len(hessians), _stream(stream)))


def materialize_grouped(hessians, damp_percent: float = 0.01, outs=None, neutralize: bool = True, stream=None):
    """Materialize many Hessians of one width in two launches per 64; returns [(H, dead, damp)] as
    ``Hessian.materialize`` would for each (the same bits)."""
    if not hessians:
        return []
    d = hessians[0].d
    dev = torch.device("cuda", hessians[0]._device)
    if outs is None:
        outs = [torch.empty((d, d), dtype=torch.float32, device=dev) for _ in hessians]
    if len(outs) != len(hessians):
        raise ValueError("one output per Hessian")
    for o in outs:
        if o.dtype != torch.float32 or tuple(o.shape) != (d, d) or not o.is_contiguous():
            raise ValueError("each output must be a contiguous float32 (d, d) GPU tensor")
    dead = torch.empty((len(hessians), d), dtype=torch.uint8, device=dev)
    damp = torch.empty((len(hessians), 1), dtype=torch.float32, device=dev)
    n = len(hessians)
    hs_arr = (ctypes.c_void_p * n)(*[h._h.value for h in hessians])
    h_arr = (ctypes.c_void_p * n)(*[o.data_ptr() for o in outs])
    d_arr = (ctypes.c_void_p * n)(*[dead[e].data_ptr() for e in range(n)])
    p_arr = (ctypes.c_void_p * n)(*[damp[e].data_ptr() for e in range(n)])
    flags = 0 if neutralize else HESS_NO_NEUTRALIZE
    _check(_load().hess_materialize_grouped(hs_arr, n, float(damp_percent), flags, h_arr, d_arr, p_arr,
                                            _stream(stream)))
    return [(outs[e], dead[e].view(torch.bool), damp[e]) for e in range(n)]


# -- the gated feed-forward block -----------------------------------------------------------------

_ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
_PREACT_F32 = 16
_PREACT_I8 = 64
_FEW = 64  # tokens of a forward call up to which the library takes rows of any alignment
_CODES = {torch.bfloat16: HESS_BF16, torch.float32: HESS_F32, torch.float16: HESS_F16}


def _float_code(name: str, t: torch.Tensor) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be on the GPU")
    if index != _current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current device")
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} of {name}; use torch.bfloat16, torch.float16 or torch.float32")
    return code


def _rows(t: torch.Tensor, step: int = 1):
    """(tensor, pointer, row stride) of a 2-D tensor whose rows are contiguous, do not overlap and start at
    multiples of ``step`` elements: 1, or 16 bytes' worth for rows of a multiple of that (copied if need be)."""
    ptr = t.data_ptr()
    if t.is_contiguous() and (step == 1 or ptr % 16 == 0):
        return t, ptr, t.shape[1] or 1
    n, c = t.shape
    s0, s1 = t.stride()
    if (s1 != 1 and c > 1) or (n > 1 and (s0 < c or s0 % step != 0)) or (step > 1 and ptr % 16 != 0):
        t = t.clone(memory_format=torch.contiguous_format)
        return t, t.data_ptr(), c or 1
    return t, ptr, (s0 if n > 1 else c or 1)


def _out(name: str, out, shape, like: torch.Tensor) -> torch.Tensor:
    """``out`` checked, or a new tensor: ``shape`` on like's device and of its dtype, rows contiguous."""
    if out is None:
        return like.new_empty(shape)
    if out.dtype != like.dtype or out.device != like.device or tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name} must be a {like.dtype} {tuple(shape)} tensor on {like.device}")
    if out.dim() != 2 and not out.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if out.dim() == 2 and ((out.stride(1) != 1 and shape[1] > 1) or (shape[0] > 1 and out.stride(0) < shape[1])):
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return out


def _workspace(work, need: int, like: torch.Tensor):
    """(pointer, bytes, tensor) of ``work`` if it is large enough, else of a new workspace."""
    if need == 0:
        return None, 0, None
    if need < 0:
        raise HessError(-1, _load().hess_last_error().decode(errors="replace"))
    if work is None or work.numel() * work.element_size() < need:
        work = like.new_empty(need, dtype=torch.uint8)
    elif work.device != like.device or not work.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return work.data_ptr(), work.numel() * work.element_size(), work


def _act_mode(act: str) -> int:
    mode = _ACTS.get(act)
    if mode is None:
        raise ValueError(f"unknown activation {act!r}; use one of {sorted(_ACTS)}")
    return mode


def _ffn_weights(like, w_gate, w_up, name):
    """(code, f, d, tensors to keep, (gate, stride, up, stride)) of weights of like's type, for tiles."""
    code = _float_code(name, like)
    shape = w_gate.shape
    if len(shape) != 2 or shape != w_up.shape:
        raise ValueError("w_gate and w_up must be (f, d) matrices of one shape")
    for w, t in (("w_gate", w_gate), ("w_up", w_up)):
        if t.dtype != like.dtype or t.get_device() != like.get_device():
            raise ValueError(f"{w} must have {name}'s dtype and device")
    f, d = shape
    step = 4 if code == HESS_F32 else 8
    step = step if d % step == 0 else 1
    wg, gp, ldg = _rows(w_gate, step)
    wu, up, ldu = _rows(w_up, step)
    return code, f, d, (wg, wu), (gp, ldg, up, ldu)


def _ffn_args(x, w_gate, w_up, any_rows=0):
    """(code, n, d, f, tensors to keep, (x, stride, gate, stride, up, stride) for the library).

    any_rows: up to how many tokens the call reads rows of any alignment where they are."""
    code = _float_code("x", x)
    shape = w_gate.shape
    if len(shape) != 2 or shape != w_up.shape:
        raise ValueError("w_gate and w_up must be (f, d) matrices of one shape")
    f, d = shape
    given = x.shape
    if len(given) < 1 or given[-1] != d:
        raise ValueError(f"last dimension of x {tuple(given)} != d = {d}")
    dtype, index = x.dtype, x.get_device()
    if w_gate.dtype != dtype or w_gate.get_device() != index:
        raise ValueError("w_gate must have x's dtype and device")
    if w_up.dtype != dtype or w_up.get_device() != index:
        raise ValueError("w_up must have x's dtype and device")
    x2 = x if len(given) == 2 else x.reshape(-1, d)
    # the tiles read rows of a multiple of 16 bytes where they are, if they start at 16 bytes
    step = 4 if code == HESS_F32 else 8
    if d % step != 0 or x2.shape[0] <= any_rows:
        step = 1
    x2, xp, ldx = _rows(x2, step)
    wg, gp, ldg = _rows(w_gate, step)
    wu, up, ldu = _rows(w_up, step)
    return code, x2.shape[0], d, f, (x2, wg, wu), (xp, ldx, gp, ldg, up, ldu)


def gated_ffn_forward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, act: str = "silu",
                      save: bool | torch.dtype = False, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None):
    """``h = act(x w_gate^T) * (x w_up^T)`` for x (..., d) and weights (f, d); not recorded by autograd.

    bfloat16, float16 or float32 throughout; ``act`` is ``"silu"``, ``"gelu"`` or ``"gelu_tanh"``.
    With ``save`` returns ``(h, preact)``, preact being what gated_ffn_backward needs: the
    (tokens, 2 f') pair of pre-activations, f' = f rounded up to a multiple of 8, in float32
    (``save=True``) or in the dtype given: float32 or x's, which takes half the memory and leaves
    16-bit gradients about 1.3 times as far off.  ``save=torch.int8`` keeps an 8-bit checkpoint, a
    quarter of the memory: codes in blocks of 32 features with a step each, as quantize_int8 with
    ``block=32`` makes them, in one int8 tensor (h of up to 64 tokens may then differ in its last bit).
    """
    if stream is not None:  # the call, its temporaries and its outputs belong to it
        with torch.cuda.stream(stream):
            return gated_ffn_forward(x, w_gate, w_up, act, save, out, workspace)
    lib = _load()
    mode = _act_mode(act)
    in8 = save is torch.int8
    code, n, d, f, keep, ins = _ffn_args(x, w_gate, w_up, 0 if in8 else _FEW)
    h = _out("out", out, (*x.shape[:-1], f), x)
    pre = None
    if in8:
        pre = x.new_empty((n, lib.hess_gated_ffn_preact_i8_cols(f)), dtype=torch.int8)
        mode |= _PREACT_I8
    elif save:
        kept = torch.float32 if save is True else save
        if kept not in (torch.float32, x.dtype):
            raise ValueError(f"save must be a bool, torch.float32, torch.int8 or the dtype of x, not {save}")
        pre = x.new_empty((n, 2 * (-(-f // 8) * 8)), dtype=kept)
        if kept == torch.float32:
            mode |= _PREACT_F32
    if n > 0:
        ldh = h.stride(0) if out is not None and h.dim() == 2 and n > 1 else f
        need = lib.hess_gated_ffn_i8_workspace(n, d, f, code) if in8 else lib.hess_gated_ffn_workspace(n, d, f, code, 0)
        wp, wb, work = _workspace(workspace, need, x) if need else (None, 0, None)
        rc = lib.hess_gated_ffn_forward(*ins, code, mode, n, d, f, h.data_ptr(), ldh,
                                        pre.data_ptr() if save else None, wp, wb, _stream(None, x.get_device()))
        if rc != 0:
            _check(rc)
    return (h, pre) if save else h


def gated_ffn_backward(dh: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                       preact: torch.Tensor, act: str = "silu", need_x: bool = True, need_w: bool = True,
                       workspace: torch.Tensor | None = None, stream=None):
    """``(dx, dw_gate, dw_up)`` for the gradient dh of gated_ffn_forward's h (entries not needed are None).

    Sums are float32.  For 16-bit types the gradients of the two pre-activations are rounded to that type
    before the products, which leaves the results about 1.4 times as far off as their own last rounding;
    float32 inputs have no such rounding.  ``preact`` from ``save=torch.int8`` gives the derivatives at
    what its codes stand for.  ``x`` may be an 8-bit checkpoint too (quantize_int8 with ``block=32``), which
    dw_gate and dw_up then take, or None where they are not needed.
    """
    if stream is not None:  # the call, its temporaries and its outputs belong to it
        with torch.cuda.stream(stream):
            return gated_ffn_backward(dh, x, w_gate, w_up, preact, act, need_x, need_w, workspace)
    lib = _load()
    mode = _act_mode(act)
    x8 = None
    if isinstance(x, Int8Rows) or x is None:
        if need_w and x is None:
            raise ValueError("dw_gate and dw_up need x")
        code, f, d, keep, (gp, ldg, up, ldu) = _ffn_weights(dh, w_gate, w_up, "dh")
        lead = dh.shape[:-1]
        xp, ldx, n = None, d, lead.numel()
        if dh.dim() < 1 or dh.shape[-1] != f:
            raise ValueError(f"dh must be (..., {f})")
        if x is not None:
            keep_x, lead_x, _, dx8, xp, ldx, x8 = _int8_args("x", x, 32)
            if lead_x != lead or dx8 != d:
                raise ValueError(f"x must hold {(*lead, d)} codes, not {tuple(x.codes.shape)}")
        x = dh
    else:
        code, n, d, f, keep, (xp, ldx, gp, ldg, up, ldu) = _ffn_args(x, w_gate, w_up)
        lead = x.shape[:-1]
        if tuple(dh.shape) != (*lead, f) or dh.dtype != x.dtype or dh.device != x.device:
            raise ValueError(f"dh must be a {x.dtype} {(*lead, f)} tensor on {x.device}")
    in8 = preact.dtype == torch.int8
    cols = lib.hess_gated_ffn_preact_i8_cols(f) if in8 else 2 * (-(-f // 8) * 8)
    if tuple(preact.shape) != (n, cols) or not (in8 or preact.dtype in (torch.float32, x.dtype)) \
            or preact.device != x.device or not preact.is_contiguous():
        raise ValueError(f"preact must be the contiguous ({n}, {cols}) tensor gated_ffn_forward saved")
    if in8:
        mode |= _PREACT_I8
    elif preact.dtype == torch.float32:
        mode |= _PREACT_F32
    dh2, dhp, lddh = _rows(dh.reshape(-1, f) if dh.dim() != 2 else dh)
    dx = x.new_empty((*lead, d)) if need_x else None
    dwg = x.new_empty((f, d)) if need_w else None
    dwu = x.new_empty((f, d)) if need_w else None
    wp, wb, work = _workspace(workspace, lib.hess_gated_ffn_workspace(n, d, f, code, 1 if x8 is None else 3), x)
    rest = (gp, ldg, up, ldu, preact.data_ptr() if n > 0 else None, code, mode, n, d, f,
            dx.data_ptr() if need_x and n > 0 else None, d, dwg.data_ptr() if need_w else None, d,
            dwu.data_ptr() if need_w else None, d, wp, wb, _stream(None, x.get_device()))
    if x8 is None:
        rc = lib.hess_gated_ffn_backward(dhp if n > 0 else None, lddh, xp if n > 0 else None, ldx, *rest)
    else:
        rc = lib.hess_gated_ffn_backward_x8(dhp if n > 0 else None, lddh, xp if n > 0 else None, ldx,
                                            x8 if n > 0 else None, *rest)
    if rc != 0:
        _check(rc)
    return dx, dwg, dwu


def _refuse_forward_mode(name: str, *tensors) -> None:
    """A dual tensor does not require a gradient: without this its tangent would be dropped in silence."""
    if _forward_ad._current_level < 0:
        return
    for t in tensors:
        if t is not None and _forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError(f"{name} has no forward-mode derivative")


class _GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, act, save):
        h, preact = gated_ffn_forward(x, w_gate, w_up, act=act, save=save)
        ctx.act, ctx.block = act, None
        if save is torch.int8:
            need = ctx.needs_input_grad
            kept = quantize_int8(x, block=32) if need[1] or need[2] else Int8Rows(None, None, 32)
            ctx.block = 32
            ctx.save_for_backward(kept.codes, w_gate, w_up, preact, kept.scale)
        else:
            ctx.save_for_backward(x, w_gate, w_up, preact)
        return h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh):
        x, w_gate, w_up, preact, *scale = ctx.saved_tensors
        need = ctx.needs_input_grad
        if ctx.block is not None and x is not None:
            x = Int8Rows(x, scale[0], ctx.block)
        dx, dwg, dwu = gated_ffn_backward(dh, x, w_gate, w_up, preact, act=ctx.act, need_x=need[0],
                                          need_w=need[1] or need[2])
        return dx, (dwg if need[1] else None), (dwu if need[2] else None), None, None


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, act: str = "silu",
              save: bool | torch.dtype = True) -> torch.Tensor:
    """gated_ffn_forward under autograd: the backward pass is gated_ffn_backward (once differentiable).

    ``save``: in which type the pre-activations are kept for it, as for gated_ffn_forward; with torch.int8
    x is kept in 8 bits too (in blocks of 32 columns), and not at all where no weight needs a gradient:
    the gradients are those at the values so held.  Reverse mode only: dual tensors of forward mode raise
    NotImplementedError.
    """
    _refuse_forward_mode("gated_ffn", x, w_gate, w_up)
    if torch.is_grad_enabled() and (x.requires_grad or w_gate.requires_grad or w_up.requires_grad):
        return _GatedFfn.apply(x, w_gate, w_up, act, save or True)
    return gated_ffn_forward(x, w_gate, w_up, act=act)


# -- distillation from a teacher's top logits -----------------------------------------------------

def _distill_args(logits, ids, values, weight, temperature):
    """(tensors to keep, leading shape, n, vocab, code, arguments for the library)."""
    code = _float_code("logits", logits)
    shape, short = logits.shape, ids.shape
    if len(shape) < 1:
        raise ValueError("logits must be (..., vocab)")
    lead, vocab = shape[:-1], shape[-1]
    if len(short) < 1 or short != values.shape or short[:-1] != lead:
        raise ValueError("ids and values must be (..., k) with the leading dimensions of logits")
    if ids.dtype == torch.int64:
        ids64 = 1
    elif ids.dtype == torch.int32:
        ids64 = 0
    else:
        raise TypeError("ids must be int32 or int64")
    index = logits.get_device()
    vcode = _CODES.get(values.dtype)
    if vcode is None or values.get_device() != index:
        vcode = _float_code("values", values)
    if ids.get_device() != index:
        raise ValueError("ids must be on the device of logits")
    k = short[-1]
    if len(shape) != 2:
        logits, ids, values = logits.reshape(-1, vocab), ids.reshape(-1, k), values.reshape(-1, k)
    z2, zp, ldz = _rows(logits)
    i2, ip, ldi = _rows(ids)
    v2, vp, ldv = _rows(values)
    n = z2.shape[0]
    w = _row_floats("weight", weight, lead, logits) if weight is not None else None
    return (z2, i2, v2, w), lead, n, vocab, code, (zp, ldz, code, n, vocab, ip, ids64, ldi, vp, vcode, ldv, k,
                                                   w.data_ptr() if w is not None else None, float(temperature))


def _row_floats(name, t, lead, like):
    """A float32 value for each row, contiguous (a broadcast one is written out)."""
    if t.shape != lead or t.dtype != torch.float32 or t.get_device() != like.get_device():
        raise ValueError(f"{name} must be a float32 {tuple(lead)} tensor on {like.device}")
    return t if t.is_contiguous() else t.contiguous()


def _grad_out(out, logits):
    if out is None:
        # contiguous whatever the strides of logits
        return torch.empty_like(logits, memory_format=torch.contiguous_format), logits.shape[-1]
    grad = _out("out", out, logits.shape, logits)
    return grad, (grad.stride(0) if grad.dim() == 2 and grad.shape[0] > 1 else logits.shape[-1])


def _distill_call(logits, ids, values, weight, temperature, want_stats, want_grad, out, workspace):
    lib = _load()
    keep, lead, n, vocab, code, args = _distill_args(logits, ids, values, weight, temperature)
    w = keep[3]
    loss = torch.empty_like(w) if w is not None else logits.new_empty(lead, dtype=torch.float32)
    stats = logits.new_empty((*lead, 2), dtype=torch.float32) if want_stats else None
    grad, ldg = _grad_out(out, logits) if want_grad else (None, 0)
    need = lib.hess_distill_topk_workspace(n, vocab, code)
    wp, wb, work = _workspace(workspace, need, logits) if need else (None, 0, None)
    rc = lib.hess_distill_topk(*args, loss.data_ptr(), stats.data_ptr() if want_stats else None,
                               grad.data_ptr() if want_grad else None, ldg, wp, wb,
                               _stream(None, logits.get_device()))
    if rc != 0:
        _check(rc)
    return loss, stats, grad


def distill_topk_forward(logits: torch.Tensor, ids: torch.Tensor, values: torch.Tensor,
                         weight: torch.Tensor | None = None, temperature: float = 1.0,
                         workspace: torch.Tensor | None = None, stream=None):
    """``(loss, stats)``: each row's divergence from the teacher's top entries, and what the backward pass needs.

    logits (..., vocab) bfloat16, float16 or float32; ids (..., k) int32 or int64 (negative: absent);
    values (..., k) the teacher's logits there; weight (...) float32, 0 for rows to leave out.  loss (...)
    and stats (..., 2), the largest logit and the sum of exp((logits - largest) / temperature), are float32.
    """
    if stream is not None:  # the call, its temporaries and its outputs belong to it
        with torch.cuda.stream(stream):
            return distill_topk_forward(logits, ids, values, weight, temperature, workspace)
    return _distill_call(logits, ids, values, weight, temperature, True, False, None, workspace)[:2]


def distill_topk_step(logits: torch.Tensor, ids: torch.Tensor, values: torch.Tensor,
                      weight: torch.Tensor | None = None, temperature: float = 1.0, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None):
    """``(loss, dlogits)`` in one call: each row's loss and the gradient of their sum (``out`` may be logits)."""
    if stream is not None:  # the call, its temporaries and its outputs belong to it
        with torch.cuda.stream(stream):
            return distill_topk_step(logits, ids, values, weight, temperature, out, workspace)
    loss, _, grad = _distill_call(logits, ids, values, weight, temperature, False, True, out, workspace)
    return loss, grad


def distill_topk_backward(dloss: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, values: torch.Tensor,
                          stats: torch.Tensor, weight: torch.Tensor | None = None, temperature: float = 1.0,
                          out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dlogits for the gradient dloss of distill_topk_forward's loss (``out`` may be logits)."""
    if stream is not None:  # the call, its temporaries and its outputs belong to it
        with torch.cuda.stream(stream):
            return distill_topk_backward(dloss, logits, ids, values, stats, weight, temperature, out)
    lib = _load()
    keep, lead, n, vocab, code, args = _distill_args(logits, ids, values, weight, temperature)
    dl = _row_floats("dloss", dloss, lead, logits)
    if tuple(stats.shape) != (*lead, 2) or stats.dtype != torch.float32 or stats.device != logits.device \
            or not stats.is_contiguous():
        raise ValueError(f"stats must be the contiguous float32 {(*lead, 2)} tensor distill_topk_forward returned")
    grad, ldg = _grad_out(out, logits)
    rc = lib.hess_distill_topk_backward(dl.data_ptr(), *args, stats.data_ptr(), grad.data_ptr(), ldg,
                                        _stream(None, logits.get_device()))
    if rc != 0:
        _check(rc)
    return grad


class _DistillTopk(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, values, weight, temperature):
        loss, stats = distill_topk_forward(logits, ids, values, weight=weight, temperature=temperature)
        ctx.save_for_backward(logits, ids, values, weight, stats)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss):
        logits, ids, values, weight, stats = ctx.saved_tensors
        return distill_topk_backward(dloss, logits, ids, values, stats, weight=weight,
                                     temperature=ctx.temperature), None, None, None, None


def distill_topk(logits: torch.Tensor, ids: torch.Tensor, values: torch.Tensor, weight: torch.Tensor | None = None,
                 temperature: float = 1.0) -> torch.Tensor:
    """Each row's loss under autograd (gradient for logits only, once differentiable).

    ``values`` and ``weight`` are constants of the loss: an error is raised if they require a gradient.
    Reverse mode only: dual tensors of forward mode raise NotImplementedError.
    """
    _refuse_forward_mode("distill_topk", logits, values, weight)
    if torch.is_grad_enabled():
        if values.requires_grad or (weight is not None and weight.requires_grad):
            raise ValueError("values and weight are constants of the loss: detach them")
        if logits.requires_grad:
            return _DistillTopk.apply(logits, ids, values, weight, float(temperature))
    return distill_topk_forward(logits, ids, values, weight=weight, temperature=temperature)[0]


# -- 8-bit integers: rows as codes with scales, their product, a linear layer ---------------------

# powers of two by their exponent byte, as the library's block 32 has them (None: a torch without the type, where
# blocks of 32 are refused and all else runs)
_E8 = getattr(torch, "float8_e8m0fnu", None)


def _check_block(name: str, block: int) -> None:
    if block != 0 and block != 32:
        raise ValueError(f"{name} must be 0 or 32, not {block}")
    if block != 0 and _E8 is None:
        raise RuntimeError("blocks of 32 columns need a torch with float8_e8m0fnu")


class Int8Rows(NamedTuple):
    """Rows held as int8 ``codes`` (..., d) with their ``scale``: float32 (...) for ``block`` 0 (one a row),
    or for ``block`` 32 powers of two, torch.float8_e8m0fnu (..., ceil(d / 32)), for each 32 columns."""

    codes: torch.Tensor
    scale: torch.Tensor
    block: int = 0


def _int8_args(name: str, rows: Int8Rows, block=None, tokens=0):
    """(tensors to keep, leading shape, n, d, code pointer, row stride, scale pointer) of checked rows.

    tokens: rows of the left operand of the product that takes these (0: none does).  Past the few whose
    kernels take codes of any alignment, rows that do not start where its tiles need it are copied."""
    codes, scale, b = rows
    index = codes.get_device()
    if index < 0:
        raise ValueError(f"{name} must be on the GPU")
    if index != _current_device():
        raise ValueError(f"{name} is on {codes.device}, not on the current device")
    if codes.dtype != torch.int8:
        raise TypeError(f"codes of {name} must be int8, not {codes.dtype}")
    if b != 0:
        _check_block(f"block of {name}", b)
    if block is not None and b != block:
        raise ValueError(f"{name} must have " + ("a scale a row (block 0)" if block == 0 else "blocks of 32 columns"))
    shape = codes.shape
    if len(shape) < 1:
        raise ValueError(f"codes of {name} must be (..., d)")
    lead, d = shape[:-1], shape[-1]
    if scale.dtype != (torch.float32 if b == 0 else _E8) or scale.get_device() != index \
            or scale.shape != (lead if b == 0 else (*lead, -(-d // 32))):
        raise ValueError(f"scale of {name} must be a {'float32' if b == 0 else 'float8_e8m0fnu'} "
                         f"{tuple(lead) if b == 0 else (*lead, -(-d // 32))} tensor on {codes.device}")
    if not scale.is_contiguous():
        scale = scale.contiguous()
    tiles = tokens > 32 and (tokens > 64 or d >= 8192)  # as the library chooses
    c2, cp, ldc = _rows(codes if len(shape) == 2 else codes.reshape(-1, d), 16 if tiles and d % 16 == 0 else 1)
    n = c2.shape[0]
    if tiles and d % 16 != 0 and cp % 16 == 0 and ldc % 16 == 0 and n > 0 \
            and c2.storage_offset() + (n - 1) * ldc + (d + 15) // 16 * 16 > c2.untyped_storage().nbytes():
        # the tiles read such rows where they are, in whole pieces of 16 bytes: the last one's must be there
        c2 = c2.clone(memory_format=torch.contiguous_format)
        cp, ldc = c2.data_ptr(), d
    return (c2, scale), lead, n, d, cp, ldc, scale.data_ptr()


def _new_codes(shape, n: int, d: int, like: torch.Tensor):
    """(codes, row stride): int8 of a shape of n rows of d, rows of a multiple of 16 bytes apart."""
    pad = -(-d // 16) * 16
    if pad == d:
        return like.new_empty(shape, dtype=torch.int8), pad
    codes = like.new_empty((n, pad), dtype=torch.int8)
    if len(shape) == 2:
        return codes.as_strided((n, d), (pad, 1)), pad
    return codes.view(*shape[:-1], pad)[..., :d], pad


def quantize_int8(x: torch.Tensor, block: int = 0, stream=None) -> Int8Rows:
    """x (..., d) bfloat16, float16 or float32 as 8-bit codes; not recorded by autograd.

    ``block=0``: a scale a row, max |x| / 127, and codes rint(127 x / max |x|): the operands of
    int8_matmul, tokens or a weight's output channels.  ``block=32``: a power of two for each 32
    columns, s with 64 <= max |x| / s < 128: checkpoints of activations (33 / 32 bytes a value; half a
    step off, at most 1 / 128 of the block's largest magnitude, and less than a step past 127.5 of them).
    A row (block) with an infinity or NaN stands for NaN.
    """
    if stream is not None:  # the call, its temporaries and its outputs belong to it
        with torch.cuda.stream(stream):
            return quantize_int8(x, block)
    lib = _load()
    if block != 0:
        _check_block("block", block)
    code = _float_code("x", x)
    shape = x.shape
    d = shape[-1] if len(shape) > 0 else 0
    if d < 1:
        raise ValueError("x must be (..., d) with d >= 1")
    x2, xp, ldx = _rows(x if len(shape) == 2 else x.reshape(-1, d))
    n = x2.shape[0]
    codes, pad = _new_codes(shape, n, d, x)
    if block != 0:
        scale = x.new_empty((*shape[:-1], -(-d // 32)), dtype=_E8)
    else:
        scale = x.new_empty(n if len(shape) == 2 else shape[:-1], dtype=torch.float32)
    rc = lib.hess_int8_quantize(xp, ldx, code, n, d, block, codes.data_ptr(), pad, pad, scale.data_ptr(),
                                _stream(None, x.get_device()))
    if rc != 0:
        _check(rc)
    return Int8Rows(codes, scale, block)


def dequantize_int8(rows: Int8Rows, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """What the codes stand for, rounded once to ``dtype`` (exact in bfloat16 and float32 for block 32)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return dequantize_int8(rows, dtype, out)
    lib = _load()
    keep, lead, n, d, cp, ldc, sp = _int8_args("rows", rows)
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}; use torch.bfloat16, torch.float16 or torch.float32")
    ldx = d
    if out is None:
        x = keep[0].new_empty((n, d) if len(lead) == 1 else (*lead, d), dtype=dtype)
    else:
        x = _out("out", out, (*lead, d), keep[0].new_empty(0, dtype=dtype))
        ldx = x.stride(0) if x.dim() == 2 and n > 1 else d
    rc = lib.hess_int8_dequantize(cp, ldc, sp, n, d, rows.block, x.data_ptr(), ldx, code,
                                  _stream(None, x.get_device()))
    if rc != 0:
        _check(rc)
    return x


def int8_matmul(a: Int8Rows, b: Int8Rows, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``y = a b^T`` (..., f) of dtype for rows of codes a (..., d) and b (f, d) with a scale a row.

    Sums are int32 and exact (d < 2^17); not recorded by autograd.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return int8_matmul(a, b, dtype, out, workspace)
    lib = _load()
    keep, lead, n, d, ap, lda, asp = _int8_args("a", a, 0, a.codes.shape[:-1].numel())
    keep_b, lead_b, f, db, bp, ldb, bsp = _int8_args("b", b, 0, n)
    if len(lead_b) != 1 or db != d:
        raise ValueError(f"b must hold (f, {d}) codes, not {tuple(b.codes.shape)}")
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}; use torch.bfloat16, torch.float16 or torch.float32")
    like = keep[0].new_empty(0, dtype=dtype)
    y = _out("out", out, (*lead, f), like)
    ldy = y.stride(0) if out is not None and y.dim() == 2 and n > 1 else f
    wp, wb, work = _workspace(workspace, lib.hess_int8_matmul_workspace(n, d, f), like)
    rc = lib.hess_int8_matmul(ap, lda, asp, bp, ldb, bsp, n, d, f, y.data_ptr(), ldy, code, wp, wb,
                              _stream(None, like.get_device()))
    if rc != 0:
        _check(rc)
    return y


def int8_linear_forward(x: torch.Tensor, w: Int8Rows, save: bool = False, out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None):
    """``y = xq w^T`` (..., f) of x's dtype: x (..., d) as quantize_int8 holds its rows, times weights held as codes
    (f, d) with a scale for each output channel; not recorded by autograd.

    ``w``: quantize_int8 of a float weight, or what gptq_quantize left with whole rows
    (``Int8Rows((codes.to(torch.int8) - 8), scales[:, 0])``).  With ``save`` returns ``(y, xq)``, the 8-bit
    checkpoint that int8_linear_backward takes.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return int8_linear_forward(x, w, save, out, workspace)
    lib = _load()
    code = _float_code("x", x)
    lead = x.shape[:-1]
    keep, lead_w, f, d, wp8, ldw, wsp = _int8_args("w", w, 0, lead.numel())
    if len(lead_w) != 1 or x.dim() < 1 or x.shape[-1] != d:
        raise ValueError(f"w must hold (f, d) codes and x be (..., d), not {tuple(w.codes.shape)} and {tuple(x.shape)}")
    x2, xp, ldx = _rows(x if len(lead) == 1 else x.reshape(-1, d))
    n = x2.shape[0]
    ldy = f
    if out is None:
        y = x.new_empty((n, f) if len(lead) == 1 else (*lead, f))
    else:
        y = _out("out", out, (*lead, f), x)
        ldy = y.stride(0) if y.dim() == 2 and n > 1 else f
    codes = scale = None
    ldc = 0
    if save:
        codes, ldc = _new_codes(x.shape, n, d, x)
        scale = x.new_empty(n if len(lead) == 1 else lead, dtype=torch.float32)
    need = lib.hess_int8_linear_workspace(n, d, f, code, 4 if save else 0)
    wp, wb, work = _workspace(workspace, need, x) if need else (None, 0, None)
    rc = lib.hess_int8_linear_forward(xp, ldx, code, wp8, ldw, wsp, n, d, f, y.data_ptr(), ldy,
                                      codes.data_ptr() if save and n > 0 else None, ldc,
                                      scale.data_ptr() if save and n > 0 else None, wp, wb,
                                      _stream(None, x.get_device()))
    if rc != 0:
        _check(rc)
    return (y, Int8Rows(codes, scale)) if save else y


def int8_linear_backward(dy: torch.Tensor, x: Int8Rows | None, w: Int8Rows | None, need_x: bool = True,
                         need_w: bool = True, workspace: torch.Tensor | None = None, stream=None):
    """``(dx, dw)`` for the gradient dy (..., f) of int8_linear_forward's y, straight through the rounding:
    dx = dy wq, dw = dy^T xq (entries not needed are None), of dy's dtype.

    ``x``: the checkpoint that the forward call saved (None if dw is not needed); ``w``: its weights (None
    if dx is not needed).  For 16-bit types xq and wq are rounded to that type before the products, which
    leaves the results about 1.4 times as far off as their own last rounding (without it the products
    would double; float32 has none); sums are float32.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return int8_linear_backward(dy, x, w, need_x, need_w, workspace)
    lib = _load()
    code = _float_code("dy", dy)
    if dy.dim() < 1 or (need_x and w is None) or (need_w and x is None):
        raise ValueError("dy must be (..., f); dx needs w and dw needs x")
    if x is None and w is None:
        return None, None
    lead, f = dy.shape[:-1], dy.shape[-1]
    d = (w if x is None else x).codes.shape[-1]
    cp = ldc = sp = wp8 = ldw = wsp = None
    if need_w:
        keep_x, lead_x, _, dx_, cp, ldc, sp = _int8_args("x", x, 0)
        if lead_x != lead or dx_ != d:
            raise ValueError(f"x must hold {(*lead, d)} codes, not {tuple(x.codes.shape)}")
    if need_x:
        keep_w, lead_w, fw, dw_, wp8, ldw, wsp = _int8_args("w", w, 0)
        if len(lead_w) != 1 or fw != f or dw_ != d:
            raise ValueError(f"w must hold {(f, d)} codes, not {tuple(w.codes.shape)}")
    if not need_x and not need_w:
        return None, None
    step = 4 if code == HESS_F32 else 8
    dy2, dyp, lddy = _rows(dy if len(lead) == 1 else dy.reshape(-1, f), step if f % step == 0 else 1)
    n = dy2.shape[0]
    dx = dy.new_empty((*lead, d)) if need_x else None
    dw = dy.new_empty((f, d)) if need_w else None
    need = lib.hess_int8_linear_workspace(n, d, f, code, (1 if need_x else 0) + (2 if need_w else 0))
    wp, wb, work = _workspace(workspace, need, dy)
    rc = lib.hess_int8_linear_backward(dyp, lddy, code, cp, ldc or 0, sp, wp8, ldw or 0, wsp, n, d, f,
                                       dx.data_ptr() if need_x and n > 0 else None, d,
                                       dw.data_ptr() if need_w else None, d, wp, wb, _stream(None, dy.get_device()))
    if rc != 0:
        _check(rc)
    return dx, dw


class _Int8Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, codes, scale):
        w = Int8Rows(codes, scale) if weight is None else quantize_int8(weight)
        need = ctx.needs_input_grad
        y, kept = int8_linear_forward(x, w, save=True) if need[1] else (int8_linear_forward(x, w), Int8Rows(None, None))
        # (each side only where a gradient will read it)
        ctx.save_for_backward(kept.codes, kept.scale, *((w.codes, w.scale) if need[0] else (None, None)))
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        xc, xs, wc, ws = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw = int8_linear_backward(dy, Int8Rows(xc, xs) if need[1] else None, Int8Rows(wc, ws) if need[0] else None,
                                      need_x=need[0], need_w=need[1])
        return dx, dw, None, None


def int8_linear(x: torch.Tensor, w: torch.Tensor | Int8Rows) -> torch.Tensor:
    """A linear layer that computes in 8-bit integers, under autograd: int8_linear_forward and int8_linear_backward.

    ``w``: Int8Rows, weights already quantized, which take no gradient; or a float (f, d) tensor of x's dtype,
    quantized by output channel in every call, with a gradient straight through the rounding.  What is kept for
    the backward pass is in 8 bits.  Once differentiable, reverse mode only.
    """
    if isinstance(w, Int8Rows):
        _refuse_forward_mode("int8_linear", x, w.scale)
        if w.scale.requires_grad:
            raise ValueError("the scales are constants of the layer: detach them")
        if torch.is_grad_enabled() and x.requires_grad:
            return _Int8Linear.apply(x, None, w.codes, w.scale)
        return int8_linear_forward(x, w)
    _refuse_forward_mode("int8_linear", x, w)
    if w.dim() != 2 or w.dtype != x.dtype or w.get_device() != x.get_device():
        raise ValueError("w must be Int8Rows, or an (f, d) tensor of x's dtype and device")
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad):
        return _Int8Linear.apply(x, w, None, None)
    return int8_linear_forward(x, quantize_int8(w))
