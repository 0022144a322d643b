"""ctypes binding of libditattn.so (include/dit_attn.h).

Argument marshalling only (for the training operators, windowed attention and
the paged cache, whose small calls would be mostly marshalling, in the CPython
extension csrc/py_calls.cpp, loaded at the first of them): tensors are passed as device pointers with their
element strides and the current CUDA stream; every step of the computation
runs in the library's kernels.  PyTorch supplies device memory and streams.
There is no fallback: if the library is missing or a call fails, an exception
is raised.  No call is part of an autograd graph: results carry no gradient
function, and gradients are what the *_bwd calls (rope: inverse) return.

With the environment variable DIT_ATTN_DEBUG=1 at import, the binding loads
the debug library instead (libditattn_debug.so: the same kernels with
in-kernel bounds checks, include/dit_attn_debug.h); load_debug_library()
gives a handle to it beside the product library.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import build as _build
from .build import DEBUG_LIB as _DEBUG_LIB_PATH
from .build import LIB as _PRODUCT_LIB_PATH

is_debug_library = os.environ.get("DIT_ATTN_DEBUG", "") == "1"
_LIB_PATH = _DEBUG_LIB_PATH if is_debug_library else _PRODUCT_LIB_PATH
library_path = _LIB_PATH

if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"{os.path.basename(_LIB_PATH)} not found at {_LIB_PATH}; build it first with "
        "`python -m dit_long_sequence_gb300.build` (or __graft_entry__.build())")

DIT_OK, DIT_ERR_INVALID_ARG, DIT_ERR_UNSUPPORTED, DIT_ERR_ALIGNMENT, DIT_ERR_CUDA, DIT_ERR_TIMEOUT, DIT_ERR_BOUNDS = \
    range(7)
DIT_BF16, DIT_F32 = 0, 1
DIT_FAULT_NONE, DIT_FAULT_SKIP_LOAD, DIT_FAULT_SKIP_S_COMMIT, DIT_FAULT_SKIP_P_ARRIVE = range(4)


class Strides4(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("n", ctypes.c_int64), ("h", ctypes.c_int64), ("d", ctypes.c_int64)]


class AttnStrides(ctypes.Structure):
    _fields_ = [("q", Strides4), ("k", Strides4), ("v", Strides4), ("o", Strides4)]


class AttnBwdStrides(ctypes.Structure):
    _fields_ = [(n, Strides4) for n in ("q", "k", "v", "o", "dout", "dq", "dk", "dv")]


class Window(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("left", "right", "sinks", "frame")]


class PagedCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_strides", Strides4), ("v_strides", Strides4), ("pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("table_width", ctypes.c_int),
                ("kv_lens", ctypes.c_void_p)]


DIT_ROPE_INTERLEAVED, DIT_ROPE_HALF = 0, 1
_ROPE_LAYOUTS = {"interleaved": DIT_ROPE_INTERLEAVED, "half": DIT_ROPE_HALF}
_ROPE_SCALINGS = {None: 0, "linear": 1, "base": 2, "by_parts": 3}
_vp, _i, _i64, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float


def _declare(lib):
    """Argument and result types of the C ABI on a loaded library handle."""
    lib.dit_attn_fwd.restype = _i
    lib.dit_attn_fwd.argtypes = [_vp, _vp, _vp, ctypes.POINTER(AttnStrides), _i, _i, _i, _i, _i, _i, _f,
                                  _vp, _i, _vp, _vp]
    lib.dit_attn_fwd_ws.restype = _i
    lib.dit_attn_fwd_ws.argtypes = [_vp, _vp, _vp, ctypes.POINTER(AttnStrides), _i, _i, _i, _i, _i, _i, _f,
                                     _vp, _i, _vp, _vp, ctypes.c_size_t, _vp]
    lib.dit_attn_fwd_workspace_bytes.restype = ctypes.c_size_t
    lib.dit_attn_fwd_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
    lib.dit_attn_fwd_accumulate.restype = _i
    lib.dit_attn_fwd_accumulate.argtypes = [_vp, _vp, _vp, ctypes.POINTER(AttnStrides), _i, _i, _i, _i, _i, _i, _f,
                                             _vp, _vp, _vp]
    lib.dit_attn_fwd_masked.restype = _i
    lib.dit_attn_fwd_masked.argtypes = [_vp, _vp, _vp, ctypes.POINTER(AttnStrides), _i, _i, _i, _i, _i, _i, _vp, _i64,
                                         _i64, _i, _f, _vp, _i, _vp, _vp, ctypes.c_size_t, _vp]
    lib.dit_attn_fwd_masked_noalloc.restype = _i
    lib.dit_attn_fwd_masked_noalloc.argtypes = [_vp, _vp, _vp, ctypes.POINTER(AttnStrides), _i, _i, _i, _i, _i, _i, _vp,
                                                 _i64, _i64, _i, _f, _vp, _i, _vp, _vp]
    lib.dit_attn_masked_workspace_bytes.restype = ctypes.c_size_t
    lib.dit_attn_masked_workspace_bytes.argtypes = [_i, _i, _i]
    lib.dit_attn_masked_split_workspace_bytes.restype = ctypes.c_size_t
    lib.dit_attn_masked_split_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
    lib.dit_attn_fwd_fp8.restype = _i
    lib.dit_attn_fwd_fp8.argtypes = [_vp, _vp, _vp, ctypes.POINTER(AttnStrides), _i, _i, _i, _i, _i, _i, _f, _f, _f, _f,
                                      _vp, _i, _vp, _vp]
    lib.dit_attn_fwd_fp8_ws.restype = _i
    lib.dit_attn_fwd_fp8_ws.argtypes = [_vp, _vp, _vp, ctypes.POINTER(AttnStrides), _i, _i, _i, _i, _i, _i, _f, _f, _f,
                                         _f, _vp, _i, _vp, _vp, ctypes.c_size_t, _vp]
    lib.dit_qkv_cast_fp8.restype = _i
    lib.dit_qkv_cast_fp8.argtypes = [_vp, _i64, _i64, _i, _i, _i, _i, _f, _f, _f, _vp, _vp]
    lib.dit_qkv_norm_rope_to_head_major.restype = _i
    lib.dit_qkv_norm_rope_to_head_major.argtypes = [_vp, _i64, _i64, _i, _i, _i, _i, _vp, _vp, _f, _vp, _vp, _vp, _vp,
                                                     _vp, _vp]
    lib.dit_watchdog_selftest.restype = _i
    lib.dit_watchdog_selftest.argtypes = [ctypes.c_uint32, _vp]
    lib.dit_attn_lse_merge.restype = _i
    lib.dit_attn_lse_merge.argtypes = [_vp, _i64, _i64, _vp, _i64, _i, _i, _i, _i, _i, _vp, _i, _vp, _vp]
    lib.dit_qkv_to_head_major.restype = _i
    lib.dit_qkv_to_head_major.argtypes = [_vp, _i64, _i64, _i, _i, _i, _i, _vp, _vp, _vp, _vp]
    _d, _sz, _st = ctypes.c_double, ctypes.c_size_t, ctypes.POINTER(Strides4)
    lib.dit_attn_bwd.restype = _i
    lib.dit_attn_bwd.argtypes = [_vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                                 _i, _i, _f, _vp, _vp, _vp, _i, _vp, _sz, _vp]
    lib.dit_attn_bwd_masked.restype = _i
    lib.dit_attn_bwd_masked.argtypes = [_vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i,
                                        _i, _i, _i, _i, _vp, _i64, _i64, _i, _f, _vp, _vp, _vp, _i, _vp, _sz, _vp]
    lib.dit_attn_bwd_workspace_bytes.restype = _sz
    lib.dit_attn_bwd_workspace_bytes.argtypes = [_i] * 7
    _win, _cache = ctypes.POINTER(Window), ctypes.POINTER(PagedCache)
    lib.dit_attn_fwd_window.restype = _i
    lib.dit_attn_fwd_window.argtypes = [_vp, _vp, _vp, ctypes.POINTER(AttnStrides), _i, _i, _i, _i, _i, _i, _i, _win, _i, _f, _vp, _i, _vp,
                                        _vp, _sz, _vp]
    lib.dit_attn_fwd_window_workspace_bytes.restype = _sz
    lib.dit_attn_fwd_window_workspace_bytes.argtypes = [_i] * 6 + [_win, _i]
    lib.dit_attn_bwd_window.restype = _i
    lib.dit_attn_bwd_window.argtypes = [_vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, ctypes.POINTER(AttnBwdStrides), _i, _i, _i, _i, _i, _i, _i,
                                        _win, _i, _f, _vp, _vp, _vp, _i, _vp, _sz, _vp]
    lib.dit_attn_bwd_window_workspace_bytes.restype = _sz
    lib.dit_attn_bwd_window_workspace_bytes.argtypes = [_i] * 7 + [_win, _i]
    lib.dit_paged_append.restype = _i
    lib.dit_paged_append.argtypes = [_vp, _st, _vp, _st, _cache, _vp, _i, _i, _i, _i, _vp]
    lib.dit_attn_fwd_paged.restype = _i
    lib.dit_attn_fwd_paged.argtypes = [_vp, _st, _cache, _vp, _i, _i, _i, _i, _i, _win, _f, _vp, _i, _st, _vp, _vp, _sz, _vp]
    lib.dit_attn_fwd_paged_workspace_bytes.restype = _sz
    lib.dit_attn_fwd_paged_workspace_bytes.argtypes = [_i] * 7 + [_win]
    lib.dit_layer_norm_fwd.restype = _i
    lib.dit_layer_norm_fwd.argtypes = [_vp, _i, _st, _i, _i, _i, _i, _vp, _vp, _i, _f, _i, _vp, _i, _st, _vp, _vp, _vp]
    lib.dit_layer_norm_bwd.restype = _i
    lib.dit_layer_norm_bwd.argtypes = [_vp, _i, _st, _vp, _i, _st, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _st, _vp,
                                       _vp, _vp, _sz, _vp]
    lib.dit_layer_norm_bwd_workspace_bytes.restype = _sz
    lib.dit_layer_norm_bwd_workspace_bytes.argtypes = [_i] * 5
    lib.dit_rope.restype = _i
    lib.dit_rope.argtypes = [_vp, _i, _st, _i, _i, _i, _i, _i, _i, _vp, ctypes.POINTER(_i), _i, _vp, _i64, _i64, _f, _i,
                             _vp, _st, _vp]
    lib.dit_rope_inv_freq.restype = _i
    lib.dit_rope_inv_freq.argtypes = [_i, _d, _i, _d, _d, _d, _d, _vp, ctypes.POINTER(_f)]
    lib.dit_status_string.restype = ctypes.c_char_p
    lib.dit_status_string.argtypes = [_i]
    lib.dit_check_watchdog.restype = _i
    lib.dit_check_watchdog.argtypes = [_vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.dit_version.restype = ctypes.c_uint32
    if hasattr(lib, "dit_debug_configure"):
        lib.dit_debug_configure.restype = _i
        lib.dit_debug_configure.argtypes = [ctypes.c_uint32, _i, _i, ctypes.c_uint32, _i64]
        lib.dit_debug_build.restype = ctypes.c_uint32
    return lib


_lib = _declare(ctypes.CDLL(_LIB_PATH))


def _load_calls():
    """The extension of csrc/py_calls.cpp, calling this library's functions."""
    path = _build.calls_path()
    if not os.path.exists(path):
        raise ImportError(f"the training operators' extension is not at {path}; build it first with "
                          "`python -m dit_long_sequence_gb300.build` (or __graft_entry__.build())")
    loader = importlib.machinery.ExtensionFileLoader("dit_calls", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("dit_calls", loader))
    loader.exec_module(module)

    def addresses(*names):
        return [ctypes.cast(getattr(_lib, name), ctypes.c_void_p).value for name in names]

    module.bind(*addresses(
        "dit_attn_bwd", "dit_attn_bwd_masked", "dit_attn_bwd_workspace_bytes", "dit_layer_norm_fwd",
        "dit_layer_norm_bwd", "dit_layer_norm_bwd_workspace_bytes", "dit_rope"))
    module.bind_streaming(*addresses(
        "dit_attn_fwd_window", "dit_attn_fwd_window_workspace_bytes", "dit_attn_bwd_window", "dit_attn_bwd_window_workspace_bytes",
        "dit_paged_append", "dit_attn_fwd_paged", "dit_attn_fwd_paged_workspace_bytes"))
    return module


class _Calls:
    """The extension's functions, loaded when one is first asked for: the other
    calls do without it (and without what it is built with)."""
    _NAMES = ("attn_bwd", "norm_fwd", "norm_bwd", "rope", "window_fwd", "window_bwd", "append", "paged", "bind")

    def __getattr__(self, name):
        if name not in self._NAMES:
            raise AttributeError(name)
        module = _load_calls()
        for n in self._NAMES:
            setattr(self, n, getattr(module, n))     # found without coming here from now on
        return getattr(module, name)


_calls = _Calls()


def load_calls():
    """Loads the training operators' extension now; ImportError if it is missing."""
    return _calls.bind


def load_debug_library():
    """ctypes handle of libditattn_debug.so with the C ABI declared: every
    dit_attn.h entry point plus dit_debug_configure / dit_debug_build.  Its
    kernels and device status word are its own (check it with its own
    dit_check_watchdog)."""
    if not os.path.exists(_DEBUG_LIB_PATH):
        raise ImportError(f"libditattn_debug.so not found at {_DEBUG_LIB_PATH}; build it first")
    return _declare(ctypes.CDLL(_DEBUG_LIB_PATH))


EXPORTS = ("dit_attn_fwd", "dit_attn_fwd_ws", "dit_attn_fwd_workspace_bytes", "dit_attn_fwd_masked", "dit_attn_fwd_masked_noalloc", "dit_attn_masked_workspace_bytes",
           "dit_attn_masked_split_workspace_bytes",
           "dit_attn_fwd_accumulate", "dit_attn_lse_merge", "dit_qkv_to_head_major",
           "dit_qkv_norm_rope_to_head_major", "dit_qkv_cast_fp8", "dit_attn_fwd_fp8", "dit_attn_fwd_fp8_ws", "dit_status_string",
           "dit_check_watchdog",
           "dit_watchdog_selftest", "dit_version",
           "dit_attn_bwd", "dit_attn_bwd_masked", "dit_attn_bwd_workspace_bytes", "dit_layer_norm_fwd",
           "dit_layer_norm_bwd", "dit_layer_norm_bwd_workspace_bytes", "dit_rope", "dit_rope_inv_freq",
           "dit_attn_fwd_window", "dit_attn_fwd_window_workspace_bytes", "dit_attn_bwd_window", "dit_attn_bwd_window_workspace_bytes",
           "dit_paged_append", "dit_attn_fwd_paged", "dit_attn_fwd_paged_workspace_bytes")


class DitError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_lib.dit_status_string(status).decode()}")


def _check(status: int, where: str):
    if status != DIT_OK:
        raise DitError(status, where)


def raw():
    """The ctypes library handle (for callers that marshal pointers themselves)."""
    return _lib


def _stream_ptr(stream) -> int:
    if stream is None:   # the current device's current stream, without a Stream object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return int(stream.cuda_stream)


def _strides4(t: torch.Tensor) -> Strides4:
    return Strides4(*t.stride())


def _attn_args(q, k, v, key_valid_len, scale, out, lse, out_dtype):
    B, Nq, H, D = q.shape
    Nkv = k.shape[1]
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a bf16 CUDA tensor")
    if k.shape != (B, Nkv, H, D) or v.shape != (B, Nkv, H, D):
        raise ValueError("k and v must be [B, Nkv, H, D] matching q")
    kvl = Nkv if key_valid_len is None else int(key_valid_len)
    sc = float(D) ** -0.5 if scale is None else float(scale)
    if out is None:
        out = torch.empty((B, Nq, H, D), dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if out.dtype not in (torch.float32, torch.bfloat16) or tuple(out.shape) != (B, Nq, H, D):
        raise ValueError("out must be a [B, Nq, H, D] fp32 or bf16 tensor")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, Nq) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, H, Nq] tensor")
    st = AttnStrides(_strides4(q), _strides4(k), _strides4(v), _strides4(out))
    return B, Nq, Nkv, H, D, kvl, sc, out, lse, st


def attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, key_valid_len: int | None = None,
             scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
             out_dtype: torch.dtype = torch.float32, stream=None):
    """O = softmax(scale Q K^T) V and LSE, through `dit_attn_fwd`.

    q [B, Nq, H, D], k/v [B, Nkv, H, D]: bf16 CUDA tensors with any strides whose
    last dimension is contiguous (strided views of a fused QKV buffer work as is).
    Returns (out [B, Nq, H, D] in out_dtype, lse [B, H, Nq] fp32).
    """
    B, Nq, Nkv, H, D, kvl, sc, out, lse, st = _attn_args(q, k, v, key_valid_len, scale, out, lse, out_dtype)
    rc = _lib.dit_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(st), B, Nq, Nkv, H, D, kvl,
                           sc, out.data_ptr(), DIT_F32 if out.dtype == torch.float32 else DIT_BF16,
                           lse.data_ptr(), _stream_ptr(stream))
    _check(rc, "dit_attn_fwd")
    return out, lse


def attn_fwd_workspace_bytes(B: int, Nq: int, H: int, D: int, key_valid_len: int) -> int:
    """Workspace that lets attn_fwd_ws balance the grid's last wave (current device; 0: no split)."""
    return int(_lib.dit_attn_fwd_workspace_bytes(int(B), int(Nq), int(H), int(D), int(key_valid_len)))


def attn_fwd_ws(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, key_valid_len: int | None = None,
                scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                out_dtype: torch.dtype = torch.float32, workspace: torch.Tensor | None = None, stream=None):
    """attn_fwd through `dit_attn_fwd_ws`: the items of the grid's last partial
    wave are split over key ranges and merged.  The workspace (a uint8 CUDA
    tensor of attn_fwd_workspace_bytes) is allocated here unless given."""
    B, Nq, Nkv, H, D, kvl, sc, out, lse, st = _attn_args(q, k, v, key_valid_len, scale, out, lse, out_dtype)
    if workspace is None:
        nbytes = attn_fwd_workspace_bytes(B, Nq, H, D, kvl)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = _lib.dit_attn_fwd_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(st), B, Nq, Nkv, H, D, kvl,
                              sc, out.data_ptr(), DIT_F32 if out.dtype == torch.float32 else DIT_BF16,
                              lse.data_ptr(), ws_ptr, ws_bytes, _stream_ptr(stream))
    _check(rc, "dit_attn_fwd_ws")
    return out, lse


def masked_workspace_bytes(B: int, Nq: int, key_valid_len: int) -> int:
    """Workspace that lets attn_fwd_masked skip key tiles the mask leaves empty."""
    return int(_lib.dit_attn_masked_workspace_bytes(int(B), int(Nq), int(key_valid_len)))


def masked_split_workspace_bytes(B: int, Nq: int, H: int, D: int, key_valid_len: int) -> int:
    """Workspace that lets attn_fwd_masked skip empty key tiles and split the
    grid's last partial wave (current device)."""
    return int(_lib.dit_attn_masked_split_workspace_bytes(int(B), int(Nq), int(H), int(D), int(key_valid_len)))


def attn_fwd_masked(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, mask_bits: torch.Tensor, *,
                    mask_rows: int | None = None, key_valid_len: int | None = None, scale: float | None = None,
                    out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    out_dtype: torch.dtype = torch.float32, workspace: torch.Tensor | None = None,
                    skip_empty_tiles: bool = True, stream=None):
    """Attention with a general bit mask through `dit_attn_fwd_masked`.

    mask_bits: int32 CUDA tensor [B or 1, R, W] of packed bits (bit j&31 of word
    j>>5 of row i: query i may attend key j), W a multiple of 4 with
    W >= 4*ceil(key_valid_len/128); a leading dimension of 1 shares the mask
    across the batch.  Rows i >= mask_rows (default R) attend every valid key.
    With skip_empty_tiles (default) a workspace (allocated here unless given,
    of masked_split_workspace_bytes) lets the kernel skip key tiles the mask
    leaves empty and split the grid's last partial wave over key ranges; a
    given workspace of only masked_workspace_bytes skips without splitting.
    """
    B, Nq, H, D = q.shape
    Nkv = k.shape[1]
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a bf16 CUDA tensor")
    if k.shape != (B, Nkv, H, D) or v.shape != (B, Nkv, H, D):
        raise ValueError("k and v must be [B, Nkv, H, D] matching q")
    if mask_bits.dtype != torch.int32 or mask_bits.dim() != 3 or mask_bits.stride(2) != 1 or not mask_bits.is_cuda:
        raise ValueError("mask_bits must be an int32 CUDA tensor [B or 1, rows, words], words contiguous")
    if mask_bits.shape[0] not in (1, B):
        raise ValueError("mask_bits must have B or 1 batch entries")
    rows = mask_bits.shape[1] if mask_rows is None else int(mask_rows)
    if rows > mask_bits.shape[1]:
        raise ValueError("mask_rows exceeds the mask's rows")
    kvl = Nkv if key_valid_len is None else int(key_valid_len)
    sc = float(D) ** -0.5 if scale is None else float(scale)
    if out is None:
        out = torch.empty((B, Nq, H, D), dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if out.dtype not in (torch.float32, torch.bfloat16) or tuple(out.shape) != (B, Nq, H, D):
        raise ValueError("out must be a [B, Nq, H, D] fp32 or bf16 tensor")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, Nq) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, H, Nq] tensor")
    sb = 0 if mask_bits.shape[0] == 1 else mask_bits.stride(0)
    ws_ptr, ws_bytes = None, 0
    if skip_empty_tiles:
        need = masked_split_workspace_bytes(B, Nq, H, D, kvl)
        if workspace is None and need > 0:
            workspace = torch.empty((need + 15) // 16 * 16, dtype=torch.uint8, device=q.device)
        if workspace is not None:
            ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = AttnStrides(_strides4(q), _strides4(k), _strides4(v), _strides4(out))
    rc = _lib.dit_attn_fwd_masked(q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(st), B, Nq, Nkv, H, D, kvl,
                                  mask_bits.data_ptr(), sb, mask_bits.stride(1), rows, sc, out.data_ptr(),
                                  DIT_F32 if out.dtype == torch.float32 else DIT_BF16, lse.data_ptr(),
                                  ws_ptr, ws_bytes, _stream_ptr(stream))
    _check(rc, "dit_attn_fwd_masked")
    return out, lse


def attn_fwd_masked_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, mask_bits: torch.Tensor, *,
                            mask_rows: int | None = None, key_valid_len: int | None = None,
                            scale: float | None = None, out: torch.Tensor | None = None,
                            lse: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32, stream=None):
    """attn_fwd_masked through `dit_attn_fwd_masked_noalloc`: the tile-occupancy
    scratch is the library's fixed per-device array, no workspace is passed.
    out and lse must be given (or are allocated here by PyTorch, not by the
    library)."""
    B, Nq, H, D = q.shape
    Nkv = k.shape[1]
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a bf16 CUDA tensor")
    if mask_bits.dtype != torch.int32 or mask_bits.dim() != 3 or mask_bits.stride(2) != 1 or not mask_bits.is_cuda:
        raise ValueError("mask_bits must be an int32 CUDA tensor [B or 1, rows, words], words contiguous")
    rows = mask_bits.shape[1] if mask_rows is None else int(mask_rows)
    kvl = Nkv if key_valid_len is None else int(key_valid_len)
    sc = float(D) ** -0.5 if scale is None else float(scale)
    if out is None:
        out = torch.empty((B, Nq, H, D), dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    sb = 0 if mask_bits.shape[0] == 1 else mask_bits.stride(0)
    st = AttnStrides(_strides4(q), _strides4(k), _strides4(v), _strides4(out))
    rc = _lib.dit_attn_fwd_masked_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(st), B, Nq, Nkv, H,
                                          D, kvl, mask_bits.data_ptr(), sb, mask_bits.stride(1), rows, sc,
                                          out.data_ptr(), DIT_F32 if out.dtype == torch.float32 else DIT_BF16,
                                          lse.data_ptr(), _stream_ptr(stream))
    _check(rc, "dit_attn_fwd_masked_noalloc")
    return out, lse


def attn_fwd_accumulate(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor, *,
                        key_valid_len: int | None = None, scale: float | None = None, stream=None):
    """Fold attention of q over this key chunk into the running fp32 (out, lse)
    in place, through `dit_attn_fwd_accumulate`.  Start from lse = -inf."""
    B, Nq, H, D = q.shape
    Nkv = k.shape[1]
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a bf16 CUDA tensor")
    if k.shape != (B, Nkv, H, D) or v.shape != (B, Nkv, H, D):
        raise ValueError("k and v must be [B, Nkv, H, D] matching q")
    if out.dtype != torch.float32 or tuple(out.shape) != (B, Nq, H, D):
        raise ValueError("out must be an fp32 [B, Nq, H, D] tensor")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, Nq) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, H, Nq] tensor")
    kvl = Nkv if key_valid_len is None else int(key_valid_len)
    sc = float(D) ** -0.5 if scale is None else float(scale)
    st = AttnStrides(_strides4(q), _strides4(k), _strides4(v), _strides4(out))
    rc = _lib.dit_attn_fwd_accumulate(q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(st), B, Nq, Nkv, H, D,
                                      kvl, sc, out.data_ptr(), lse.data_ptr(), _stream_ptr(stream))
    _check(rc, "dit_attn_fwd_accumulate")
    return out, lse


def lse_merge(o_parts: torch.Tensor, lse_parts: torch.Tensor, *, out: torch.Tensor | None = None,
              lse_out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32, stream=None):
    """Merge n partials through `dit_attn_lse_merge`.

    o_parts [n, B, Nq, H, D] fp32: any view whose (B, Nq, H) dims collapse to one
    row index with a common row stride and d contiguous -- chunk-major
    (contiguous [n, B, Nq, H, D]) or interleaved (a [B, Nq, H, n, D] buffer seen
    through .permute(3, 0, 1, 2, 4)); lse_parts [n, B, H, Nq] fp32 with every
    chunk contiguous.  Returns (out [B, Nq, H, D], lse_out [B, H, Nq]).
    """
    n, B, Nq, H, D = o_parts.shape
    if o_parts.dtype != torch.float32 or lse_parts.dtype != torch.float32:
        raise TypeError("partials must be fp32")
    if tuple(lse_parts.shape) != (n, B, H, Nq):
        raise ValueError("lse_parts must be [n, B, H, Nq]")
    rs = o_parts.stride(3)
    if o_parts.stride(4) != 1 or o_parts.stride(2) != H * rs or o_parts.stride(1) != Nq * H * rs:
        raise ValueError("o_parts rows must share one stride with d contiguous")
    if not lse_parts[0].is_contiguous():
        raise ValueError("each LSE chunk must be contiguous")
    if out is None:
        out = torch.empty((B, Nq, H, D), dtype=out_dtype, device=o_parts.device)
    if lse_out is None:
        lse_out = torch.empty((B, H, Nq), dtype=torch.float32, device=o_parts.device)
    if not out.is_contiguous() or not lse_out.is_contiguous():
        raise ValueError("outputs must be contiguous")
    rc = _lib.dit_attn_lse_merge(o_parts.data_ptr(), o_parts.stride(0), rs, lse_parts.data_ptr(),
                                 lse_parts.stride(0), n, B, Nq, H, D, out.data_ptr(),
                                 DIT_F32 if out.dtype == torch.float32 else DIT_BF16, lse_out.data_ptr(),
                                 _stream_ptr(stream))
    _check(rc, "dit_attn_lse_merge")
    return out, lse_out


def qkv_to_head_major(qkv: torch.Tensor, *, outs=None, stream=None):
    """Split a fused [B, N, 3, H, D] bf16 buffer (b and n strides free, inner
    [3, H, D] contiguous) into three contiguous [B, H, N, D] tensors."""
    B, N, three, H, D = qkv.shape
    if three != 3 or qkv.dtype != torch.bfloat16:
        raise ValueError("expected a bf16 [B, N, 3, H, D] tensor")
    if qkv.stride(4) != 1 or qkv.stride(3) != D or qkv.stride(2) != H * D:
        raise ValueError("the [3, H, D] block of every sequence row must be contiguous")
    if outs is None:
        outs = tuple(torch.empty((B, H, N, D), dtype=torch.bfloat16, device=qkv.device) for _ in range(3))
    for o in outs:
        if not o.is_contiguous() or tuple(o.shape) != (B, H, N, D):
            raise ValueError("outputs must be contiguous [B, H, N, D]")
    rc = _lib.dit_qkv_to_head_major(qkv.data_ptr(), qkv.stride(0), qkv.stride(1), B, N, H, D,
                                    outs[0].data_ptr(), outs[1].data_ptr(), outs[2].data_ptr(),
                                    _stream_ptr(stream))
    _check(rc, "dit_qkv_to_head_major")
    return outs


def qkv_norm_rope_to_head_major(qkv: torch.Tensor, *, q_weight: torch.Tensor | None = None,
                                k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                                rope_cos: torch.Tensor | None = None, rope_sin: torch.Tensor | None = None,
                                outs=None, stream=None):
    """dit_qkv_to_head_major with Q/K RMSNorm (fp32 [D] weights; None skips)
    and RoPE on consecutive pairs (fp32 [N, D/2] cos/sin tables; None skips)
    fused in, through `dit_qkv_norm_rope_to_head_major`."""
    B, N, three, H, D = qkv.shape
    if three != 3 or qkv.dtype != torch.bfloat16 or not qkv.is_cuda:
        raise ValueError("expected a bf16 CUDA [B, N, 3, H, D] tensor")
    if qkv.stride(4) != 1 or qkv.stride(3) != D or qkv.stride(2) != H * D:
        raise ValueError("the [3, H, D] block of every sequence row must be contiguous")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and (w.dtype != torch.float32 or tuple(w.shape) != (D,) or not w.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous fp32 [D] tensor")
    if (rope_cos is None) != (rope_sin is None):
        raise ValueError("pass both rope tables or neither")
    for name, tb in (("rope_cos", rope_cos), ("rope_sin", rope_sin)):
        if tb is not None and (tb.dtype != torch.float32 or tuple(tb.shape) != (N, D // 2) or not tb.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous fp32 [N, D/2] tensor")
    if outs is None:
        outs = tuple(torch.empty((B, H, N, D), dtype=torch.bfloat16, device=qkv.device) for _ in range(3))
    for o in outs:
        if not o.is_contiguous() or tuple(o.shape) != (B, H, N, D) or o.dtype != torch.bfloat16:
            raise ValueError("outputs must be contiguous bf16 [B, H, N, D]")

    def ptr(t):
        return None if t is None else t.data_ptr()
    rc = _lib.dit_qkv_norm_rope_to_head_major(qkv.data_ptr(), qkv.stride(0), qkv.stride(1), B, N, H, D,
                                              ptr(q_weight), ptr(k_weight), float(eps), ptr(rope_cos),
                                              ptr(rope_sin), outs[0].data_ptr(), outs[1].data_ptr(),
                                              outs[2].data_ptr(), _stream_ptr(stream))
    _check(rc, "dit_qkv_norm_rope_to_head_major")
    return outs


_FP8_DTYPES = (torch.uint8, torch.float8_e4m3fn)


def qkv_cast_fp8(qkv: torch.Tensor, scales, *, out: torch.Tensor | None = None, stream=None):
    """One-pass E4M3 cast of a stacked [B, N, 3, H, D] bf16 buffer (b and n
    strides free, inner [3, H, D] contiguous), q/k/v scaled by scales[0..2],
    through `dit_qkv_cast_fp8`.  Returns the contiguous [B, N, 3, H, D] result
    (uint8 codes unless `out` is given as float8_e4m3fn)."""
    B, N, three, H, D = qkv.shape
    if three != 3 or qkv.dtype != torch.bfloat16 or not qkv.is_cuda:
        raise ValueError("expected a bf16 CUDA [B, N, 3, H, D] tensor")
    if qkv.stride(4) != 1 or qkv.stride(3) != D or qkv.stride(2) != H * D:
        raise ValueError("the [3, H, D] block of every sequence row must be contiguous")
    sq, sk, sv = (float(x) for x in scales)
    if out is None:
        out = torch.empty((B, N, 3, H, D), dtype=torch.uint8, device=qkv.device)
    if out.dtype not in _FP8_DTYPES or tuple(out.shape) != (B, N, 3, H, D) or not out.is_contiguous():
        raise ValueError("out must be a contiguous uint8 / float8_e4m3fn [B, N, 3, H, D] tensor")
    rc = _lib.dit_qkv_cast_fp8(qkv.data_ptr(), qkv.stride(0), qkv.stride(1), B, N, H, D, sq, sk, sv,
                               out.data_ptr(), _stream_ptr(stream))
    _check(rc, "dit_qkv_cast_fp8")
    return out


def _attn_fp8_args(q, k, v, descales, key_valid_len, scale, out, lse, out_dtype):
    B, Nq, H, D = q.shape
    Nkv = k.shape[1]
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype not in _FP8_DTYPES or not t.is_cuda:
            raise TypeError(f"{name} must be a uint8 / float8_e4m3fn CUDA tensor")
    if k.shape != (B, Nkv, H, D) or v.shape != (B, Nkv, H, D):
        raise ValueError("k and v must be [B, Nkv, H, D] matching q")
    dq, dk, dv = (float(x) for x in descales)
    kvl = Nkv if key_valid_len is None else int(key_valid_len)
    sc = float(D) ** -0.5 if scale is None else float(scale)
    if out is None:
        out = torch.empty((B, Nq, H, D), dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if out.dtype not in (torch.float32, torch.bfloat16) or tuple(out.shape) != (B, Nq, H, D):
        raise ValueError("out must be a [B, Nq, H, D] fp32 or bf16 tensor")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, Nq) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, H, Nq] tensor")
    st = AttnStrides(_strides4(q), _strides4(k), _strides4(v), _strides4(out))
    return B, Nq, Nkv, H, D, kvl, sc, dq, dk, dv, out, lse, st


def attn_fwd_fp8(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, descales, *, key_valid_len: int | None = None,
                 scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                 out_dtype: torch.dtype = torch.float32, stream=None):
    """Attention on E4M3 codes through `dit_attn_fwd_fp8`: q, k, v [B, N, H, D]
    uint8 / float8_e4m3fn views (e.g. of qkv_cast_fp8's output) standing for
    q * descales[0], k * descales[1], v * descales[2].  Returns (out, lse)."""
    B, Nq, Nkv, H, D, kvl, sc, dq, dk, dv, out, lse, st = _attn_fp8_args(q, k, v, descales, key_valid_len, scale,
                                                                         out, lse, out_dtype)
    rc = _lib.dit_attn_fwd_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(st), B, Nq, Nkv, H, D, kvl,
                               sc, dq, dk, dv, out.data_ptr(), DIT_F32 if out.dtype == torch.float32 else DIT_BF16,
                               lse.data_ptr(), _stream_ptr(stream))
    _check(rc, "dit_attn_fwd_fp8")
    return out, lse


def attn_fwd_fp8_ws(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, descales, *,
                    key_valid_len: int | None = None, scale: float | None = None, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32,
                    workspace: torch.Tensor | None = None, stream=None):
    """attn_fwd_fp8 through `dit_attn_fwd_fp8_ws`: the grid's last partial wave
    split over key ranges and merged.  The workspace (a uint8 CUDA tensor of
    attn_fwd_workspace_bytes) is allocated here unless given."""
    B, Nq, Nkv, H, D, kvl, sc, dq, dk, dv, out, lse, st = _attn_fp8_args(q, k, v, descales, key_valid_len, scale,
                                                                         out, lse, out_dtype)
    if workspace is None:
        nbytes = attn_fwd_workspace_bytes(B, Nq, H, D, kvl)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = _lib.dit_attn_fwd_fp8_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(st), B, Nq, Nkv, H, D, kvl,
                                  sc, dq, dk, dv, out.data_ptr(), DIT_F32 if out.dtype == torch.float32 else DIT_BF16,
                                  lse.data_ptr(), ws_ptr, ws_bytes, _stream_ptr(stream))
    _check(rc, "dit_attn_fwd_fp8_ws")
    return out, lse


def split_stacked_fp8(qkv8: torch.Tensor):
    """The q, k, v [B, N, H, D] views of a stacked [B, N, 3, H, D] FP8 buffer."""
    return qkv8[:, :, 0], qkv8[:, :, 1], qkv8[:, :, 2]


def attn_bwd_workspace_bytes(B: int, Nq: int, Nkv: int, H: int, D: int, key_valid_len: int, masked: bool = False) -> int:
    """Workspace of attn_bwd / attn_bwd_masked (current device)."""
    return int(_lib.dit_attn_bwd_workspace_bytes(int(B), int(Nq), int(Nkv), int(H), int(D), int(key_valid_len),
                                                 1 if masked else 0))


def _as_stream(stream):
    """A torch stream of a given one (any object with a cuda_stream).  The default
    stream's handle is 0, of which ExternalStream would make a stream of its own."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = int(stream.cuda_stream)
    return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()


def _on_stream(function, args, stream, given, workspace_bytes=None):
    """function(*args, stream) of the extension on a stream that was given:
    (status, results).

    What it allocates is that stream's memory: a workspace (the last of `args`
    where there is one, of workspace_bytes(args)), freed when the call returns, and
    a result, dropped at any time, must not be handed to the current stream's work
    while the given stream writes it, nor be memory that the current stream still
    reads.  Results (those not among `given`) count as used by the current stream
    too, which reads them once it has waited."""
    handle, here = int(stream.cuda_stream), torch.cuda.current_stream()
    if handle == here.cuda_stream:
        return function(*args, handle)
    with torch.cuda.stream(_as_stream(stream)):
        if workspace_bytes is not None and args[-1] is None:
            args = (*args[:-1], torch.empty(workspace_bytes(args), dtype=torch.uint8, device="cuda"))
        status, *results = function(*args, handle)
    for t in results:
        if t is not None and not any(t is g for g in given):
            t.record_stream(here)
    return (status, *results)


def _attn_bwd_space(args):
    q, k, mask_bits, key_valid_len = args[0], args[1], args[7], args[9]
    (B, Nq, H, D), Nkv = q.shape, k.shape[1]
    return attn_bwd_workspace_bytes(B, Nq, Nkv, H, D, Nkv if key_valid_len is None else key_valid_len, mask_bits is not None)


def _norm_bwd_space(args):
    x, parameters = args[1], (args[4], args[7], args[8])
    B, N, H, C = x.shape if x.dim() == 4 else (x.shape[0], x.shape[1], 1, x.shape[-1])
    sets = B if any(t is not None and t.dim() == 2 for t in parameters) else 1
    return layer_norm_bwd_workspace_bytes(B, N, H, C, sets)


def _is_fp32(dtype: torch.dtype) -> bool:
    if dtype is torch.float32:
        return True
    if dtype is torch.bfloat16:
        return False
    raise ValueError("results are fp32 or bf16")


def attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
             dout: torch.Tensor, *, dlse: torch.Tensor | None = None, key_valid_len: int | None = None,
             scale: float | None = None, dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
             dv: torch.Tensor | None = None, grad_dtype: torch.dtype = torch.bfloat16,
             workspace: torch.Tensor | None = None, stream=None):
    """Gradients of attn_fwd through `dit_attn_bwd`, the probabilities recomputed
    from lse.

    q, k, v, key_valid_len, scale as in the forward call, out and lse its
    results, dout (bf16, strided like q) the gradient of out and dlse (optional)
    that of lse.  dq [B, Nq, H, D], dk and dv [B, Nkv, H, D] may be given (e.g.
    views of one fused [B, N, 3, H, D] gradient) or are allocated in grad_dtype;
    keys past key_valid_len get zeros.  Returns (dq, dk, dv)."""
    if stream is None:
        rc, *grads = _calls.attn_bwd(q, k, v, out, lse, dout, dlse, None, None, key_valid_len, scale, dq, dk, dv,
                                     _is_fp32(grad_dtype), workspace, _stream_ptr(None))
    else:
        args = (q, k, v, out, lse, dout, dlse, None, None, key_valid_len, scale, dq, dk, dv, _is_fp32(grad_dtype), workspace)
        rc, *grads = _on_stream(_calls.attn_bwd, args, stream, (dq, dk, dv), _attn_bwd_space)
    if rc != DIT_OK:
        raise DitError(rc, "dit_attn_bwd")
    return tuple(grads)


def attn_bwd_masked(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
                    dout: torch.Tensor, mask_bits: torch.Tensor, *, mask_rows: int | None = None,
                    dlse: torch.Tensor | None = None, key_valid_len: int | None = None, scale: float | None = None,
                    dq: torch.Tensor | None = None, dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
                    grad_dtype: torch.dtype = torch.bfloat16, workspace: torch.Tensor | None = None, stream=None):
    """Gradients of attn_fwd_masked through `dit_attn_bwd_masked`: attn_bwd with
    the forward call's mask_bits and mask_rows."""
    if mask_bits is None:
        raise ValueError("mask_bits is missing")
    if stream is None:
        rc, *grads = _calls.attn_bwd(q, k, v, out, lse, dout, dlse, mask_bits, mask_rows, key_valid_len, scale, dq, dk, dv,
                                     _is_fp32(grad_dtype), workspace, _stream_ptr(None))
    else:
        args = (q, k, v, out, lse, dout, dlse, mask_bits, mask_rows, key_valid_len, scale, dq, dk, dv, _is_fp32(grad_dtype), workspace)
        rc, *grads = _on_stream(_calls.attn_bwd, args, stream, (dq, dk, dv), _attn_bwd_space)
    if rc != DIT_OK:
        raise DitError(rc, "dit_attn_bwd_masked")
    return tuple(grads)


def _window(left, right, sinks, frame):
    # (in the struct a negative bound is none)
    if any(bound is not None and bound < 0 for bound in (left, right)):
        raise ValueError("left and right are None or at least 0")
    if sinks < 0 or frame < 1:
        raise ValueError("sinks must be at least 0 and frame at least 1")
    if max(left or 0, right or 0, sinks, frame) > 0x7fffffff:
        raise ValueError("an integer argument is out of range")
    return ctypes.byref(Window(-1 if left is None else int(left), -1 if right is None else int(right), int(sinks), int(frame)))


def attn_fwd_window_workspace_bytes(B: int, Nq: int, H: int, Hkv: int, D: int, key_valid_len: int, *, left: int | None = None,
                                    right: int | None = 0, sinks: int = 0, frame: int = 1, offset: int = 0) -> int:
    """Workspace of attn_fwd_window (current device; 0: none)."""
    return int(_lib.dit_attn_fwd_window_workspace_bytes(int(B), int(Nq), int(H), int(Hkv), int(D), int(key_valid_len),
                                                        _window(left, right, sinks, frame), int(offset)))


def _window_fwd_space(args):
    q, k, left, right, sinks, frame, offset, key_valid_len = args[0], args[1], *args[3:9]
    (B, Nq, H, D), (Nkv, Hkv) = q.shape, k.shape[1:3]
    return attn_fwd_window_workspace_bytes(B, Nq, H, Hkv, D, Nkv if key_valid_len is None else key_valid_len, left=left, right=right,
                                           sinks=sinks, frame=frame, offset=offset)


def attn_fwd_window(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, left: int | None = None, right: int | None = 0,
                    sinks: int = 0, frame: int = 1, offset: int = 0, key_valid_len: int | None = None, scale: float | None = None,
                    out: torch.Tensor | None = None, lse: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32,
                    workspace: torch.Tensor | None = None, stream=None):
    """attn_fwd over a sliding window with sinks, through `dit_attn_fwd_window`.

    A query at position p (its row plus offset), in frame f = p // frame, sees the
    keys of the frames f - left to f + right (None: no bound on that side) and, of
    what lies before them, the first `sinks` tokens.  The defaults are the causal
    mask; frame=n, right=0 lets a video's frames of n tokens see themselves and
    the past.  q [B, Nq, H, D], k/v [B, Nkv, Hkv, D] bf16, strided as in attn_fwd; query head
    h reads K/V head h // (H // Hkv).  Returns (out [B, Nq, H, D] in out_dtype, lse [B, H, Nq]
    fp32); a row that sees nothing gets 0 and -inf."""
    args = (q, k, v, left, right, sinks, frame, offset, key_valid_len, scale, out, lse, _is_fp32(out_dtype), workspace)
    if stream is None:
        rc, o, l = _calls.window_fwd(*args, _stream_ptr(None))
    else:
        rc, o, l = _on_stream(_calls.window_fwd, args, stream, (out, lse), _window_fwd_space)
    if rc != DIT_OK:
        raise DitError(rc, "dit_attn_fwd_window")
    return o, l


def attn_bwd_window_workspace_bytes(B: int, Nq: int, Nkv: int, H: int, Hkv: int, D: int, key_valid_len: int, *, left: int | None = None,
                                    right: int | None = 0, sinks: int = 0, frame: int = 1, offset: int = 0) -> int:
    """Workspace of attn_bwd_window (current device)."""
    return int(_lib.dit_attn_bwd_window_workspace_bytes(int(B), int(Nq), int(Nkv), int(H), int(Hkv), int(D), int(key_valid_len),
                                                        _window(left, right, sinks, frame), int(offset)))


def _window_bwd_space(args):
    left, right, sinks, frame, offset, q, k, key_valid_len = *args[:7], args[14]
    (B, Nq, H, D), (Nkv, Hkv) = q.shape, k.shape[1:3]
    return attn_bwd_window_workspace_bytes(B, Nq, Nkv, H, Hkv, D, Nkv if key_valid_len is None else key_valid_len, left=left, right=right,
                                           sinks=sinks, frame=frame, offset=offset)


def attn_bwd_window(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor, dout: torch.Tensor, *,
                    left: int | None = None, right: int | None = 0, sinks: int = 0, frame: int = 1, offset: int = 0,
                    dlse: torch.Tensor | None = None, key_valid_len: int | None = None, scale: float | None = None,
                    dq: torch.Tensor | None = None, dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
                    grad_dtype: torch.dtype = torch.bfloat16, workspace: torch.Tensor | None = None, stream=None):
    """Gradients of attn_fwd_window through `dit_attn_bwd_window`: attn_bwd with the
    forward call's window; dk and dv [B, Nkv, Hkv, D] are summed over the query heads
    that share them (zeros without any).  Unlike the forward call it multiplies hidden
    keys of the tiles it visits, so they must be finite.  Returns (dq, dk, dv)."""
    args = (left, right, sinks, frame, offset, q, k, v, out, lse, dout, dlse, None, None, key_valid_len, scale, dq, dk, dv,
            _is_fp32(grad_dtype), workspace)
    if stream is None:
        rc, *grads = _calls.window_bwd(*args, _stream_ptr(None))
    else:
        rc, *grads = _on_stream(_calls.window_bwd, args, stream, (dq, dk, dv), _window_bwd_space)
    if rc != DIT_OK:
        raise DitError(rc, "dit_attn_bwd_window")
    return tuple(grads)


def paged_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                 kv_lens: torch.Tensor, *, new_lens: torch.Tensor | None = None, stream=None):
    """New tokens' K and V [B, T, Hkv, D] (bf16, channels contiguous, other strides free)
    into a paged cache, through `dit_paged_append`.

    k_cache, v_cache: bf16 [pages, page_size, Hkv, D], page_size a multiple of 8 (two
    tensors, or views of one).  page_table: int32 [B, width], the pages of each
    sequence in order; kv_lens: int32 [B], its tokens, the new ones included; new_lens:
    int32 [B], how many of the T are new (None: all).  Token t of sequence b goes to
    position kv_lens[b] - new_lens[b] + t; one without a page is dropped."""
    args = (k, v, k_cache, v_cache, page_table, kv_lens, new_lens)
    if stream is None:
        rc, = _calls.append(*args, _stream_ptr(None))
    else:
        rc, = _on_stream(_calls.append, args, stream, ())
    if rc != DIT_OK:
        raise DitError(rc, "dit_paged_append")


def attn_fwd_paged_workspace_bytes(B: int, T: int, H: int, Hkv: int, D: int, page_size: int, table_width: int, *, left: int | None = None,
                                   right: int | None = 0, sinks: int = 0, frame: int = 1) -> int:
    """Workspace of attn_fwd_paged (current device)."""
    return int(_lib.dit_attn_fwd_paged_workspace_bytes(int(B), int(T), int(H), int(Hkv), int(D), int(page_size), int(table_width),
                                                       _window(left, right, sinks, frame)))


def _paged_space(args):
    q, cache, table = args[0], args[1], args[3]
    B, T, H, D = q.shape
    left, right, sinks, frame = args[6:10]
    return attn_fwd_paged_workspace_bytes(B, T, H, cache.shape[2], D, cache.shape[1], table.shape[1], left=left, right=right, sinks=sinks,
                                          frame=frame)


def attn_fwd_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor, *,
                   q_lens: torch.Tensor | None = None, left: int | None = None, right: int | None = 0, sinks: int = 0, frame: int = 1,
                   scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                   out_dtype: torch.dtype = torch.bfloat16, workspace: torch.Tensor | None = None, stream=None):
    """attn_fwd_window of a chunk of new tokens, from one to thousands a sequence, over a
    paged cache that they have been appended to, through `dit_attn_fwd_paged`.

    q [B, T, H, D] bf16; the cache as in paged_append.  Row t < q_lens[b] (None: T) of
    sequence b is the query at position kv_lens[b] - q_lens[b] + t; the rows behind are
    left as they were in out and lse (results allocated here hold anything there).  A page index outside the cache (an evicted page)
    holds no keys.  The window as in attn_fwd_window.  Returns (out, lse [B, H, T])."""
    args = (q, k_cache, v_cache, page_table, kv_lens, q_lens, left, right, sinks, frame, scale, out, lse, _is_fp32(out_dtype), workspace)
    if stream is None:
        rc, o, l = _calls.paged(*args, _stream_ptr(None))
    else:
        rc, o, l = _on_stream(_calls.paged, args, stream, (out, lse), _paged_space)
    if rc != DIT_OK:
        raise DitError(rc, "dit_attn_fwd_paged")
    return o, l


def layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *,
                   eps: float = 1e-6, center: bool = True, out: torch.Tensor | None = None,
                   out_dtype: torch.dtype | None = None, stream=None):
    """Layer norm (center=False: RMS norm) of the last dimension of x through
    `dit_layer_norm_fwd`.

    x [B, N, C] or [B, N, H, C], bf16 or fp32, channels contiguous, other
    strides free; weight and bias fp32 [C], or [B, C] for one set per batch entry
    (modulation).  Returns (y, mean, rstd): y in out_dtype (default x's; fp32 x
    may give bf16 y), mean (None without center) and rstd fp32 without the
    channel dimension."""
    fp32 = None if out_dtype is None else _is_fp32(out_dtype)
    if stream is None:
        rc, y, mean, rstd = _calls.norm_fwd(x, weight, bias, eps, center, out, fp32, _stream_ptr(None))
    else:
        rc, y, mean, rstd = _on_stream(_calls.norm_fwd, (x, weight, bias, eps, center, out, fp32), stream, (out,))
    if rc != DIT_OK:
        raise DitError(rc, "dit_layer_norm_fwd")
    return y, mean, rstd


def layer_norm_bwd_workspace_bytes(B: int, N: int, H: int, C: int, param_batches: int = 1) -> int:
    """Workspace of layer_norm_bwd (current device)."""
    return int(_lib.dit_layer_norm_bwd_workspace_bytes(int(B), int(N), int(H), int(C), int(param_batches)))


def layer_norm_bwd(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor | None, rstd: torch.Tensor,
                   weight: torch.Tensor | None = None, *, has_bias: bool = True, dx: torch.Tensor | None = None,
                   dweight: torch.Tensor | None = None, dbias: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None):
    """Gradients of layer_norm_fwd through `dit_layer_norm_bwd`.

    dy has the forward result's type, mean is None for an RMS norm, weight as
    in the forward call.  Returns (dx, dweight, dbias): dx in x's type; dweight
    and dbias fp32 in weight's shape, None without a weight (dbias also without
    has_bias) unless a tensor to fill is given."""
    if stream is None:
        rc, gx, gw, gb = _calls.norm_bwd(dy, x, mean, rstd, weight, has_bias, dx, dweight, dbias, workspace, _stream_ptr(None))
    else:
        args = (dy, x, mean, rstd, weight, has_bias, dx, dweight, dbias, workspace)
        rc, gx, gw, gb = _on_stream(_calls.norm_bwd, args, stream, (dx, dweight, dbias), _norm_bwd_space)
    if rc != DIT_OK:
        raise DitError(rc, "dit_layer_norm_bwd")
    return gx, gw, gb


def rope_inv_freq(rotary_dim: int, *, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                  original_len: float = 4096.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """The frequency schedule of one position axis through `dit_rope_inv_freq`:
    base^(-2i / rotary_dim), scaled for long contexts by factor: "linear"
    (interpolated positions), "base" (a larger base) or "by_parts" (slow pairs
    only, by the turns they make over original_len).  Returns (inv_freq, mscale):
    a CPU fp64 tensor [rotary_dim / 2] for rope() and its amplitude factor.
    Schedules of several axes are concatenated with torch.cat."""
    if scaling not in _ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(k for k in _ROPE_SCALINGS if k)} or None")
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even")
    freq = torch.empty(rotary_dim // 2, dtype=torch.float64)
    mscale = ctypes.c_float()
    rc = _lib.dit_rope_inv_freq(rotary_dim // 2, float(base), _ROPE_SCALINGS[scaling], float(factor), float(original_len),
                                float(beta_fast), float(beta_slow), freq.data_ptr(), ctypes.byref(mscale))
    _check(rc, "dit_rope_inv_freq")
    return freq, mscale.value


def rope(x: torch.Tensor, inv_freq: torch.Tensor, positions: torch.Tensor | None = None, *,
         layout: str = "interleaved", axis_pairs=None, offset: int = 0, mscale: float = 1.0, inverse: bool = False,
         out: torch.Tensor | None = None, stream=None):
    """Rotary positions of x [B, N, H, D] (bf16 or fp32, channels contiguous,
    other strides free) through `dit_rope`.

    inv_freq: CPU fp64 tensor, one angle per position step for each of the
    rotary_dim / 2 pairs; layout "interleaved" (channels 2i, 2i+1) or "half"
    (i, i + rotary_dim / 2).  positions: int32 CUDA tensor [N] or [B or 1, N, axes]
    (None: 0, 1, ...), offset added; axis_pairs: how many pairs turn with each
    axis.  inverse turns back (the gradient).  out may be x."""
    if layout not in _ROPE_LAYOUTS:
        raise ValueError('layout must be "interleaved" or "half"')
    half = _ROPE_LAYOUTS[layout]
    if stream is None:
        rc, y = _calls.rope(x, inv_freq, positions, half, axis_pairs, offset, mscale, inverse, out, _stream_ptr(None))
    else:
        rc, y = _on_stream(_calls.rope, (x, inv_freq, positions, half, axis_pairs, offset, mscale, inverse, out), stream, (out,))
    if rc != DIT_OK:
        raise DitError(rc, "dit_rope")
    return y


def watchdog_selftest(limit_us: int = 100_000, stream=None):
    """Enqueue the library's watchdog self-test (a bounded wait that must run
    out); read the outcome with check_watchdog()."""
    _check(_lib.dit_watchdog_selftest(int(limit_us), _stream_ptr(stream)), "dit_watchdog_selftest")


def check_watchdog(stream=None):
    """Synchronise and read/clear the device status word: (status, info[4])."""
    info = (ctypes.c_uint32 * 4)()
    rc = _lib.dit_check_watchdog(_stream_ptr(stream), info)
    return rc, list(info)
