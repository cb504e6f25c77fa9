"""Thin Python binding of libdsv.so (the C ABI declared in include/dsv.h).

Argument marshalling only: torch tensors supply device memory and the current
CUDA stream; every step of the hot path runs in the library's kernels.  There
is no fallback: if the library has not been built (``__graft_entry__.build()``
or ``python -m dynamic_block_sparse_projection_gb300.build``) importing this
module raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import importlib.machinery
import importlib.util
import math
from pathlib import Path
from typing import Optional, Sequence, Tuple

import torch

_LIB_PATH = Path(__file__).resolve().parent / "_build" / "libdsv.so"
_CALLS_PATH = _LIB_PATH.with_name("dsv_calls" + importlib.machinery.EXTENSION_SUFFIXES[0])

DSV_OK, DSV_ERR_INVALID_ARG, DSV_ERR_UNSUPPORTED, DSV_ERR_CUDA, DSV_ERR_BAD_INDEX, DSV_ERR_TIMEOUT, DSV_ERR_INTERNAL = range(7)

# Every symbol the header declares; checked at load time.
EXPORTS = (
    "dsv_predict_workspace_bytes", "dsv_predict_scores",
    "dsv_topk_workspace_bytes", "dsv_topk_blocks",
    "dsv_sparse_attn_fwd",
    "dsv_attn_bwd_workspace_bytes", "dsv_sparse_attn_bwd",
    "dsv_status_string", "dsv_get_device_error", "dsv_clear_device_error",
    "dsv_set_wait_limit_ns", "dsv_version",
    "dsv_topk_blocks_noalloc",
    "dsv_attn_bwd_preprocess", "dsv_attn_bwd_dkdv", "dsv_attn_bwd_dq",
    "dsv_cube_permute", "dsv_topk_mass_workspace_bytes", "dsv_topk_mass_blocks",
    "dsv_predict_max_workspace_bytes", "dsv_predict_scores_max",
    "dsv_selftest_wait_timeout",
    "dsv_predict_topk_workspace_bytes", "dsv_predict_topk_blocks",
    "dsv_dispatch_heads",
    "dsv_rope_axes_fwd", "dsv_rope_axes_bwd_workspace_bytes", "dsv_rope_axes_bwd",
    "dsv_packed_attn_fwd_workspace_bytes", "dsv_packed_attn_fwd",
    "dsv_packed_attn_bwd_workspace_bytes", "dsv_packed_attn_bwd",
    "dsv_layer_norm_fwd", "dsv_layer_norm_bwd_workspace_bytes", "dsv_layer_norm_bwd",
    "dsv_quantize_fp8", "dsv_matmul_fp8",
)
SELFTEST_WAIT_ID = 0xD5F0


class _NoCalls:
    """In the place of the C module where it has not been built: the calls that go through it raise, the others work."""

    def __getattr__(self, name):
        raise ImportError(f"dsv_calls is not built for this interpreter ({_CALLS_PATH}); "
                          "run __graft_entry__.build() first")


def _load_calls():
    if not _CALLS_PATH.exists():
        return _NoCalls()
    loader = importlib.machinery.ExtensionFileLoader("dsv_calls", str(_CALLS_PATH))
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("dsv_calls", loader))
    loader.exec_module(module)
    return module


_calls = _load_calls()
View = None if isinstance(_calls, _NoCalls) else _calls.View       # dsv_view
Rows = None if isinstance(_calls, _NoCalls) else _calls.Rows       # dsv_rows
DSV_BF16, DSV_F32, DSV_E4M3, DSV_E5M2 = range(4)                   # dsv_type
if Rows is not None:
    _calls.set_types(torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e5m2, torch.int32)


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32),
                ("d", ctypes.c_int32), ("block", ctypes.c_int32), ("r", ctypes.c_int32)]


class Rope(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32), ("d", ctypes.c_int32),
                ("axes", ctypes.c_int32), ("section", ctypes.c_int32 * 4), ("theta", ctypes.c_double)]


class Packed(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int32), ("H", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("Tq", ctypes.c_int32),
                ("Tk", ctypes.c_int32), ("d", ctypes.c_int32)]


class Norm(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("C", ctypes.c_int32), ("S", ctypes.c_int32), ("eps", ctypes.c_float)]


class Matmul(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("a_rows", ctypes.c_int32),
                ("b_rows", ctypes.c_int32), ("accumulate", ctypes.c_int32)]


class DsvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def _load() -> ctypes.CDLL:
    if not _LIB_PATH.exists():
        raise ImportError(f"libdsv.so is not built ({_LIB_PATH}); run __graft_entry__.build() first")
    lib = ctypes.CDLL(str(_LIB_PATH))
    missing = [s for s in EXPORTS if not hasattr(lib, s)]
    if missing:
        raise ImportError(f"libdsv.so lacks symbols: {missing}")
    vp, sz, i32, u32p = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.POINTER(ctypes.c_uint32)
    lib.dsv_predict_workspace_bytes.argtypes = [Shape]
    lib.dsv_predict_workspace_bytes.restype = sz
    lib.dsv_predict_scores.argtypes = [vp, vp, vp, vp, Shape, vp, vp, sz, vp]
    lib.dsv_predict_scores.restype = ctypes.c_int
    lib.dsv_predict_max_workspace_bytes.argtypes = [Shape]
    lib.dsv_predict_max_workspace_bytes.restype = sz
    lib.dsv_predict_scores_max.argtypes = [vp, vp, vp, vp, Shape, vp, vp, sz, vp]
    lib.dsv_predict_scores_max.restype = ctypes.c_int
    lib.dsv_topk_workspace_bytes.argtypes = [Shape]
    lib.dsv_topk_workspace_bytes.restype = sz
    lib.dsv_topk_blocks.argtypes = [vp, Shape, ctypes.POINTER(i32), vp, vp, vp, vp, vp, sz, vp]
    lib.dsv_topk_blocks.restype = ctypes.c_int
    lib.dsv_sparse_attn_fwd.argtypes = [vp, vp, vp, Shape, vp, vp, ctypes.c_float, vp, vp, vp]
    lib.dsv_sparse_attn_fwd.restype = ctypes.c_int
    lib.dsv_attn_bwd_workspace_bytes.argtypes = [Shape]
    lib.dsv_attn_bwd_workspace_bytes.restype = sz
    lib.dsv_sparse_attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, Shape, vp, vp, vp, vp, ctypes.c_float,
                                        vp, vp, vp, vp, sz, vp]
    lib.dsv_sparse_attn_bwd.restype = ctypes.c_int
    lib.dsv_status_string.argtypes = [ctypes.c_int]
    lib.dsv_status_string.restype = ctypes.c_char_p
    lib.dsv_get_device_error.argtypes = [vp, u32p]
    lib.dsv_get_device_error.restype = ctypes.c_int
    lib.dsv_clear_device_error.argtypes = [vp]
    lib.dsv_clear_device_error.restype = ctypes.c_int
    lib.dsv_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.dsv_set_wait_limit_ns.restype = ctypes.c_int
    lib.dsv_topk_blocks_noalloc.argtypes = [vp, Shape, ctypes.POINTER(i32), vp, vp, vp, vp, vp]
    lib.dsv_topk_blocks_noalloc.restype = ctypes.c_int
    lib.dsv_attn_bwd_preprocess.argtypes = [vp, vp, vp, Shape, vp, sz, vp]
    lib.dsv_attn_bwd_preprocess.restype = ctypes.c_int
    lib.dsv_attn_bwd_dkdv.argtypes = [vp, vp, vp, vp, Shape, vp, vp, ctypes.c_float, vp, vp, vp, sz, vp]
    lib.dsv_attn_bwd_dkdv.restype = ctypes.c_int
    lib.dsv_attn_bwd_dq.argtypes = [vp, vp, vp, vp, Shape, vp, vp, ctypes.c_float, vp, vp, sz, vp]
    lib.dsv_attn_bwd_dq.restype = ctypes.c_int
    lib.dsv_topk_mass_workspace_bytes.argtypes = [Shape]
    lib.dsv_topk_mass_workspace_bytes.restype = sz
    lib.dsv_topk_mass_blocks.argtypes = [vp, Shape, ctypes.c_float, ctypes.c_float, i32, i32, vp, vp, vp, vp, sz, vp,
                                         sz, vp]
    lib.dsv_topk_mass_blocks.restype = ctypes.c_int
    lib.dsv_cube_permute.argtypes = [vp, vp, Shape, i32, i32, i32, i32, i32, i32, i32, vp]
    lib.dsv_cube_permute.restype = ctypes.c_int
    lib.dsv_predict_topk_workspace_bytes.argtypes = [Shape]
    lib.dsv_predict_topk_workspace_bytes.restype = sz
    lib.dsv_predict_topk_blocks.argtypes = [vp, vp, vp, vp, Shape, ctypes.POINTER(i32), vp, vp, vp, vp, vp, vp, sz,
                                            vp]
    lib.dsv_predict_topk_blocks.restype = ctypes.c_int
    f32p = ctypes.POINTER(ctypes.c_float)
    lib.dsv_dispatch_heads.argtypes = [ctypes.POINTER(i32), i32, i32, f32p, f32p, i32, ctypes.POINTER(i32),
                                       ctypes.POINTER(i32)]
    lib.dsv_dispatch_heads.restype = ctypes.c_int
    lib.dsv_selftest_wait_timeout.argtypes = [vp]
    lib.dsv_selftest_wait_timeout.restype = ctypes.c_int
    lib.dsv_rope_axes_bwd_workspace_bytes.argtypes = [Rope]
    lib.dsv_rope_axes_bwd_workspace_bytes.restype = sz
    lib.dsv_packed_attn_fwd_workspace_bytes.argtypes = [Packed]
    lib.dsv_packed_attn_fwd_workspace_bytes.restype = sz
    lib.dsv_packed_attn_bwd_workspace_bytes.argtypes = [Packed]
    lib.dsv_packed_attn_bwd_workspace_bytes.restype = sz
    lib.dsv_layer_norm_bwd_workspace_bytes.argtypes = [Norm]
    lib.dsv_layer_norm_bwd_workspace_bytes.restype = sz
    lib.dsv_version.argtypes = []
    lib.dsv_version.restype = i32
    # the calls with several structures, by C (pycalls.c): the same arguments
    if View is not None:
        for name in ("dsv_rope_axes_fwd", "dsv_rope_axes_bwd", "dsv_packed_attn_fwd", "dsv_packed_attn_bwd",
                     "dsv_layer_norm_fwd", "dsv_layer_norm_bwd", "dsv_quantize_fp8", "dsv_matmul_fp8"):
            setattr(lib, name, getattr(_calls, name))
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.dsv_status_string(status).decode()


def _check(status: int, what: str) -> None:
    if status != DSV_OK:
        raise DsvError(status, what)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# The current stream's handle without a Stream object around it (2 us a call), where torch has the call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device, stream=None) -> Optional[int]:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _call(fn, what: str, device: torch.device, *args) -> None:
    """fn(*args) under `device`: nothing to switch where it is the current one
    already (torch.cuda.device costs as much as a small kernel's launch)."""
    if device.type == "cuda" and device.index == torch.cuda.current_device():
        _check(fn(*args), what)
    else:
        with torch.cuda.device(device):
            _check(fn(*args), what)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, device: Optional[torch.device] = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_rows(t: torch.Tensor, name: str, device: Optional[torch.device] = None):
    """t is a bf16 CUDA tensor whose last dimension is contiguous; the library checks its other strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _need_on(device: torch.device, index: int, dtype: torch.dtype, **tensors) -> None:
    """_need for each tensor (None: left out)."""
    for name, t in tensors.items():
        if t is not None and (t.dtype is not dtype or t.get_device() != index or not t.is_contiguous()):
            _need(t, name, dtype, device)


def _dims(t, name: str, n: int) -> Tuple[int, ...]:
    """The shape of t, which must be an n-dimensional tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = tuple(t.shape)
    if len(shape) != n:
        raise ValueError(f"{name} must have {n} dimensions, got shape {shape}")
    return shape


def _shape(t, name: str, shape) -> None:
    """t must have exactly this shape (the library reads and writes whole tensors)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _room(t, name: str, n: int) -> None:
    """t must hold at least n elements (a CSR array may be longer than its contents)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} elements, needs at least {n}")


def _groups(N: int, block: int) -> int:
    return N // block if block > 0 else 0


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def nnz_of(B: int, G: int, k_per_head: Sequence[int]) -> int:
    return B * G * int(sum(int(k) for k in k_per_head))


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace needs {nbytes} bytes")
        return workspace
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def predict_workspace_bytes(B: int, H: int, N: int, d: int, block: int, r: int) -> int:
    return lib.dsv_predict_workspace_bytes(Shape(B, H, N, d, block, r))


def topk_workspace_bytes(B: int, H: int, N: int, d: int, block: int) -> int:
    return lib.dsv_topk_workspace_bytes(Shape(B, H, N, d, block, 8))


def attn_bwd_workspace_bytes(B: int, H: int, N: int, d: int, block: int) -> int:
    return lib.dsv_attn_bwd_workspace_bytes(Shape(B, H, N, d, block, 8))


# ---------------------------------------------------------------------------
# The four calls of the hot path
# ---------------------------------------------------------------------------

def predict_scores(Q, K, Wq, Wk, block: int, *, out=None, workspace=None, stream=None) -> torch.Tensor:
    """scores[b,h,g,j] = qbar_g . kbar_j (fp32 [B,H,G,nb]); see dsv_predict_scores."""
    return _predict(lib.dsv_predict_scores, lib.dsv_predict_workspace_bytes, "dsv_predict_scores",
                    Q, K, Wq, Wk, block, out, workspace, stream)


def _predict(fn, ws_fn, what, Q, K, Wq, Wk, block, out, workspace, stream):
    B, H, N, d = _dims(Q, "Q", 4)
    _shape(K, "K", (B, H, N, d))
    r = _dims(Wq, "Wq", 3)[2]
    _shape(Wq, "Wq", (H, d, r))
    _shape(Wk, "Wk", (H, d, r))
    G = _groups(N, block)
    if out is not None:
        _shape(out, "out", (B, H, G, G))
    _need(Q, "Q", torch.bfloat16)
    dev = Q.device
    _need(K, "K", torch.bfloat16, dev)
    _need(Wq, "Wq", torch.float32, dev)
    _need(Wk, "Wk", torch.float32, dev)
    s = Shape(B, H, N, d, block, r)
    if out is None:
        out = torch.empty(B, H, G, G, dtype=torch.float32, device=dev)
    _need(out, "out", torch.float32, dev)
    nbytes = ws_fn(s)
    ws = _workspace(nbytes, dev, workspace)
    with torch.cuda.device(dev):
        _check(fn(_ptr(Q), _ptr(K), _ptr(Wq), _ptr(Wk), s, _ptr(out), _ptr(ws), nbytes, _stream(dev, stream)), what)
    return out


def predict_max_workspace_bytes(B: int, H: int, N: int, d: int, block: int, r: int) -> int:
    return int(lib.dsv_predict_max_workspace_bytes(Shape(B, H, N, d, block, r)))


def predict_scores_max(Q, K, Wq, Wk, block: int, *, out=None, workspace=None, stream=None) -> torch.Tensor:
    """scores[b,h,g,j] = max low-rank logit of tile (g, j) (fp32 [B,H,G,nb]); see dsv_predict_scores_max."""
    return _predict(lib.dsv_predict_scores_max, lib.dsv_predict_max_workspace_bytes, "dsv_predict_scores_max",
                    Q, K, Wq, Wk, block, out, workspace, stream)


def topk_blocks(scores, k_per_head: Sequence[int], block: int, N: int, d: int = 128, *, outs=None,
                workspace=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(fwd_ptr, fwd_col, bwd_ptr, bwd_col) int32 CSR lists; see dsv_topk_blocks."""
    B, H, G, nb = _score_dims(scores, block, N, k_per_head)
    nnz = nnz_of(B, G, k_per_head)
    if outs is not None:
        _csr_room(outs, B * H * G + 1, nnz, B * H * nb + 1, nnz)
    _need(scores, "scores", torch.float32)
    dev = scores.device
    s = Shape(B, H, N, d, block, 8)
    if outs is None:
        outs = (torch.empty(B * H * G + 1, dtype=torch.int32, device=dev),
                torch.empty(max(nnz, 1), dtype=torch.int32, device=dev),
                torch.empty(B * H * nb + 1, dtype=torch.int32, device=dev),
                torch.empty(max(nnz, 1), dtype=torch.int32, device=dev))
    for name, t in zip(("fwd_ptr", "fwd_col", "bwd_ptr", "bwd_col"), outs):
        _need(t, name, torch.int32, dev)
    karr = (ctypes.c_int32 * max(H, 1))(*[int(k) for k in k_per_head])
    nbytes = lib.dsv_topk_workspace_bytes(s)
    ws = _workspace(nbytes, dev, workspace)
    with torch.cuda.device(dev):
        _check(lib.dsv_topk_blocks(_ptr(scores), s, karr, *[_ptr(t) for t in outs], _ptr(ws), nbytes,
                                   _stream(dev, stream)), "dsv_topk_blocks")
    fp, fc, bp, bc = outs
    return fp, fc[:nnz], bp, bc[:nnz]


def predict_topk_workspace_bytes(B: int, H: int, N: int, d: int, block: int, r: int) -> int:
    return int(lib.dsv_predict_topk_workspace_bytes(Shape(B, H, N, d, block, r)))


def predict_topk_blocks(Q, K, Wq, Wk, k_per_head: Sequence[int], block: int, *, outs=None, scores=None,
                        workspace=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(fwd_ptr, fwd_col, bwd_ptr, bwd_col) int32 CSR lists of the fused
    predictor + top-k (the score matrix stays on chip); see
    dsv_predict_topk_blocks.  `scores`, if given (fp32 [B, H, G, G]),
    receives the scores the selection used."""
    B, H, N, d = _dims(Q, "Q", 4)
    _shape(K, "K", (B, H, N, d))
    r = _dims(Wq, "Wq", 3)[2]
    _shape(Wq, "Wq", (H, d, r))
    _shape(Wk, "Wk", (H, d, r))
    if len(k_per_head) != H:
        raise ValueError(f"k_per_head has {len(k_per_head)} entries, expected one per head ({H})")
    G = _groups(N, block)
    nnz = nnz_of(B, G, k_per_head)
    if outs is not None:
        _csr_room(outs, B * H * G + 1, nnz, B * H * G + 1, nnz)
    if scores is not None:
        _shape(scores, "scores", (B, H, G, G))
    _need(Q, "Q", torch.bfloat16)
    dev = Q.device
    _need(K, "K", torch.bfloat16, dev)
    _need(Wq, "Wq", torch.float32, dev)
    _need(Wk, "Wk", torch.float32, dev)
    if scores is not None:
        _need(scores, "scores", torch.float32, dev)
    if outs is None:
        outs = (torch.empty(B * H * G + 1, dtype=torch.int32, device=dev),
                torch.empty(max(nnz, 1), dtype=torch.int32, device=dev),
                torch.empty(B * H * G + 1, dtype=torch.int32, device=dev),
                torch.empty(max(nnz, 1), dtype=torch.int32, device=dev))
    for name, t in zip(("fwd_ptr", "fwd_col", "bwd_ptr", "bwd_col"), outs):
        _need(t, name, torch.int32, dev)
    s = Shape(B, H, N, d, block, r)
    karr = (ctypes.c_int32 * max(H, 1))(*[int(k) for k in k_per_head])
    nbytes = lib.dsv_predict_topk_workspace_bytes(s)
    ws = _workspace(nbytes, dev, workspace)
    with torch.cuda.device(dev):
        _check(lib.dsv_predict_topk_blocks(_ptr(Q), _ptr(K), _ptr(Wq), _ptr(Wk), s, karr, *[_ptr(t) for t in outs],
                                           _ptr(scores), _ptr(ws), nbytes, _stream(dev, stream)),
               "dsv_predict_topk_blocks")
    fp, fc, bp, bc = outs
    return fp, fc[:nnz], bp, bc[:nnz]


def _score_dims(scores, block: int, N: int, k_per_head=None) -> Tuple[int, int, int, int]:
    """[B, H, G, nb] of a score matrix, which must be square with G = N / block."""
    B, H, G, nb = _dims(scores, "scores", 4)
    if G != nb or G != _groups(N, block):
        raise ValueError(f"scores has shape {(B, H, G, nb)}, expected [B, H, N/block, N/block] "
                         f"with N = {N}, block = {block}")
    if k_per_head is not None and len(k_per_head) != H:
        raise ValueError(f"k_per_head has {len(k_per_head)} entries, expected one per head ({H})")
    return B, H, G, nb


def _csr_room(outs, n_fptr: int, n_fcol: int, n_bptr: int, n_bcol: int) -> None:
    if len(outs) != 4:
        raise ValueError("outs must be (fwd_ptr, fwd_col, bwd_ptr, bwd_col)")
    for name, t, n in zip(("fwd_ptr", "fwd_col", "bwd_ptr", "bwd_col"), outs, (n_fptr, n_fcol, n_bptr, n_bcol)):
        _room(t, name, n)


def topk_mass_workspace_bytes(B: int, H: int, N: int, d: int, block: int) -> int:
    return lib.dsv_topk_mass_workspace_bytes(Shape(B, H, N, d, block, 8))


def topk_mass_blocks(scores, tau: float, block: int, N: int, d: int = 128, *, temperature: float = 0.0,
                     kmin: int = 1, kmax: int = 0, outs=None, workspace=None, stream=None, trim: bool = True):
    """(fwd_ptr, fwd_col, bwd_ptr, bwd_col) int32 CSR lists of the
    mass-threshold selection; see dsv_topk_mass_blocks.  temperature <= 0
    selects 1/sqrt(d), kmax <= 0 selects nb.  With trim the column arrays are
    returned cut to nnz = fwd_ptr[-1], which this reads back from the device
    (a synchronisation); without it they are returned whole."""
    B, H, G, nb = _score_dims(scores, block, N)
    if outs is not None:
        _csr_room(outs, B * H * G + 1, 0, B * H * nb + 1, 0)     # the columns' capacity goes to the library
    _need(scores, "scores", torch.float32)
    dev = scores.device
    s = Shape(B, H, N, d, block, 8)
    temperature = float(temperature) if temperature > 0 else 1.0 / math.sqrt(d)
    kmax = int(kmax) if kmax > 0 else nb
    cap = B * H * G * kmax
    if outs is None:
        outs = (torch.empty(B * H * G + 1, dtype=torch.int32, device=dev),
                torch.empty(max(cap, 1), dtype=torch.int32, device=dev),
                torch.empty(B * H * nb + 1, dtype=torch.int32, device=dev),
                torch.empty(max(cap, 1), dtype=torch.int32, device=dev))
    for name, t in zip(("fwd_ptr", "fwd_col", "bwd_ptr", "bwd_col"), outs):
        _need(t, name, torch.int32, dev)
    cap = min(outs[1].numel(), outs[3].numel())
    nbytes = lib.dsv_topk_mass_workspace_bytes(s)
    ws = _workspace(nbytes, dev, workspace)
    with torch.cuda.device(dev):
        _check(lib.dsv_topk_mass_blocks(_ptr(scores), s, float(tau), temperature, int(kmin), kmax,
                                        *[_ptr(t) for t in outs], cap, _ptr(ws), nbytes, _stream(dev, stream)),
               "dsv_topk_mass_blocks")
    fp, fc, bp, bc = outs
    if not trim:
        return fp, fc, bp, bc
    nnz = int(fp[-1].item()) if B * H * G > 0 else 0
    return fp, fc[:nnz], bp, bc[:nnz]


def topk_blocks_noalloc(scores, k_per_head: Sequence[int], block: int, N: int, d: int = 128, *, outs,
                        stream=None) -> None:
    """dsv_topk_blocks_noalloc into caller-provided `outs`; it allocates nothing.

    For callers that cannot allocate device memory: the library's fixed
    device scratch replaces the workspace.  Calls share that scratch, so do
    not let two of them overlap on the GPU.
    """
    B, H, G, nb = _score_dims(scores, block, N, k_per_head)
    nnz = nnz_of(B, G, k_per_head)
    _csr_room(outs, B * H * G + 1, nnz, B * H * nb + 1, nnz)
    _need(scores, "scores", torch.float32)
    dev = scores.device
    for name, t in zip(("fwd_ptr", "fwd_col", "bwd_ptr", "bwd_col"), outs):
        _need(t, name, torch.int32, dev)
    karr = (ctypes.c_int32 * max(H, 1))(*[int(k) for k in k_per_head])
    with torch.cuda.device(dev):
        _check(lib.dsv_topk_blocks_noalloc(_ptr(scores), Shape(B, H, N, d, block, 8), karr,
                                           *[_ptr(t) for t in outs], _stream(dev, stream)), "dsv_topk_blocks_noalloc")


def sparse_attn_fwd(Q, K, V, fwd_ptr, fwd_col, block: int, softmax_scale: float = 0.0, *, out=None, lse=None,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(O bf16 [B,H,N,d], lse fp32 [B,H,N]); see dsv_sparse_attn_fwd."""
    B, H, N, d = _dims(Q, "Q", 4)
    for name, t in (("K", K), ("V", V)) + ((("out", out),) if out is not None else ()):
        _shape(t, name, (B, H, N, d))
    if lse is not None:
        _shape(lse, "lse", (B, H, N))
    _room(fwd_ptr, "fwd_ptr", B * H * _groups(N, block) + 1)
    _need(Q, "Q", torch.bfloat16)
    dev = Q.device
    for name, t in (("K", K), ("V", V)):
        _need(t, name, torch.bfloat16, dev)
    for name, t in (("fwd_ptr", fwd_ptr), ("fwd_col", fwd_col)):
        _need(t, name, torch.int32, dev)
    B, H, N, d = Q.shape
    s = Shape(B, H, N, d, block, 8)
    if out is None:
        out = torch.empty_like(Q)
    if lse is None:
        lse = torch.empty(B, H, N, dtype=torch.float32, device=dev)
    _need(out, "out", torch.bfloat16, dev)
    _need(lse, "lse", torch.float32, dev)
    with torch.cuda.device(dev):
        _check(lib.dsv_sparse_attn_fwd(_ptr(Q), _ptr(K), _ptr(V), s, _ptr(fwd_ptr), _ptr(fwd_col),
                                       float(softmax_scale), _ptr(out), _ptr(lse), _stream(dev, stream)),
               "dsv_sparse_attn_fwd")
    return out, lse


def sparse_attn_bwd(Q, K, V, O, dO, lse, fwd_ptr, fwd_col, bwd_ptr, bwd_col, block: int,
                    softmax_scale: float = 0.0, *, outs=None, workspace=None, stream=None):
    """(dQ, dK, dV) bf16 [B,H,N,d]; see dsv_sparse_attn_bwd."""
    B, H, N, d = _dims(Q, "Q", 4)
    for name, t in (("K", K), ("V", V), ("O", O), ("dO", dO)):
        _shape(t, name, (B, H, N, d))
    if outs is not None:
        if len(outs) != 3:
            raise ValueError("outs must be (dQ, dK, dV)")
        for name, t in zip(("dQ", "dK", "dV"), outs):
            _shape(t, name, (B, H, N, d))
    _shape(lse, "lse", (B, H, N))
    rows = B * H * _groups(N, block) + 1
    _room(fwd_ptr, "fwd_ptr", rows)
    _room(bwd_ptr, "bwd_ptr", rows)
    _need(Q, "Q", torch.bfloat16)
    dev = Q.device
    for name, t in (("K", K), ("V", V), ("O", O), ("dO", dO)):
        _need(t, name, torch.bfloat16, dev)
    _need(lse, "lse", torch.float32, dev)
    for name, t in (("fwd_ptr", fwd_ptr), ("fwd_col", fwd_col), ("bwd_ptr", bwd_ptr), ("bwd_col", bwd_col)):
        _need(t, name, torch.int32, dev)
    B, H, N, d = Q.shape
    s = Shape(B, H, N, d, block, 8)
    if outs is None:
        outs = (torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V))
    for name, t in zip(("dQ", "dK", "dV"), outs):
        _need(t, name, torch.bfloat16, dev)
    nbytes = lib.dsv_attn_bwd_workspace_bytes(s)
    ws = _workspace(nbytes, dev, workspace)
    with torch.cuda.device(dev):
        _check(lib.dsv_sparse_attn_bwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(lse), s,
                                       _ptr(fwd_ptr), _ptr(fwd_col), _ptr(bwd_ptr), _ptr(bwd_col),
                                       float(softmax_scale), *[_ptr(t) for t in outs], _ptr(ws), nbytes,
                                       _stream(dev, stream)), "dsv_sparse_attn_bwd")
    return outs


def cube_permute(x, grid, cube, *, inverse: bool = False, out=None, stream=None) -> torch.Tensor:
    """x bf16 [B,H,N,d] between raster and cube token order; see dsv_cube_permute.

    grid = (T, Hl, Wl) with N = T*Hl*Wl; cube = (ct, cy, cx), whose volume is
    the group / block size of the hot path."""
    _dims(x, "x", 4)
    if out is not None:
        _shape(out, "out", x.shape)
    _need(x, "x", torch.bfloat16)
    dev = x.device
    B, H, N, d = x.shape
    T, Hl, Wl = (int(v) for v in grid)
    ct, cy, cx = (int(v) for v in cube)
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", torch.bfloat16, dev)
    s = Shape(B, H, N, d, ct * cy * cx, 8)
    with torch.cuda.device(dev):
        _check(lib.dsv_cube_permute(_ptr(x), _ptr(out), s, T, Hl, Wl, ct, cy, cx, 1 if inverse else 0,
                                    _stream(dev, stream)), "dsv_cube_permute")
    return out


def attn_bwd_preprocess(O, dO, lse, block: int, *, workspace, stream=None) -> None:
    """D and lse * log2(e) into `workspace`; see dsv_attn_bwd_preprocess."""
    B, H, N, d = _dims(O, "O", 4)
    _shape(dO, "dO", (B, H, N, d))
    _shape(lse, "lse", (B, H, N))
    _need(O, "O", torch.bfloat16)
    dev = O.device
    _need(dO, "dO", torch.bfloat16, dev)
    _need(lse, "lse", torch.float32, dev)
    _need(workspace, "workspace", workspace.dtype, dev)
    s = Shape(B, H, N, d, block, 8)
    with torch.cuda.device(dev):
        _check(lib.dsv_attn_bwd_preprocess(_ptr(O), _ptr(dO), _ptr(lse), s, _ptr(workspace), _nbytes(workspace),
                                           _stream(dev, stream)), "dsv_attn_bwd_preprocess")


def attn_bwd_dkdv(Q, K, V, dO, bwd_ptr, bwd_col, block: int, softmax_scale: float = 0.0, *, outs, workspace,
                  stream=None) -> None:
    """dK, dV into outs = (dK, dV) after attn_bwd_preprocess; see dsv_attn_bwd_dkdv."""
    B, H, N, d = _dims(Q, "Q", 4)
    if len(outs) != 2:
        raise ValueError("outs must be (dK, dV)")
    for name, t in (("K", K), ("V", V), ("dO", dO), ("dK", outs[0]), ("dV", outs[1])):
        _shape(t, name, (B, H, N, d))
    _room(bwd_ptr, "bwd_ptr", B * H * _groups(N, block) + 1)
    _need(Q, "Q", torch.bfloat16)
    dev = Q.device
    for name, t in (("K", K), ("V", V), ("dO", dO), ("dK", outs[0]), ("dV", outs[1])):
        _need(t, name, torch.bfloat16, dev)
    for name, t in (("bwd_ptr", bwd_ptr), ("bwd_col", bwd_col)):
        _need(t, name, torch.int32, dev)
    B, H, N, d = Q.shape
    s = Shape(B, H, N, d, block, 8)
    _need(workspace, "workspace", workspace.dtype, dev)
    with torch.cuda.device(dev):
        _check(lib.dsv_attn_bwd_dkdv(_ptr(Q), _ptr(K), _ptr(V), _ptr(dO), s, _ptr(bwd_ptr), _ptr(bwd_col),
                                     float(softmax_scale), _ptr(outs[0]), _ptr(outs[1]), _ptr(workspace),
                                     _nbytes(workspace), _stream(dev, stream)), "dsv_attn_bwd_dkdv")


def attn_bwd_dq(Q, K, V, dO, fwd_ptr, fwd_col, block: int, softmax_scale: float = 0.0, *, out, workspace,
                stream=None) -> None:
    """dQ into `out` after attn_bwd_preprocess; see dsv_attn_bwd_dq."""
    B, H, N, d = _dims(Q, "Q", 4)
    for name, t in (("K", K), ("V", V), ("dO", dO), ("dQ", out)):
        _shape(t, name, (B, H, N, d))
    _room(fwd_ptr, "fwd_ptr", B * H * _groups(N, block) + 1)
    _need(Q, "Q", torch.bfloat16)
    dev = Q.device
    for name, t in (("K", K), ("V", V), ("dO", dO), ("dQ", out)):
        _need(t, name, torch.bfloat16, dev)
    for name, t in (("fwd_ptr", fwd_ptr), ("fwd_col", fwd_col)):
        _need(t, name, torch.int32, dev)
    B, H, N, d = Q.shape
    s = Shape(B, H, N, d, block, 8)
    _need(workspace, "workspace", workspace.dtype, dev)
    with torch.cuda.device(dev):
        _check(lib.dsv_attn_bwd_dq(_ptr(Q), _ptr(K), _ptr(V), _ptr(dO), s, _ptr(fwd_ptr), _ptr(fwd_col),
                                   float(softmax_scale), _ptr(out), _ptr(workspace), _nbytes(workspace),
                                   _stream(dev, stream)), "dsv_attn_bwd_dq")


# ---------------------------------------------------------------------------
# Rotary positions with several axes, and attention of packed sequences
# ---------------------------------------------------------------------------

def _scratch(nbytes: int, device, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    """`workspace`, which must be contiguous memory of this device with room for nbytes, or a new one."""
    if workspace is not None:
        _need(workspace, "workspace", workspace.dtype, device)
    return _workspace(nbytes, device, workspace)


_AS_IT_IS = contextlib.nullcontext()


def _alloc_on(stream):
    """The context in which a call launched on `stream` allocates: the allocator
    then knows the stream that uses the memory."""
    if stream is None:
        return _AS_IT_IS
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    return torch.cuda.stream(stream)


def _rows(device: torch.device, index: int, **tensors) -> Tuple[View, ...]:
    """The views of [.., heads, tokens, d] tensors (None: the null view), each
    checked as _need_rows does; index: the device's, as get_device() gives it."""
    views = _calls.row_views(torch.bfloat16, index, *tensors.values())
    if views is None:
        for name, t in tensors.items():
            if t is not None:
                _need_rows(t, name, device)
        raise ValueError("the tensors must be rows of bf16 on one device: " + ", ".join(tensors))
    return views


def _fit32(**sizes: int) -> None:
    """Sizes that the library takes as 32-bit integers (ctypes would keep their low bits)."""
    for name, v in sizes.items():
        if not -(1 << 31) <= v < 1 << 31:
            raise ValueError(f"{name} = {v} does not fit in 32 bits")


@functools.lru_cache(maxsize=64)
def _rope(B: int, H: int, N: int, d: int, sections: Tuple[int, ...], theta: float) -> Rope:
    _fit32(B=B, H=H, N=N, d=d, **{f"sections[{i}]": c for i, c in enumerate(sections)})
    return Rope(B, H, N, d, len(sections), (ctypes.c_int32 * 4)(*sections), theta)


def _rope_shape(t, name: str, pos, sections: Sequence[int], theta: float) -> Tuple[Rope, int]:
    """(dsv_rope, elements between batches of pos)."""
    B, H, N, d = _dims(t, name, 4)
    A = len(sections)
    if not 1 <= A <= 4:
        raise ValueError(f"sections has {A} entries, expected one per axis, 1 to 4")
    if not isinstance(pos, torch.Tensor):
        raise TypeError("pos must be a torch.Tensor")
    if pos.shape != (N, A) and pos.shape != (B, N, A):
        raise ValueError(f"pos has shape {tuple(pos.shape)}, expected {(N, A)} or {(B, N, A)}")
    return _rope(B, H, N, d, tuple(sections), theta), N * A if pos.dim() == 3 else 0


def rope_axes(x, pos, sections: Sequence[int], *, theta: float = 10000.0, weight=None, eps: float = 1e-6, out=None,
              stream=None) -> torch.Tensor:
    """Rotary positions with several axes, bf16 [B,H,N,d], behind the RMS norm
    of each row where a weight (fp32 [d]) is given; see dsv_rope_axes_fwd.

    sections: channels of each axis' band; pos: int32 [N, axes] or [B, N,
    axes].  x may be a view such as the transposed [B,N,H,d] of a projection:
    the last dimension contiguous, the other strides multiples of 8 elements, no
    broadcast dimension.  out may be x; without it the result has x's dimension
    order in memory."""
    r, pos_b = _rope_shape(x, "x", pos, sections, theta)
    if out is not None:
        _shape(out, "out", x.shape)
    if weight is not None:
        _shape(weight, "weight", (r.d,))
    _need_rows(x, "x")
    dev, at = x.device, x.get_device()
    _need_on(dev, at, torch.int32, pos=pos)
    if weight is not None:
        _need_on(dev, at, torch.float32, weight=weight)
    if out is None:
        with _alloc_on(stream):
            out = torch.empty_like(x)
    vx, vy = _rows(dev, at, x=x, out=out)
    _call(lib.dsv_rope_axes_fwd, "dsv_rope_axes_fwd", dev, vx, pos.data_ptr(), pos_b, r, _ptr(weight), eps, vy,
          _stream(dev, stream))
    return out


def rope_axes_bwd_workspace_bytes(d: int) -> int:
    return int(lib.dsv_rope_axes_bwd_workspace_bytes(_rope(1, 1, 1, d, (d,), 10000.0)))


def rope_axes_bwd(dy, pos, sections: Sequence[int], *, theta: float = 10000.0, x=None, weight=None, eps: float = 1e-6,
                  dx=None, dweight=None, workspace=None, stream=None):
    """Gradient of rope_axes: dx, or (dx, dweight fp32 [d]) with a weight (then
    x, the forward's input, is needed); see dsv_rope_axes_bwd.  dx may be dy or x."""
    r, pos_b = _rope_shape(dy, "dy", pos, sections, theta)
    if dx is not None:
        _shape(dx, "dx", dy.shape)
    if weight is not None:
        if x is None:
            raise ValueError("the gradient through the norm needs x")
        _shape(x, "x", dy.shape)
        _shape(weight, "weight", (r.d,))
        if dweight is not None:
            _shape(dweight, "dweight", (r.d,))
    elif dweight is not None:
        raise ValueError("dweight without a weight")
    _need_rows(dy, "dy")
    dev, at = dy.device, dy.get_device()
    _need_on(dev, at, torch.int32, pos=pos)
    nbytes, ws = 0, None
    if weight is not None:
        _need_on(dev, at, torch.float32, weight=weight, dweight=dweight)
    with _alloc_on(stream):
        if dx is None:
            dx = torch.empty_like(dy)
        if weight is not None:
            if dweight is None:
                dweight = torch.empty(r.d, dtype=torch.float32, device=dev)
            nbytes = lib.dsv_rope_axes_bwd_workspace_bytes(r)
            ws = _scratch(nbytes, dev, workspace)
    vdy, vx, vdx = _rows(dev, at, dy=dy, x=x if weight is not None else None, dx=dx)
    _call(lib.dsv_rope_axes_bwd, "dsv_rope_axes_bwd", dev, vdy, vx, pos.data_ptr(), pos_b, r, _ptr(weight), eps, vdx,
          _ptr(dweight), _ptr(ws), nbytes, _stream(dev, stream))
    return dx if weight is None else (dx, dweight)


@functools.lru_cache(maxsize=64)
def _packed(S: int, H: int, Hkv: int, Tq: int, Tk: int, d: int) -> Packed:
    _fit32(S=S, H=H, Hkv=Hkv, Tq=Tq, Tk=Tk, d=d)
    return Packed(S, H, Hkv, Tq, Tk, d)


def _packed_shape(Q, K, V, q_ptr, k_ptr) -> Packed:
    H, Tq, d = _dims(Q, "Q", 3)
    Hkv, Tk, dk = _dims(K, "K", 3)
    if dk != d:
        raise ValueError(f"K has head dimension {dk}, expected {d}")
    if Hkv < 1 or H % Hkv != 0:
        raise ValueError(f"Q has {H} heads, expected a multiple of K's {Hkv}")
    _shape(V, "V", K.shape)
    S = _dims(q_ptr, "q_ptr", 1)[0] - 1
    if S < 0:
        raise ValueError("q_ptr must hold at least one element")
    _shape(k_ptr, "k_ptr", q_ptr.shape)
    return _packed(S, H, Hkv, Tq, Tk, d)


def packed_attn_fwd_workspace_bytes(S: int, H: int, Hkv: int, Tq: int, Tk: int, d: int) -> int:
    return int(lib.dsv_packed_attn_fwd_workspace_bytes(_packed(S, H, Hkv, Tq, Tk, d)))


def packed_attn_bwd_workspace_bytes(S: int, H: int, Hkv: int, Tq: int, Tk: int, d: int) -> int:
    return int(lib.dsv_packed_attn_bwd_workspace_bytes(_packed(S, H, Hkv, Tq, Tk, d)))


def packed_attn_fwd(Q, K, V, q_ptr, k_ptr, softmax_scale: float = 0.0, *, causal: bool = False, out=None, lse=None,
                    workspace=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(O bf16 [H,Tq,d], lse fp32 [H,Tq]) of sequences packed along the token
    axis: sequence s owns the queries q_ptr[s]:q_ptr[s+1] and the keys
    k_ptr[s]:k_ptr[s+1]; see dsv_packed_attn_fwd.

    Q [H,Tq,d], K and V [Hkv,Tk,d] may be views such as transposed [T,H,d]
    projections: the last dimension contiguous, the other strides multiples of 8
    elements, no broadcast dimension.  Rows outside the sequences are not
    written: in an output that this call allocates they are uninitialised."""
    p = _packed_shape(Q, K, V, q_ptr, k_ptr)
    if out is not None:
        _shape(out, "out", Q.shape)
    if lse is not None:
        _shape(lse, "lse", (p.H, p.Tq))
    _need_rows(Q, "Q")
    dev, at = Q.device, Q.get_device()
    _need_on(dev, at, torch.int32, q_ptr=q_ptr, k_ptr=k_ptr)
    if lse is not None:
        _need_on(dev, at, torch.float32, lse=lse)
    nbytes = lib.dsv_packed_attn_fwd_workspace_bytes(p)
    with _alloc_on(stream):
        if out is None:
            out = torch.empty_like(Q)
        if lse is None:
            lse = torch.empty(p.H, p.Tq, dtype=torch.float32, device=dev)
        ws = _scratch(nbytes, dev, workspace) if nbytes else None
    vq, vk, vv, vo = _rows(dev, at, Q=Q, K=K, V=V, out=out)
    _call(lib.dsv_packed_attn_fwd, "dsv_packed_attn_fwd", dev, vq, vk, vv, p, q_ptr.data_ptr(), k_ptr.data_ptr(),
          1 if causal else 0, softmax_scale, vo, lse.data_ptr(), _ptr(ws), nbytes, _stream(dev, stream))
    return out, lse


def packed_attn_bwd(Q, K, V, O, dO, lse, q_ptr, k_ptr, softmax_scale: float = 0.0, *, causal: bool = False, outs=None,
                    workspace=None, stream=None):
    """(dQ [H,Tq,d], dK, dV [Hkv,Tk,d]) bf16 of packed_attn_fwd, from its O and
    lse; see dsv_packed_attn_bwd.  Views and rows outside the sequences as there
    (the gradient of a sum is a broadcast tensor: pass dO.contiguous())."""
    p = _packed_shape(Q, K, V, q_ptr, k_ptr)
    _shape(O, "O", Q.shape)
    _shape(dO, "dO", Q.shape)
    _shape(lse, "lse", (p.H, p.Tq))
    if outs is not None:
        if len(outs) != 3:
            raise ValueError("outs must be (dQ, dK, dV)")
        for name, t, like in zip(("dQ", "dK", "dV"), outs, (Q, K, V)):
            _shape(t, name, like.shape)
    _need_rows(Q, "Q")
    dev, at = Q.device, Q.get_device()
    _need_on(dev, at, torch.int32, q_ptr=q_ptr, k_ptr=k_ptr)
    _need_on(dev, at, torch.float32, lse=lse)
    nbytes = lib.dsv_packed_attn_bwd_workspace_bytes(p)
    with _alloc_on(stream):
        if outs is None:
            outs = (torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V))
        ws = _scratch(nbytes, dev, workspace) if nbytes else None
    vq, vk, vv, vo, vdo, vdq, vdk, vdv = _rows(dev, at, Q=Q, K=K, V=V, O=O, dO=dO, dQ=outs[0], dK=outs[1], dV=outs[2])
    _call(lib.dsv_packed_attn_bwd, "dsv_packed_attn_bwd", dev, vq, vk, vv, vo, vdo, lse.data_ptr(), p,
          q_ptr.data_ptr(), k_ptr.data_ptr(), 1 if causal else 0, softmax_scale, vdq, vdk, vdv, _ptr(ws), nbytes,
          _stream(dev, stream))
    return outs


# ---------------------------------------------------------------------------
# Layer norm, 8-bit quantiser and product
# ---------------------------------------------------------------------------

def _need_matrix(t, name: str, dtypes, device: Optional[torch.device] = None) -> None:
    """t is a 2D CUDA tensor of one of the dtypes with contiguous rows; the library checks its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.stride(1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


# The current device's index without the checks around it.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _ready(x, stream) -> int:
    """The device of x where a call can go out at once: the current device's, on its current stream; else -1.  The
    C module then checks the arguments; where it does not take them, the checks below say why."""
    if stream is None and Rows is not None and _raw_stream is not None and isinstance(x, torch.Tensor):
        at = x.get_device()
        if at >= 0 and x.dim() == 2 and at == _current_device():
            return at
    return -1


_BF16, _REAL, _FP8 = (torch.bfloat16,), (torch.bfloat16, torch.float32), (torch.float8_e4m3fn, torch.float8_e5m2)


def _matrices(device: torch.device, index: int, **tensors):
    """dsv_rows of (tensor, its allowed dtypes) pairs (a None tensor: null)."""
    for name, (t, dtypes) in tensors.items():
        if t is not None and t.dtype not in dtypes:
            _need_matrix(t, name, dtypes, device)
    rows = _calls.matrices(index, *[t for t, _ in tensors.values()])
    if rows is None:
        for name, (t, dtypes) in tensors.items():
            if t is not None:
                _need_matrix(t, name, dtypes, device)
        raise ValueError("the tensors must be matrices on one device: " + ", ".join(tensors))
    return rows


@functools.lru_cache(maxsize=64)
def _norm(T: int, C: int, S: int, eps: float) -> Norm:
    _fit32(T=T, C=C, S=S)
    return Norm(T, C, S, eps)


def _norm_shape(x, weight, seq_ptr, eps: float) -> Norm:
    T, C = _dims(x, "x", 2)
    S = 1
    if seq_ptr is not None:
        S = _dims(seq_ptr, "seq_ptr", 1)[0] - 1
        if S < 0:
            raise ValueError("seq_ptr must hold at least one element")
        if weight is not None:
            _shape(weight, "weight", (S, C))
    elif weight is not None:
        if not isinstance(weight, torch.Tensor):
            raise TypeError("weight must be a torch.Tensor")
        if weight.dim() == 2:
            S = weight.shape[0]
            _shape(weight, "weight", (S, C))
            if S < 1 or T % S != 0:
                raise ValueError(f"{T} rows do not divide into {S} sequences of equal lengths: pass seq_ptr")
        else:
            _shape(weight, "weight", (C,))
    return _norm(T, C, S, eps)


def layer_norm(x, weight=None, bias=None, seq_ptr=None, *, eps: float = 1e-6, out=None, stats=None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(y bf16 [T,C], stats fp32 [2,T]: mean, 1/deviation) of the rows of x, bf16
    or fp32 [T,C] with any row stride; see dsv_layer_norm_fwd.

    weight and bias: fp32 [C], or [S,C] with a row for each sequence: sequence s
    owns the rows seq_ptr[s]:seq_ptr[s+1] (int32 [S+1]), or without seq_ptr the
    s-th part of T/S rows.  Rows outside the sequences are not written: in an
    output that this call allocates they are uninitialised.  out may be x."""
    at = _ready(x, stream)
    if at >= 0:
        T, C = x.shape
        y = torch.empty(T, C, dtype=torch.bfloat16, device=x.device) if out is None else out
        kept = torch.empty(2, T, dtype=torch.float32, device=x.device) if stats is None else stats
        st = _calls.norm_fwd(x, weight, bias, seq_ptr, eps, y, kept, at, _raw_stream(at))
        if st is not None:
            _check(st, "dsv_layer_norm_fwd")
            return y, kept
    p = _norm_shape(x, weight, seq_ptr, eps)
    if bias is not None:
        if weight is None:
            raise ValueError("bias without a weight")
        _shape(bias, "bias", weight.shape)
    if out is not None:
        _shape(out, "out", x.shape)
    if stats is not None:
        _shape(stats, "stats", (2, p.T))
    _need_matrix(x, "x", _REAL)
    dev, at = x.device, x.get_device()
    _need_on(dev, at, torch.float32, weight=weight, bias=bias, stats=stats)
    if seq_ptr is not None:
        _need_on(dev, at, torch.int32, seq_ptr=seq_ptr)
    with _alloc_on(stream):
        if out is None:
            out = torch.empty(p.T, p.C, dtype=torch.bfloat16, device=dev)
        if stats is None:
            stats = torch.empty(2, p.T, dtype=torch.float32, device=dev)
    vx, vy = _matrices(dev, at, x=(x, _REAL), out=(out, _BF16))
    _call(lib.dsv_layer_norm_fwd, "dsv_layer_norm_fwd", dev, vx, p, _ptr(seq_ptr), _ptr(weight), _ptr(bias), vy,
          stats.data_ptr(), _stream(dev, stream))
    return out, stats


def layer_norm_bwd_workspace_bytes(T: int, C: int, S: int = 1) -> int:
    return int(lib.dsv_layer_norm_bwd_workspace_bytes(_norm(T, C, S, 1e-6)))


def layer_norm_bwd(dy, x, stats, weight=None, seq_ptr=None, *, dx=None, dweight=None, dbias=None, workspace=None,
                   stream=None):
    """Gradient of layer_norm from its input x and stats: dx (x's type), or with a
    weight (dx, dweight, dbias fp32 of the weight's shape); see
    dsv_layer_norm_bwd.  dx may be dy or x."""
    at = _ready(x, stream)
    if at >= 0 and workspace is None and (weight is not None or (dweight is None and dbias is None)):
        dev, dw, db, ws = x.device, dweight, dbias, None
        nbytes = 0 if weight is None else _calls.norm_bwd_bytes(x, weight, seq_ptr, at)
        if nbytes is not None:
            to = torch.empty(x.shape, dtype=x.dtype, device=dev) if dx is None else dx
            if weight is not None:
                ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
                dw = torch.empty(weight.shape, dtype=torch.float32, device=dev) if dw is None else dw
                db = torch.empty(weight.shape, dtype=torch.float32, device=dev) if db is None else db
            st = _calls.norm_bwd(dy, x, stats, weight, seq_ptr, to, dw, db, _ptr(ws), nbytes, at, _raw_stream(at))
            if st is not None:
                _check(st, "dsv_layer_norm_bwd")
                return to if weight is None else (to, dw, db)
    p = _norm_shape(x, weight, seq_ptr, 1e-6)
    _shape(dy, "dy", x.shape)
    _shape(stats, "stats", (2, p.T))
    if dx is not None:
        _shape(dx, "dx", x.shape)
    for name, t in (("dweight", dweight), ("dbias", dbias)):
        if t is not None:
            if weight is None:
                raise ValueError(f"{name} without a weight")
            _shape(t, name, weight.shape)
    _need_matrix(x, "x", _REAL)
    dev, at = x.device, x.get_device()
    _need_on(dev, at, torch.float32, stats=stats, weight=weight, dweight=dweight, dbias=dbias)
    if seq_ptr is not None:
        _need_on(dev, at, torch.int32, seq_ptr=seq_ptr)
    nbytes, ws = 0, None
    with _alloc_on(stream):
        if dx is None:
            dx = torch.empty(p.T, p.C, dtype=x.dtype, device=dev)
        if weight is not None:
            if dweight is None:
                dweight = torch.empty(weight.shape, dtype=torch.float32, device=dev)
            if dbias is None:
                dbias = torch.empty(weight.shape, dtype=torch.float32, device=dev)
            nbytes = lib.dsv_layer_norm_bwd_workspace_bytes(p)
            ws = _scratch(nbytes, dev, workspace)
    vdy, vx, vdx = _matrices(dev, at, dy=(dy, _BF16), x=(x, _REAL), dx=(dx, (x.dtype,)))
    _call(lib.dsv_layer_norm_bwd, "dsv_layer_norm_bwd", dev, vdy, vx, stats.data_ptr(), p, _ptr(seq_ptr), _ptr(weight),
          vdx, _ptr(dweight), _ptr(dbias), _ptr(ws), nbytes, _stream(dev, stream))
    return dx if weight is None else (dx, dweight, dbias)


def _fp8_matrix(R: int, C: int, dtype: torch.dtype, device) -> torch.Tensor:
    """[R, C] with rows a multiple of 16 bytes apart."""
    t = torch.empty(R, (C + 15) // 16 * 16, dtype=dtype, device=device)
    return t if C % 16 == 0 else t[:, :C]


def quantize_fp8(x, *, rows: int = 1, transpose: bool = False, dtype: torch.dtype = torch.float8_e4m3fn, outs=None,
                 stream=None):
    """(q, scale) of x, bf16 or fp32 [R,C] with any row stride: 8-bit floating
    point with a power-of-two scale for each block of 128 columns of one row
    (rows=1) or of 128 rows (rows=128); see dsv_quantize_fp8.

    q [R,C] of `dtype` (float8_e4m3fn or float8_e5m2), its rows a multiple of 16
    bytes apart; scale fp32 [ceil(C/128), R] or [ceil(C/128), ceil(R/128)].  With
    transpose (q, scale, qt, scale_t): also the transposed matrix [C,R] with its
    own blocks along R.  outs: those tensors."""
    at = _ready(x, stream)
    if at >= 0 and outs is None and dtype in _FP8 and (rows == 1 or rows == 128):
        (R, C), dev = x.shape, x.device
        cb, rb = (C + 127) // 128, (R + 127) // 128
        q = _fp8_matrix(R, C, dtype, dev)
        scale = torch.empty(cb, R if rows == 1 else rb, dtype=torch.float32, device=dev)
        qt = scale_t = None
        if transpose:
            qt = _fp8_matrix(C, R, dtype, dev)
            scale_t = torch.empty(rb, C if rows == 1 else cb, dtype=torch.float32, device=dev)
        st = _calls.quantize(x, rows, q, scale, qt, scale_t, at, _raw_stream(at))
        if st is not None:
            _check(st, "dsv_quantize_fp8")
            return (q, scale, qt, scale_t) if transpose else (q, scale)
    R, C = _dims(x, "x", 2)
    if rows not in (1, 128):
        raise ValueError(f"rows is {rows}, expected 1 or 128")
    if dtype not in _FP8:
        raise TypeError(f"dtype must be {_FP8[0]} or {_FP8[1]}, got {dtype}")
    cb, rb = (C + 127) // 128, (R + 127) // 128
    shapes = ((R, C), (cb, R if rows == 1 else rb), (C, R), (rb, C if rows == 1 else cb))
    if outs is not None:
        names = ("q", "scale", "qt", "scale_t")[:4 if transpose else 2]
        if len(outs) != len(names):
            raise ValueError(f"outs must be ({', '.join(names)})")
        for name, t, shape in zip(names, outs, shapes):
            _shape(t, name, shape)
    _need_matrix(x, "x", _REAL)
    dev, at = x.device, x.get_device()
    if outs is None:
        with _alloc_on(stream):
            outs = (_fp8_matrix(R, C, dtype, dev), torch.empty(shapes[1], dtype=torch.float32, device=dev))
            if transpose:
                outs += (_fp8_matrix(C, R, dtype, dev), torch.empty(shapes[3], dtype=torch.float32, device=dev))
    qt, scale_t = (outs[2], outs[3]) if transpose else (None, None)
    _need_on(dev, at, torch.float32, scale=outs[1], scale_t=scale_t)
    vx, vq, vqt = _matrices(dev, at, x=(x, _REAL), q=(outs[0], (dtype,)), qt=(qt, (dtype,)))
    _call(lib.dsv_quantize_fp8, "dsv_quantize_fp8", dev, vx, R, C, rows, vq, outs[1].data_ptr(), vqt, _ptr(scale_t),
          _stream(dev, stream))
    return outs


@functools.lru_cache(maxsize=64)
def _matmul(M: int, N: int, K: int, a_rows: int, b_rows: int, accumulate: int) -> Matmul:
    _fit32(M=M, N=N, K=K)
    return Matmul(M, N, K, a_rows, b_rows, accumulate)


def _scale_rows(scale, name: str, R: int, K: int) -> int:
    """The rows of a block that the scale's shape stands for."""
    kb, got = (K + 127) // 128, _dims(scale, name, 2)
    for rows in (1, 128):
        if got == (kb, -(-R // rows)):
            return rows
    raise ValueError(f"{name} has shape {got}, expected {(kb, R)} or {(kb, -(-R // 128))}")


def matmul_fp8(a, a_scale, b, b_scale, *, out_dtype: torch.dtype = torch.bfloat16, out=None, accumulate: bool = False,
               stream=None) -> torch.Tensor:
    """[M,N] = a b^T of 8-bit matrices a [M,K] and b [N,K] as quantize_fp8 makes
    them (e4m3 or e5m2 each, rows a multiple of 16 bytes apart) with fp32 scales
    [ceil(K/128), rows] or [ceil(K/128), ceil(rows/128)]; see dsv_matmul_fp8.

    out_dtype: bf16 or fp32, or that of `out` [M,N] (any row stride).
    accumulate: adds to `out` (fp32).  A projection y = x w^T and its gradients:
        y  = matmul_fp8(*quantize_fp8(x), *quantize_fp8(w, rows=128))
        dx = matmul_fp8(*quantize_fp8(dy), wt, wt_scale)          # w's transposed copy
        dw = matmul_fp8(dyt, dyt_scale, xt, xt_scale)             # both transposed copies"""
    at = _ready(a, stream)
    if at >= 0 and isinstance(b, torch.Tensor) and b.dim() == 2 and out_dtype in _REAL and (out is not None or not accumulate):
        c = torch.empty(a.shape[0], b.shape[0], dtype=out_dtype, device=a.device) if out is None else out
        st = _calls.matmul(a, a_scale, b, b_scale, c, 1 if accumulate else 0, at, _raw_stream(at))
        if st is not None:
            _check(st, "dsv_matmul_fp8")
            return c
    M, K = _dims(a, "a", 2)
    N, Kb = _dims(b, "b", 2)
    if Kb != K:
        raise ValueError(f"b has {Kb} columns, expected {K}")
    p = _matmul(M, N, K, _scale_rows(a_scale, "a_scale", M, K), _scale_rows(b_scale, "b_scale", N, K),
                1 if accumulate else 0)
    if out is not None:
        _shape(out, "out", (M, N))
        out_dtype = out.dtype
    elif accumulate:
        raise ValueError("accumulate needs out")
    if out_dtype not in _REAL:
        raise TypeError(f"out must be {_REAL[0]} or {_REAL[1]}, got {out_dtype}")
    if accumulate and out_dtype != torch.float32:
        raise TypeError("accumulate needs an fp32 out")
    _need_matrix(a, "a", _FP8)
    dev, at = a.device, a.get_device()
    _need_on(dev, at, torch.float32, a_scale=a_scale, b_scale=b_scale)
    if out is None:
        with _alloc_on(stream):
            out = torch.empty(M, N, dtype=out_dtype, device=dev)
    va, vb, vc = _matrices(dev, at, a=(a, _FP8), b=(b, _FP8), out=(out, (out_dtype,)))
    _call(lib.dsv_matmul_fp8, "dsv_matmul_fp8", dev, va, a_scale.data_ptr(), vb, b_scale.data_ptr(), p, vc,
          _stream(dev, stream))
    return out


# ---------------------------------------------------------------------------
# Device-side error word
# ---------------------------------------------------------------------------

def device_error(stream=None, device=None) -> Tuple[int, int]:
    """(status, info) recorded by the kernels on the current device; synchronises."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    info = ctypes.c_uint32(0)
    st = lib.dsv_get_device_error(_stream(dev, stream), ctypes.byref(info))
    return st, info.value


def clear_device_error(stream=None, device=None) -> None:
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    _check(lib.dsv_clear_device_error(_stream(dev, stream)), "dsv_clear_device_error")


def set_wait_limit_ns(limit_ns: int) -> None:
    _check(lib.dsv_set_wait_limit_ns(int(limit_ns)), "dsv_set_wait_limit_ns")



def selftest_wait_timeout(stream=None, device=None) -> None:
    """Enqueue the library's failure-detection self-test: a kernel whose only
    wait can never be satisfied runs out of its time limit (set_wait_limit_ns)
    and records DSV_ERR_TIMEOUT; read it with device_error()."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    _check(lib.dsv_selftest_wait_timeout(_stream(dev, stream)), "dsv_selftest_wait_timeout")


def dispatch_heads(k_per_head: Sequence[int], nb: int, rho: Sequence[float], ratio: Sequence[float]):
    """The OP dispatcher (host-only): per head, dense (k = nb) when the profile's
    sparse/dense time ratio at the head's kept fraction is >= 1, else sparse.
    Returns (k_out, dense) as lists; see dsv_dispatch_heads."""
    H, n = len(k_per_head), len(rho)
    if len(ratio) != n:
        raise ValueError("rho and ratio must have the same length")
    karr = (ctypes.c_int32 * max(H, 1))(*[int(k) for k in k_per_head])
    rarr = (ctypes.c_float * max(n, 1))(*[float(v) for v in rho])
    qarr = (ctypes.c_float * max(n, 1))(*[float(v) for v in ratio])
    kout = (ctypes.c_int32 * max(H, 1))()
    dout = (ctypes.c_int32 * max(H, 1))()
    _check(lib.dsv_dispatch_heads(karr, H, int(nb), rarr, qarr, n, kout, dout), "dsv_dispatch_heads")
    return [int(kout[h]) for h in range(H)], [bool(dout[h]) for h in range(H)]
