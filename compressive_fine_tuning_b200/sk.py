"""Thin Python binding of libsk.so (the sketched linear layer's C ABI).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  Importing
this module fails loudly when the library has not been built; there is no
fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsk.so")

SK_OK = 0
SK_OP_FWD, SK_OP_BWD_INPUT, SK_OP_BWD_LUT, SK_OP_BWD_LUT_CKPT8 = 0, 1, 2, 3
SK_F32, SK_BF16, SK_F16 = 0, 1, 2
SK_CE_NONE, SK_CE_MEAN, SK_CE_SUM = 0, 1, 2
SK_CHECK_TASK_RANGE = 1
SK_CHECK_INDEX_RANGE = 2
SK_CHECK_TIMEOUT = 4
SK_CHECK_NOT_SPD = 8
SK_CHECK_LUT_ORDER = 16
SK_CHECK_TARGET_RANGE = 32

EXPORTED = (
    "sk_abi_version", "sk_status_string", "sk_last_error", "sk_packed_row_bytes", "sk_packed_bytes",
    "sk_pack", "sk_unpack", "sk_dequant", "sk_workspace_bytes", "sk_linear_fwd", "sk_linear_fwd_group",
    "sk_linear_bwd_input",
    "sk_linear_bwd_lut", "sk_linear_bwd_lut_noalloc", "sk_bin_counts", "sk_lut_adamw", "sk_lut_sgd",
    "sk_device_check", "sk_inverse_factor_workspace_bytes", "sk_sketch_round_workspace_bytes", "sk_gram",
    "sk_inverse_factor", "sk_lloyd", "sk_sketch_round",
    "sk_ckpt8_quantize", "sk_ckpt8_dequantize", "sk_linear_bwd_lut_ckpt8",
    "sk_layer_norm_bwd_workspace_bytes", "sk_layer_norm_fwd", "sk_layer_norm_bwd",
    "sk_cross_entropy_workspace_bytes", "sk_cross_entropy", "sk_scale_bf16",
)


SK_MAX_GROUP_LAYERS = 8


class _Layer(ctypes.Structure):
    """sk_layer of sk.h: one layer of a grouped forward."""
    _fields_ = [("packed", ctypes.c_void_p), ("lut", ctypes.c_void_p), ("gpr", ctypes.c_int),
                ("n", ctypes.c_int64), ("d", ctypes.c_int64), ("X", ctypes.c_void_p), ("Y", ctypes.c_void_p)]


class SketchError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with `python -m compressive_fine_tuning_b200.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i64, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    f64 = ctypes.c_double
    sigs = {
        "sk_abi_version": ([], i32),
        "sk_status_string": ([i32], ctypes.c_char_p),
        "sk_last_error": ([], ctypes.c_char_p),
        "sk_packed_row_bytes": ([i64, i32], sz),
        "sk_packed_bytes": ([i64, i64, i32], sz),
        "sk_pack": ([vp, i64, i64, i32, vp, sz, vp], i32),
        "sk_unpack": ([vp, i64, i64, i32, vp, vp], i32),
        "sk_dequant": ([vp, vp, i32, i32, i64, i64, i32, i32, vp, vp], i32),
        "sk_workspace_bytes": ([i32, i64, i64, i32, i32, i64, i32], sz),
        "sk_linear_fwd": ([vp, vp, i32, i32, i64, i64, vp, i64, vp, i32, vp, vp, sz, vp], i32),
        "sk_linear_fwd_group": ([ctypes.POINTER(_Layer), i32, i32, i64, vp, i32, vp], i32),
        "sk_linear_bwd_input": ([vp, vp, i32, i32, i64, i64, vp, i64, vp, i32, vp, vp, sz, vp], i32),
        "sk_linear_bwd_lut": ([vp, i32, i32, i64, i64, vp, vp, i64, vp, i32, vp, i32, vp, sz, vp], i32),
        "sk_linear_bwd_lut_noalloc": ([vp, i32, i32, i64, i64, vp, vp, i64, vp, i32, vp, i32, vp], i32),
        "sk_bin_counts": ([vp, i32, i32, i64, i64, vp, vp], i32),
        "sk_lut_adamw": ([vp, vp, vp, vp, vp, i32, i64, i32, i32, f32, f32, f32, f32, f32, i32, vp, vp], i32),
        "sk_lut_sgd": ([vp, vp, vp, i32, i64, i32, i32, f32, vp, vp], i32),
        "sk_device_check": ([ctypes.POINTER(ctypes.c_uint32), i32, vp], i32),
        "sk_inverse_factor_workspace_bytes": ([i64], sz),
        "sk_sketch_round_workspace_bytes": ([i64, i64], sz),
        "sk_gram": ([vp, i64, i64, vp, i32, vp], i32),
        "sk_inverse_factor": ([vp, i64, f64, vp, vp, vp, sz, vp], i32),
        "sk_lloyd": ([vp, vp, i32, i32, i64, i64, i32, vp, vp, vp], i32),
        "sk_sketch_round": ([vp, vp, vp, i32, i32, i64, i64, vp, vp, sz, vp], i32),
        "sk_ckpt8_quantize": ([vp, i64, i64, vp, vp, vp], i32),
        "sk_ckpt8_dequantize": ([vp, vp, i64, i64, vp, vp], i32),
        "sk_linear_bwd_lut_ckpt8": ([vp, i32, i32, i64, i64, vp, vp, vp, i64, vp, i32, vp, i32, vp, sz, vp], i32),
        "sk_layer_norm_bwd_workspace_bytes": ([i64, i64], sz),
        "sk_layer_norm_fwd": ([vp, i32, i64, i64, vp, vp, i32, f32, i32, vp, vp, vp, vp, vp, vp], i32),
        "sk_layer_norm_bwd": ([vp, vp, i32, i64, i64, vp, i32, vp, vp, i32, vp, vp, vp, vp, sz, vp], i32),
        "sk_cross_entropy_workspace_bytes": ([i64, i64, i64, i32, i32], sz),
        "sk_cross_entropy": ([vp, vp, vp, i32, i64, i64, i64, i64, i32, vp, vp, vp, vp, vp, sz, vp], i32),
        "sk_scale_bf16": ([vp, i64, vp, i64, vp, vp], i32),
    }
    for name, (args, res) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


lib = _load()


def _check(status: int) -> None:
    if status != SK_OK:
        name = lib.sk_status_string(status).decode()
        raise SketchError(status, f"{name}: {lib.sk_last_error().decode()}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# the current stream's handle without building a Stream object (2 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device):
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _need(t: torch.Tensor, dtype: torch.dtype, name: str, ndim: Optional[int] = None) -> None:
    if (isinstance(t, torch.Tensor) and t.dtype == dtype and t.is_cuda and t.is_contiguous()
            and (ndim is None or t.dim() == ndim)):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


def packed_row_bytes(d: int, bits: int) -> int:
    return int(lib.sk_packed_row_bytes(d, bits))


def packed_bytes(n: int, d: int, bits: int) -> int:
    return int(lib.sk_packed_bytes(n, d, bits))


def workspace_bytes(op: int, n: int, d: int, bits: int, gpr: int, T: int, ntask: int) -> int:
    return int(lib.sk_workspace_bytes(op, n, d, bits, gpr, T, ntask))


def _workspace(op, n, d, bits, gpr, T, ntask, device):
    nb = workspace_bytes(op, n, d, bits, gpr, T, ntask)
    if nb == 0:
        return None, 0
    return torch.empty(nb, dtype=torch.uint8, device=device), nb


def pack(idx: torch.Tensor, bits: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """uint8 [n, d] indices -> uint8 [n, packed_row_bytes] packed rows (on the GPU)."""
    _need(idx, torch.uint8, "idx", 2)
    n, d = idx.shape
    rb = packed_row_bytes(d, bits)
    if out is None:
        out = torch.empty((n, max(rb, 1)), dtype=torch.uint8, device=idx.device)
    _need(out, torch.uint8, "out")
    _check(lib.sk_pack(_ptr(idx), n, d, bits, _ptr(out), out.numel(), _stream(idx.device)))
    return out


def unpack(packed: torch.Tensor, n: int, d: int, bits: int) -> torch.Tensor:
    _need(packed, torch.uint8, "packed")
    out = torch.empty((n, d), dtype=torch.uint8, device=packed.device)
    _check(lib.sk_unpack(_ptr(packed), n, d, bits, _ptr(out), _stream(packed.device)))
    return out


def _lut_shape(lut: torch.Tensor, bits: int):
    _need(lut, torch.float16, "lut", 4)
    ntask, n, gpr, k = lut.shape
    if k != (1 << bits):
        raise ValueError(f"lut's last dimension must be 2**bits = {1 << bits}")
    return ntask, n, gpr


def dequant(packed: torch.Tensor, lut: torch.Tensor, bits: int, d: int, task: int = 0) -> torch.Tensor:
    """Dense bf16 [n, d] effective weight of LUT set `task` (test / comparison aid)."""
    ntask, n, gpr = _lut_shape(lut, bits)
    _need(packed, torch.uint8, "packed")
    out = torch.empty((n, d), dtype=torch.bfloat16, device=lut.device)
    _check(lib.sk_dequant(_ptr(packed), _ptr(lut), bits, gpr, n, d, task, ntask, _ptr(out), _stream(lut.device)))
    return out


def _task_arg(task: Optional[torch.Tensor], T: int):
    if task is None:
        return None
    _need(task, torch.int32, "task", 1)
    if task.numel() != T:
        raise ValueError("task must hold one id per token")
    return task


def linear_fwd(packed: torch.Tensor, lut: torch.Tensor, bits: int, X: torch.Tensor,
               task: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y [T, n] = X Theta_hat^T (bf16 in, bf16 out, fp32 accumulation)."""
    ntask, n, gpr = _lut_shape(lut, bits)
    _need(X, torch.bfloat16, "X", 2)
    _need(packed, torch.uint8, "packed")
    T, d = X.shape
    task = _task_arg(task, T)
    if out is None:
        out = torch.empty((T, n), dtype=torch.bfloat16, device=X.device)
    _need(out, torch.bfloat16, "out", 2)
    ws, nb = _workspace(SK_OP_FWD, n, d, bits, gpr, T, ntask, X.device)
    _check(lib.sk_linear_fwd(_ptr(packed), _ptr(lut), bits, gpr, n, d, _ptr(X), T, _ptr(task), ntask,
                             _ptr(out), _ptr(ws), nb, _stream(X.device)))
    return out


def linear_fwd_group(layers, bits: int, task: Optional[torch.Tensor] = None, outs=None):
    """Y_l = X_l Theta_hat_l^T for a list of layers (packed, lut, X) that see the
    same number of tokens, in one library call (one launch at decode sizes).
    Returns the list of Y_l; `outs` may give them."""
    if not 1 <= len(layers) <= SK_MAX_GROUP_LAYERS:
        raise ValueError(f"1 to {SK_MAX_GROUP_LAYERS} layers per group")
    arr = (_Layer * len(layers))()
    T = None
    ntask = None
    ys = []
    for i, (packed, lut, X) in enumerate(layers):
        nt, n, gpr = _lut_shape(lut, bits)
        _need(X, torch.bfloat16, "X", 2)
        _need(packed, torch.uint8, "packed")
        if T is None:
            T, ntask = X.shape[0], nt
        elif X.shape[0] != T or nt != ntask:
            raise ValueError("every layer of a group must see the same tokens and LUT sets")
        Y = outs[i] if outs is not None else torch.empty((T, n), dtype=torch.bfloat16, device=X.device)
        _need(Y, torch.bfloat16, "out", 2)
        ys.append(Y)
        arr[i] = _Layer(packed.data_ptr(), lut.data_ptr(), gpr, n, X.shape[1], X.data_ptr(), Y.data_ptr())
    task = _task_arg(task, T)
    _check(lib.sk_linear_fwd_group(arr, len(layers), bits, T, _ptr(task), ntask, _stream(layers[0][2].device)))
    return ys


def linear_bwd_input(packed: torch.Tensor, lut: torch.Tensor, bits: int, d: int, dY: torch.Tensor,
                     task: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dX [T, d] = dY Theta_hat."""
    ntask, n, gpr = _lut_shape(lut, bits)
    _need(dY, torch.bfloat16, "dY", 2)
    _need(packed, torch.uint8, "packed")
    T = dY.shape[0]
    if dY.shape[1] != n:
        raise ValueError("dY must be [T, n]")
    task = _task_arg(task, T)
    if out is None:
        out = torch.empty((T, d), dtype=torch.bfloat16, device=dY.device)
    _need(out, torch.bfloat16, "out", 2)
    ws, nb = _workspace(SK_OP_BWD_INPUT, n, d, bits, gpr, T, ntask, dY.device)
    _check(lib.sk_linear_bwd_input(_ptr(packed), _ptr(lut), bits, gpr, n, d, _ptr(dY), T, _ptr(task), ntask,
                                   _ptr(out), _ptr(ws), nb, _stream(dY.device)))
    return out


def linear_bwd_lut(packed: torch.Tensor, bits: int, gpr: int, X: torch.Tensor, dY: torch.Tensor,
                   task: Optional[torch.Tensor] = None, ntask: int = 1, out: Optional[torch.Tensor] = None,
                   accumulate: bool = False) -> torch.Tensor:
    """dlut [ntask, n, gpr, k] fp32: the binned dY^T X of the corrected Eq. 6."""
    _need(X, torch.bfloat16, "X", 2)
    _need(dY, torch.bfloat16, "dY", 2)
    _need(packed, torch.uint8, "packed")
    T, d = X.shape
    n = dY.shape[1]
    if dY.shape[0] != T:
        raise ValueError("X and dY must have the same number of tokens")
    task = _task_arg(task, T)
    k = 1 << bits
    if out is None:
        out = torch.empty((ntask, n, gpr, k), dtype=torch.float32, device=X.device)
    _need(out, torch.float32, "out")
    ws, nb = _workspace(SK_OP_BWD_LUT, n, d, bits, gpr, T, ntask, X.device)
    _check(lib.sk_linear_bwd_lut(_ptr(packed), bits, gpr, n, d, _ptr(X), _ptr(dY), T, _ptr(task), ntask,
                                 _ptr(out), int(accumulate), _ptr(ws), nb, _stream(X.device)))
    return out


def device_check(clear: bool = True, device=None) -> int:
    """Synchronise and return the device check word (SK_CHECK_* bits)."""
    device = torch.device("cuda") if device is None else torch.device(device)
    flags = ctypes.c_uint32(0)
    st = lib.sk_device_check(ctypes.byref(flags), int(clear), _stream(device))
    if st not in (SK_OK, 4):
        _check(st)
    return int(flags.value)


def bin_counts(packed: torch.Tensor, bits: int, gpr: int, n: int, d: int) -> torch.Tensor:
    """Static bin sizes counts[i][g][c] of the index map (int32 [n, gpr, 2^bits])."""
    _need(packed, torch.uint8, "packed")
    out = torch.empty((n, gpr, 1 << bits), dtype=torch.int32, device=packed.device)
    _check(lib.sk_bin_counts(_ptr(packed), bits, gpr, n, d, _ptr(out), _stream(packed.device)))
    return out


def _lut_update_shape(master: torch.Tensor, bits: int):
    if master.dtype != torch.float32 or master.dim() != 4 or master.shape[-1] != (1 << bits) or not master.is_contiguous():
        raise ValueError("master LUTs must be contiguous fp32 [ntask, n, gpr, 2^bits]")
    return master.shape[0], master.shape[1], master.shape[2]


def lut_adamw_(master: torch.Tensor, m: torch.Tensor, v: torch.Tensor, grad: torch.Tensor, bits: int, step: int,
               lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
               counts: Optional[torch.Tensor] = None, lut: Optional[torch.Tensor] = None) -> None:
    """One AdamW step on fp32 master LUTs (in place); writes the fp16 LUTs when given.
    counts (from bin_counts) selects the averaging variant of the gradient."""
    ntask, n, gpr = _lut_update_shape(master, bits)
    for t, name in ((m, "m"), (v, "v"), (grad, "grad")):
        if t.shape != master.shape or t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError(f"{name} must match the master LUTs")
    if lut is not None and (lut.shape != master.shape or lut.dtype != torch.float16 or not lut.is_contiguous()):
        raise ValueError("lut must be contiguous fp16 of the master's shape")
    _check(lib.sk_lut_adamw(_ptr(master), _ptr(m), _ptr(v), _ptr(grad), _ptr(counts), ntask, n, gpr, bits, lr, beta1,
                            beta2, eps, weight_decay, step, _ptr(lut), _stream(master.device)))


def lut_sgd_(master: torch.Tensor, grad: torch.Tensor, bits: int, lr: float, counts: Optional[torch.Tensor] = None,
             lut: Optional[torch.Tensor] = None) -> None:
    """One SGD step on fp32 master LUTs (in place); writes the fp16 LUTs when given."""
    ntask, n, gpr = _lut_update_shape(master, bits)
    if grad.shape != master.shape or grad.dtype != torch.float32 or not grad.is_contiguous():
        raise ValueError("grad must match the master LUTs")
    if lut is not None and (lut.shape != master.shape or lut.dtype != torch.float16 or not lut.is_contiguous()):
        raise ValueError("lut must be contiguous fp16 of the master's shape")
    _check(lib.sk_lut_sgd(_ptr(master), _ptr(grad), _ptr(counts), ntask, n, gpr, bits, lr, _ptr(lut),
                          _stream(master.device)))


# ---------------------------------------------------------------------------
# Sketching stage: dense weight + calibration activations -> index map + LUTs
# ---------------------------------------------------------------------------

def gram(X: torch.Tensor, H: Optional[torch.Tensor] = None, accumulate: bool = False) -> torch.Tensor:
    """H = X^T X (fp32 [d, d]) of bf16 calibration activations X [s, d];
    H += X^T X when accumulate."""
    _need(X, torch.bfloat16, "X", 2)
    s, d = X.shape
    if H is None:
        H = torch.empty((d, d), dtype=torch.float32, device=X.device)
    _need(H, torch.float32, "H", 2)
    _check(lib.sk_gram(_ptr(X), s, d, _ptr(H), int(accumulate), _stream(X.device)))
    return H


def inverse_factor(H: torch.Tensor, damp: float = 0.01):
    """(U, hinv_diag): the upper factor U of the damped H^-1 (H^-1 = U^T U,
    float64 [d, d]) and the diagonal of H^-1 (float64 [d])."""
    _need(H, torch.float32, "H", 2)
    d = H.shape[0]
    U = torch.empty((d, d), dtype=torch.float64, device=H.device)
    hd = torch.empty(d, dtype=torch.float64, device=H.device)
    nb = int(lib.sk_inverse_factor_workspace_bytes(d))
    ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=H.device)
    _check(lib.sk_inverse_factor(_ptr(H), d, float(damp), _ptr(U), _ptr(hd), _ptr(ws), nb, _stream(H.device)))
    return U, hd


def lloyd(theta: torch.Tensor, hinv_diag: torch.Tensor, bits: int, gpr: int, max_iter: int = 100):
    """(lut fp16 [n, gpr, 2^bits], updates run int32 [n, gpr]): weighted
    Lloyd's centroids of every (row, group) of theta (fp32 [n, d])."""
    _need(theta, torch.float32, "theta", 2)
    _need(hinv_diag, torch.float64, "hinv_diag", 1)
    n, d = theta.shape
    lut = torch.empty((n, gpr, 1 << bits), dtype=torch.float16, device=theta.device)
    iters = torch.empty((n, gpr), dtype=torch.int32, device=theta.device)
    _check(lib.sk_lloyd(_ptr(theta), _ptr(hinv_diag), bits, gpr, n, d, max_iter, _ptr(lut), _ptr(iters),
                        _stream(theta.device)))
    return lut, iters


def sketch_round(theta: torch.Tensor, U: torch.Tensor, lut: torch.Tensor, bits: int) -> torch.Tensor:
    """Index map (uint8 [n, d]) of theta against the ascending fp16 LUTs
    [n, gpr, 2^bits], with error compensation through U."""
    _need(theta, torch.float32, "theta", 2)
    _need(U, torch.float64, "U", 2)
    _need(lut, torch.float16, "lut", 3)
    n, d = theta.shape
    gpr = lut.shape[1]
    idx = torch.empty((n, d), dtype=torch.uint8, device=theta.device)
    nb = int(lib.sk_sketch_round_workspace_bytes(n, d))
    ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=theta.device)
    _check(lib.sk_sketch_round(_ptr(theta), _ptr(U), _ptr(lut), bits, gpr, n, d, _ptr(idx), _ptr(ws), nb,
                               _stream(theta.device)))
    return idx


def sketch_layer(theta: torch.Tensor, X: torch.Tensor, bits: int, gpr: int, damp: float = 0.01,
                 max_iter: int = 100, H: Optional[torch.Tensor] = None):
    """The sketching stage of one layer: (packed index map, fp16 LUTs
    [n, gpr, 2^bits], index map uint8 [n, d]).  H, when given, is the
    calibration Gram matrix already accumulated (X is then ignored)."""
    if H is None:
        H = gram(X)
    U, hd = inverse_factor(H, damp)
    lut, _ = lloyd(theta, hd, bits, gpr, max_iter)
    idx = sketch_round(theta, U, lut, bits)
    return pack(idx, bits), lut, idx


# ---------------------------------------------------------------------------
# 8-bit activation checkpoints
# ---------------------------------------------------------------------------

class Ckpt8(NamedTuple):
    """An 8-bit checkpoint of bf16 rows [T, d]: int8 q [T, d] and one scale byte
    per 32 columns, uint8 [T, d // 32] (the format is in sk.h)."""
    q: torch.Tensor
    scale: torch.Tensor


_HERE = contextlib.nullcontext()


def _on(device: torch.device):
    """The library works on the current device: make it the tensors' own."""
    if device.index is None or device.index == torch.cuda.current_device():
        return _HERE
    return torch.cuda.device(device)


def _rows(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """Contiguous and 16-byte aligned, as the library wants it: a view into the
    middle of a buffer may be neither."""
    if t is None:
        return None
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _together(first: torch.Tensor, *others: Optional[torch.Tensor]) -> None:
    at = first.device
    for t in others:
        if t is not None and t.device != at:
            raise ValueError("every tensor of a call must be on one device")


def _has_tangent(*tensors: Optional[torch.Tensor]) -> bool:
    """Whether one of the tensors carries a forward-mode derivative.  A dual tensor
    need not require a gradient, and grad mode has no say in it: a call that passed
    its autograd function by would drop the tangent, which reads as zero later on.
    (Outside any dual level, the rule, this takes 0.2 us.)"""
    return getattr(forward_ad, "_current_level", 0) >= 0 and any(
        t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def _refuse_tangent(*tensors: Optional[torch.Tensor]) -> None:
    if _has_tangent(*tensors):
        raise NotImplementedError("the backward passes of this library have no forward-mode derivative")


def _capturing(t: torch.Tensor) -> bool:
    return t.is_cuda and torch.cuda.is_current_stream_capturing()


# workspace sizes by device and shape: a step asks for the same few again and again.
# (The LUT gradient's is not kept: SK_BWD_PATH may change it.)
@functools.lru_cache(maxsize=256)
def _norm_bwd_bytes(device: torch.device, T: int, d: int) -> int:
    return int(lib.sk_layer_norm_bwd_workspace_bytes(T, d))


@functools.lru_cache(maxsize=256)
def _cross_entropy_bytes(device: torch.device, T: int, V: int, d: int, dh: bool, dw: bool) -> int:
    return int(lib.sk_cross_entropy_workspace_bytes(T, V, d, int(dh), int(dw)))


def _need_ckpt8(ck: "Ckpt8"):
    q, scale = ck
    _need(q, torch.int8, "q", 2)
    _need(scale, torch.uint8, "scale", 2)
    T, d = q.shape
    if d % 32 or tuple(scale.shape) != (T, d // 32):
        raise ValueError("scale must hold one byte per 32 columns of q")
    _together(q, scale)
    return q, scale, T, d


def _ckpt8_for(X: torch.Tensor, ck: Ckpt8):
    """(q, scale) of a checkpoint that a caller has of X, as the backward pass will
    want them: a wrong one is refused before the forward pass, a part of a longer
    batch's one is brought to the library's alignment."""
    q, scale = ck
    if not isinstance(q, torch.Tensor) or q.dtype != torch.int8 or not isinstance(scale, torch.Tensor) \
            or scale.dtype != torch.uint8:
        raise TypeError("a checkpoint is an int8 and a uint8 tensor")
    if q.dim() != 2 or q.shape != X.shape:
        raise ValueError("the checkpoint must have X's shape")
    if q.shape[1] % 32 or scale.shape != (q.shape[0], q.shape[1] // 32):
        raise ValueError("scale must hold one byte per 32 columns of q")
    _together(X, q, scale)
    return _rows(q), _rows(scale)


def ckpt8(X: torch.Tensor) -> Ckpt8:
    """The 8-bit checkpoint of bf16 rows X [T, d] (d a multiple of 32)."""
    _need(X, torch.bfloat16, "X", 2)
    T, d = X.shape
    if d % 32:
        raise ValueError("d must be a multiple of 32")
    with _on(X.device):
        q = torch.empty((T, d), dtype=torch.int8, device=X.device)
        scale = torch.empty((T, d // 32), dtype=torch.uint8, device=X.device)
        _check(lib.sk_ckpt8_quantize(_ptr(X), T, d, _ptr(q), _ptr(scale), _stream(X.device)))
    return Ckpt8(q, scale)


def ckpt8_dequant(ck: Ckpt8) -> torch.Tensor:
    """The bf16 rows [T, d] that a checkpoint stands for."""
    q, scale, T, d = _need_ckpt8(ck)
    with _on(q.device):
        X = torch.empty((T, d), dtype=torch.bfloat16, device=q.device)
        _check(lib.sk_ckpt8_dequantize(_ptr(q), _ptr(scale), T, d, _ptr(X), _stream(q.device)))
    return X


def linear_bwd_lut_ckpt8(packed: torch.Tensor, bits: int, gpr: int, ck: Ckpt8, dY: torch.Tensor,
                         task: Optional[torch.Tensor] = None, ntask: int = 1, out: Optional[torch.Tensor] = None,
                         accumulate: bool = False) -> torch.Tensor:
    """dlut [ntask, n, gpr, k] fp32 as linear_bwd_lut computes it, for the X that
    the checkpoint stands for."""
    q, scale, T, d = _need_ckpt8(ck)
    _need(dY, torch.bfloat16, "dY", 2)
    _need(packed, torch.uint8, "packed")
    n = dY.shape[1]
    if dY.shape[0] != T:
        raise ValueError("the checkpoint and dY must have the same number of tokens")
    if packed.numel() < packed_bytes(n, d, bits):
        raise ValueError("packed does not hold [n, d] indices")
    task = _task_arg(task, T)
    _together(q, dY, packed, task, out)
    shape = (ntask, n, gpr, 1 << bits)
    if out is not None:
        _need(out, torch.float32, "out")
        if out.numel() != ntask * n * gpr << bits:
            raise ValueError(f"out must hold {shape} values")
    elif accumulate:
        raise ValueError("accumulate adds to out: give it")
    with _on(q.device):
        if out is None:
            out = torch.empty(shape, dtype=torch.float32, device=q.device)
        ws, nb = _workspace(SK_OP_BWD_LUT_CKPT8, n, d, bits, gpr, T, ntask, q.device)
        _check(lib.sk_linear_bwd_lut_ckpt8(_ptr(packed), bits, gpr, n, d, _ptr(q), _ptr(scale), _ptr(dY), T, _ptr(task),
                                           ntask, _ptr(out), int(accumulate), _ptr(ws), nb, _stream(q.device)))
    return out


# ---------------------------------------------------------------------------
# Layer norm and RMS norm
# ---------------------------------------------------------------------------

_NORM_TYPES = {torch.float32: SK_F32, torch.bfloat16: SK_BF16, torch.float16: SK_F16}


def _norm_args(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor]):
    if not isinstance(x, torch.Tensor) or x.dtype not in _NORM_TYPES:
        raise TypeError("x must be a float32, bfloat16 or float16 tensor")
    _need(x, x.dtype, "x", 2)
    if not isinstance(weight, torch.Tensor) or weight.dtype not in (x.dtype, torch.float32):
        raise TypeError("weight must have x's type or float32")
    _need(weight, weight.dtype, "weight", 1)
    T, d = x.shape
    if weight.numel() != d:
        raise ValueError("weight must hold one value per column")
    if bias is not None:
        _need(bias, weight.dtype, "bias", 1)
        if bias.numel() != d:
            raise ValueError("bias must hold one value per column")
    _together(x, weight, bias)
    return T, d, _NORM_TYPES[x.dtype], _NORM_TYPES[weight.dtype]


def layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                   rms: bool = False, ckpt: bool = False, stats: bool = True):
    """(y, mean, rstd, checkpoint) of the layer norm (or RMS norm) of x [T, d]:
    mean and rstd are fp32 [T] for layer_norm_bwd (None without `stats`; mean is
    None for an RMS norm), the checkpoint is the Ckpt8 of y (None without `ckpt`)."""
    T, d, xt, wt = _norm_args(x, weight, bias)
    if ckpt and (x.dtype != torch.bfloat16 or d % 32):
        raise ValueError("a checkpoint needs bf16 rows whose length is a multiple of 32")
    dev = x.device
    with _on(dev):
        y = torch.empty_like(x)
        mean = torch.empty(T, dtype=torch.float32, device=dev) if stats and not rms else None
        rstd = torch.empty(T, dtype=torch.float32, device=dev) if stats else None
        ck = None
        if ckpt:
            ck = Ckpt8(torch.empty((T, d), dtype=torch.int8, device=dev),
                       torch.empty((T, d // 32), dtype=torch.uint8, device=dev))
        _check(lib.sk_layer_norm_fwd(_ptr(x), xt, T, d, _ptr(weight), _ptr(bias), wt, eps, int(rms), _ptr(y), _ptr(mean),
                                     _ptr(rstd), _ptr(ck.q) if ck else None, _ptr(ck.scale) if ck else None,
                                     _stream(dev)))
    return y, mean, rstd, ck


def layer_norm_bwd(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, mean: Optional[torch.Tensor],
                   rstd: torch.Tensor, rms: bool = False, bias: bool = True, need_dx: bool = True,
                   need_dw: bool = True):
    """(dx, dw, db) of layer_norm_fwd (None where not wanted): dx has x's type, dw
    and db the weight's."""
    T, d, xt, wt = _norm_args(x, weight, None)
    _need(dy, x.dtype, "dy", 2)
    if dy.shape != x.shape:
        raise ValueError("dy must have x's shape")
    if rms:
        mean = None
    else:
        _need(mean, torch.float32, "mean", 1)
    _need(rstd, torch.float32, "rstd", 1)
    if rstd.numel() != T or (mean is not None and mean.numel() != T):
        raise ValueError("mean and rstd must hold one value per row")
    _together(x, dy, rstd, mean)
    dev = x.device
    with _on(dev):
        dx = torch.empty_like(x) if need_dx else None
        dw = torch.empty_like(weight) if need_dw else None
        db = torch.empty_like(weight) if bias else None
        ws, nb = None, 0
        if need_dw or bias:
            nb = _norm_bwd_bytes(dev, T, d)
            ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=dev)
        _check(lib.sk_layer_norm_bwd(_ptr(dy), _ptr(x), xt, T, d, _ptr(weight), wt, _ptr(mean), _ptr(rstd), int(rms), _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws), nb, _stream(dev)))
    return dx, dw, db


class LayerNormFunction(torch.autograd.Function):
    """layer_norm_fwd / layer_norm_bwd as an autograd function of x, weight and bias."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, rms, ckpt):
        y, mean, rstd, ck = layer_norm_fwd(x, weight, bias, eps, rms, ckpt)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.rms = rms
        if ck is None:
            return y
        ctx.mark_non_differentiable(ck.q, ck.scale)
        return y, ck.q, ck.scale

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, *_):
        _refuse_tangent(dy)
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = layer_norm_bwd(_rows(dy.to(x.dtype)), x, weight, mean, rstd, ctx.rms, need[2], need[0],
                                    need[1])
        return dx, dw, db, None, None, None


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
               rms: bool = False, ckpt: bool = False):
    """Layer norm (RMS norm with `rms`) over the last dimension of x [..., d], an
    autograd function of x, weight and bias.  With `ckpt` it returns (y, Ckpt8 of
    y's rows) for a SketchedLinear that keeps its input in 8 bits."""
    lead = x.shape[:-1]
    rows = _rows(x if len(lead) == 1 else x.reshape(-1, x.shape[-1]))
    weight, bias = _rows(weight), _rows(bias)
    if not (_has_tangent(x, weight, bias)
            or torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, bias))):
        y, _, _, ck = layer_norm_fwd(rows, weight, bias, eps, rms, ckpt, stats=False)
    else:
        y = LayerNormFunction.apply(rows, weight, bias, eps, rms, ckpt)
        if ckpt:
            y, ck = y[0], Ckpt8(y[1], y[2])
    if len(lead) != 1:
        y = y.reshape(*lead, x.shape[-1])
    return (y, ck) if ckpt else y


class LayerNorm(torch.nn.Module):
    """Layer norm (RMS norm with `rms`, then without a bias unless asked for) of
    [..., d] activations; forward(x, ckpt) as layer_norm."""

    def __init__(self, d: int, eps: float = 1e-5, rms: bool = False, bias: Optional[bool] = None,
                 dtype: torch.dtype = torch.float32, device=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(d, dtype=dtype, device=device))
        self.bias = (torch.nn.Parameter(torch.zeros(d, dtype=dtype, device=device))
                     if (not rms if bias is None else bias) else None)
        self.eps = eps
        self.rms = rms

    def forward(self, x: torch.Tensor, ckpt: bool = False):
        return layer_norm(x, self.weight, self.bias, self.eps, self.rms, ckpt)


# ---------------------------------------------------------------------------
# Linear cross entropy: the head product and its loss
# ---------------------------------------------------------------------------

_REDUCTIONS = {"none": SK_CE_NONE, "mean": SK_CE_MEAN, "sum": SK_CE_SUM}


def cross_entropy(H: torch.Tensor, W: torch.Tensor, target: torch.Tensor, ignore_index: int = -100,
                  reduction: str = "mean", dloss: Optional[torch.Tensor] = None, need_loss: bool = True,
                  need_dh: bool = False, need_dw: bool = False):
    """(loss, dH, dW) of the softmax cross entropy of H W^T against target, None
    where not wanted.  H bf16 [T, d], W bf16 [V, d], target int32 or int64 [T];
    loss fp32, [T] for reduction "none", else a scalar; dloss: the loss's own
    gradient (fp32, its shape), ones when None."""
    _need(H, torch.bfloat16, "H", 2)
    _need(W, torch.bfloat16, "W", 2)
    if not isinstance(target, torch.Tensor) or target.dtype not in (torch.int32, torch.int64):
        raise TypeError("target must be an int32 or int64 tensor")
    _need(target, target.dtype, "target", 1)
    T, d = H.shape
    V = W.shape[0]
    if W.shape[1] != d:
        raise ValueError("H and W must have the same number of columns")
    if target.numel() != T:
        raise ValueError("target must hold one class per token")
    if reduction not in _REDUCTIONS:
        raise ValueError('reduction must be "none", "mean" or "sum"')
    red = _REDUCTIONS[reduction]
    if dloss is not None:
        _need(dloss, torch.float32, "dloss")
        if dloss.numel() != (T if red == SK_CE_NONE else 1):
            raise ValueError("dloss must have the loss's shape")
    _together(H, W, target, dloss)
    dev = H.device
    with _on(dev):
        loss = torch.empty((T,) if red == SK_CE_NONE else (), dtype=torch.float32, device=dev) if need_loss else None
        dH = torch.empty_like(H) if need_dh else None
        dW = torch.empty_like(W) if need_dw else None
        nb = _cross_entropy_bytes(dev, T, V, d, need_dh, need_dw)
        ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=dev)
        _check(lib.sk_cross_entropy(_ptr(H), _ptr(W), _ptr(target), target.element_size() * 8, T, V, d, ignore_index,
                                    red, _ptr(dloss), _ptr(loss), _ptr(dH), _ptr(dW), _ptr(ws), nb, _stream(dev)))
    return loss, dH, dW


class LinearCrossEntropyFunction(torch.autograd.Function):
    """cross_entropy as an autograd function of H and W.

    A reduced loss's gradient is known up to one factor, so the forward pass
    computes loss and gradients together (the logits' product is not repeated)
    and the backward pass scales them in place by the incoming gradient, which a
    factor of 1 leaves alone and a power of two scales exactly; any other factor (a
    loss divided by three) rounds them to bf16 a second time.  They are handed out once; a second backward pass
    over a retained graph computes them again, as does reduction "none", whose
    gradient needs every token's factor.  So does a backward pass that is captured
    into a CUDA graph without its forward pass: its replays would scale the same
    buffers again and again."""

    @staticmethod
    def forward(ctx, H, W, target, ignore_index, reduction):
        dh, dw = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        now = reduction != "none"
        loss, dH, dW = cross_entropy(H, W, target, ignore_index, reduction, need_dh=dh and now, need_dw=dw and now)
        ctx.save_for_backward(H, W, target)
        ctx.args = (ignore_index, reduction)
        ctx.ready = (dH, dW) if now else None
        ctx.captured = _capturing(H)
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        _refuse_tangent(g)
        H, W, target = ctx.saved_tensors
        dh, dw = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        g = g.to(torch.float32).contiguous()
        if ctx.ready is None or _capturing(H) != ctx.captured:
            _, dH, dW = cross_entropy(H, W, target, *ctx.args, dloss=g, need_loss=False, need_dh=dh, need_dw=dw)
            return dH, dW, None, None, None
        dH, dW = ctx.ready
        ctx.ready = None
        with _on(H.device):
            _check(lib.sk_scale_bf16(_ptr(dH), 0 if dH is None else dH.numel(), _ptr(dW),
                                     0 if dW is None else dW.numel(), _ptr(g), _stream(H.device)))
        return dH, dW, None, None, None


def linear_cross_entropy(H: torch.Tensor, W: torch.Tensor, target: torch.Tensor, ignore_index: int = -100,
                         reduction: str = "mean") -> torch.Tensor:
    """Softmax cross entropy of the logits H W^T (H bf16 [..., d], W bf16 [V, d])
    against target [...], an autograd function of H and W that never holds the
    logits.  Tokens whose target is ignore_index take no part; "mean" divides by
    the others' number (0 when there are none)."""
    lead = H.shape[:-1]
    if target.shape != lead:
        raise ValueError("target must hold one class per token")
    args = (_rows(H if len(lead) == 1 else H.reshape(-1, H.shape[-1])), _rows(W), target.reshape(-1).contiguous())
    if _has_tangent(H, W) or torch.is_grad_enabled() and (H.requires_grad or W.requires_grad):
        loss = LinearCrossEntropyFunction.apply(*args, ignore_index, reduction)
    else:
        loss = cross_entropy(*args, ignore_index, reduction)[0]
    return loss.reshape(lead) if reduction == "none" and len(lead) != 1 else loss


# ---------------------------------------------------------------------------
# The layer as an autograd function and a module
# ---------------------------------------------------------------------------

class SketchedLinearFunction(torch.autograd.Function):
    """Y = X Theta_hat^T with gradients for X and for the LUT values only.

    `lut` is the trainable tensor that receives the LUT gradient; `lut16` holds
    the fp16 tables the kernels read (the same tensor when `lut` is fp16, else
    the round-to-nearest-even fp16 of an fp32 master).  The LUT gradient is
    computed in fp32 and returned in `lut`'s dtype: an fp32 master gets it
    unrounded."""

    @staticmethod
    def forward(ctx, X, lut, lut16, packed, bits, task):
        Y = linear_fwd(packed, lut16, bits, X.contiguous(), task)
        ctx.save_for_backward(X, lut16, packed, task if task is not None else torch.empty(0))
        ctx.bits = bits
        ctx.has_task = task is not None
        ctx.lut_dtype = lut.dtype
        return Y

    @staticmethod
    def backward(ctx, dY):
        X, lut16, packed, task = ctx.saved_tensors
        task = task if ctx.has_task else None
        dY = dY.contiguous().to(torch.bfloat16)
        dX = dlut = None
        if ctx.needs_input_grad[0]:
            dX = linear_bwd_input(packed, lut16, ctx.bits, X.shape[1], dY, task)
        if ctx.needs_input_grad[1]:
            ntask, n, gpr, _ = lut16.shape
            dlut = linear_bwd_lut(packed, ctx.bits, gpr, X, dY, task, ntask)
            if dlut.dtype != ctx.lut_dtype:
                dlut = dlut.to(ctx.lut_dtype)
        return dX, dlut, None, None, None, None


class SketchedLinearCkpt8Function(torch.autograd.Function):
    """SketchedLinearFunction that keeps X as an 8-bit checkpoint (q, scale) for
    the LUT gradient.  The forward product uses X itself, and the gradient for X
    does not need X, so only the LUT gradient sees the rounding to 8 bits."""

    @staticmethod
    def forward(ctx, X, lut, lut16, packed, bits, task, q, scale):
        Y = linear_fwd(packed, lut16, bits, X, task)
        if ctx.needs_input_grad[1]:
            if q is None:
                q, scale = ckpt8(X)
        else:
            q = scale = None
        ctx.save_for_backward(lut16, packed, task, q, scale)
        ctx.bits = bits
        ctx.in_features = X.shape[1]
        ctx.lut_dtype = lut.dtype
        return Y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        _refuse_tangent(dY)
        lut16, packed, task, q, scale = ctx.saved_tensors
        dY = _rows(dY.to(torch.bfloat16))
        ntask, n, gpr, _ = lut16.shape
        dX = dlut = None
        if ctx.needs_input_grad[0]:
            dX = linear_bwd_input(packed, lut16, ctx.bits, ctx.in_features, dY, task)
        if ctx.needs_input_grad[1]:
            dlut = linear_bwd_lut_ckpt8(packed, ctx.bits, gpr, Ckpt8(q, scale), dY, task, ntask).to(ctx.lut_dtype)
        return dX, dlut, None, None, None, None, None, None


def sketched_linear(X: torch.Tensor, lut: torch.Tensor, packed: torch.Tensor, bits: int,
                    task: Optional[torch.Tensor] = None, lut16: Optional[torch.Tensor] = None,
                    ckpt=False) -> torch.Tensor:
    """Y = X Theta_hat^T as an autograd function of X and of the LUT values.

    lut: fp32 master LUTs (their gradient stays fp32) or fp16 LUTs (their
    gradient is rounded to fp16).  lut16: the fp16 tables of an fp32 master,
    when the caller keeps them (else they are rounded from `lut` here).
    ckpt: keep X in 8 bits for the LUT gradient, either a Ckpt8 of X that the
    caller has (layers that share an input share it) or True to make one here;
    without grad mode nothing is kept and none is made."""
    if lut16 is None:
        lut16 = lut if lut.dtype == torch.float16 else lut.detach().to(torch.float16)
    if ckpt is not False and ckpt is not None:
        q, scale = (None, None) if ckpt is True else _ckpt8_for(X, ckpt)
        X = _rows(X)
        if torch.is_grad_enabled():
            return SketchedLinearCkpt8Function.apply(X, lut, lut16, packed, bits, task, q, scale)
    return SketchedLinearFunction.apply(X, lut, lut16, packed, bits, task)


class SketchedLinear(torch.nn.Module):
    """A linear layer (no bias) whose weight is the sketch Theta_hat: a frozen
    packed index map (buffer), trainable fp32 master LUTs [ntask, n, gpr,
    2**bits] (parameter `lut`, whose gradient is the library's fp32 LUT
    gradient) and the fp16 tables the kernels read (buffer `lut16`, the
    round-to-nearest-even of the master).  forward(X, task) takes bf16
    activations [..., d]; task holds one LUT-set id per token (int32), or None
    for set 0.

    `lut16` follows the master: `adamw_step` / `sgd_step` update both in one
    library call; any other in-place change of `lut` (a torch optimizer) is
    noticed by its version counter and `lut16` is rounded again before the
    next forward.

    ckpt8=True keeps the layer's input in 8 bits instead of bf16 between the
    forward and the backward pass; forward(X, task, ckpt) then takes the Ckpt8 of
    X from a caller that has one (layer_norm(..., ckpt=True)) or makes its own."""

    ckpt8 = False          # of modules pickled without the attribute

    def __init__(self, packed: torch.Tensor, lut: torch.Tensor, bits: int, in_features: int, ckpt8: bool = False):
        super().__init__()
        self.ckpt8 = ckpt8
        self.register_buffer("packed", packed)
        self.lut = torch.nn.Parameter(lut.detach().to(torch.float32).contiguous())
        self.register_buffer("lut16", lut.detach().to(torch.float16).contiguous())
        self.bits = bits
        self.in_features = in_features
        self.out_features = lut.shape[1]
        self._synced = self._lut_state()

    def _lut_state(self):
        return (self.lut.data_ptr(), self.lut._version)

    def _sync_lut16(self):
        if self._lut_state() != self._synced:
            with torch.no_grad():
                self.lut16.copy_(self.lut)
            self._synced = self._lut_state()

    @classmethod
    def from_dense(cls, weight: torch.Tensor, X_calib: torch.Tensor, bits: int, gpr: int, ntask: int = 1,
                   damp: float = 0.01, max_iter: int = 100, ckpt8: bool = False) -> "SketchedLinear":
        """Sketch a dense weight [n, d] with calibration activations [s, d]
        (bf16); every LUT set starts from the same learned centroids."""
        packed, lut, _ = sketch_layer(weight.float().contiguous(), X_calib, bits, gpr, damp, max_iter)
        return cls(packed, lut.unsqueeze(0).repeat(ntask, 1, 1, 1).contiguous(), bits, weight.shape[1], ckpt8)

    def forward(self, X: torch.Tensor, task: Optional[torch.Tensor] = None, ckpt: Optional[Ckpt8] = None) -> torch.Tensor:
        self._sync_lut16()
        lead = X.shape[:-1]
        Y = sketched_linear(X.reshape(-1, self.in_features).to(torch.bfloat16).contiguous(), self.lut, self.packed,
                            self.bits, task, lut16=self.lut16, ckpt=ckpt if ckpt is not None else self.ckpt8)
        return Y.reshape(*lead, self.out_features)

    def adamw_step(self, m: torch.Tensor, v: torch.Tensor, step: int, lr: float, beta1: float = 0.9,
                   beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
                   counts: Optional[torch.Tensor] = None) -> None:
        """One AdamW step of the master LUTs from their gradient; rewrites lut16."""
        self._sync_lut16()
        lut_adamw_(self.lut.data, m, v, self.lut.grad, self.bits, step, lr, beta1, beta2, eps, weight_decay,
                   counts, self.lut16)

    def sgd_step(self, lr: float, counts: Optional[torch.Tensor] = None) -> None:
        """One SGD step of the master LUTs from their gradient; rewrites lut16."""
        self._sync_lut16()
        lut_sgd_(self.lut.data, self.lut.grad, self.bits, lr, counts, self.lut16)
