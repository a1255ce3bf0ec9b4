"""Python binding of libmips' training operators: embedding lookup and its gradient, and
gradient-norm clipping. Argument marshalling only, as in the package's other entry points: the
work is in the HIP kernels behind include/mips.h.
"""
from __future__ import annotations

import ctypes as C
import math
from typing import List, Optional, Sequence, Tuple

import torch

from . import BF16, F32, MipsError, _check, _ptr, _stream, empty_workspace, lib


def _code(t: torch.Tensor, what: str) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"{what} must be float32 or bfloat16, got {t.dtype}")


def _on_gpu(device: torch.device, **tensors) -> None:
    """Every tensor is on `device`, a GPU and the current one (launches go there)."""
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")
    if device.type != "cuda":
        raise ValueError(f"tensors must be on the GPU, got {device}")
    if device.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {device}, the current device is {torch.cuda.current_device()}")


def _ids_arg(ids: torch.Tensor) -> Tuple[torch.Tensor, int]:
    if ids.dtype == torch.int32:
        return ids.contiguous(), 32
    if ids.dtype == torch.int64:
        return ids.contiguous(), 64
    raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")


def _rows_arg(x: torch.Tensor) -> torch.Tensor:
    """x [r, d] with unit stride along d and a row stride of at least d (else a copy)."""
    if (x.stride(1) == 1 or x.shape[1] == 1) and (x.stride(0) >= x.shape[1] or x.shape[0] <= 1):
        return x
    return x.contiguous()


def _row_stride(x: torch.Tensor) -> int:
    return max(int(x.stride(0)), int(x.shape[1])) if x.shape[0] > 1 else int(x.shape[1])


# ------------------------------------------------------------------------ embedding
def embedding_lookup(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
    """scale * table[ids], rounded once to the table's type: [*ids.shape, d].

    table: float32 or bfloat16 [rows, d] on the GPU (any row stride); ids: int32 or int64 of any
    shape. An id outside [0, rows) is padding and gives a row of zeros.
    """
    if table.dim() != 2 or table.shape[0] < 1 or table.shape[1] < 1:
        raise ValueError(f"table must be [rows >= 1, d >= 1], got {tuple(table.shape)}")
    _on_gpu(table.device, ids=ids)
    code = _code(table, "table")
    flat, bits = _ids_arg(ids)
    table = _rows_arg(table)
    rows, d = table.shape
    out = torch.empty((*ids.shape, d), dtype=table.dtype, device=table.device)
    _check(lib().mips_embedding_lookup(_ptr(table), code, rows, d, _row_stride(table), _ptr(flat), bits,
                                       flat.numel(), float(scale), _ptr(out), _stream(table.device)),
           "mips_embedding_lookup")
    return out


def embedding_grad(grad: torch.Tensor, ids: torch.Tensor, rows: int, scale: float = 1.0,
                   out: Optional[torch.Tensor] = None, accumulate: bool = False,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of embedding_lookup for its table: [rows, d], row v being scale times the
    sum of grad over the tokens with id v (binary32, in token order: reproducible bit by bit).

    grad: float32 or bfloat16 [*ids.shape, d]; ids as embedding_lookup's (ids outside
    [0, rows) take no part). out: [rows, d] of grad's type or float32 (default: a new tensor
    of grad's type); with accumulate the sums are added to it (a tied table's other gradient).
    """
    if grad.dim() != ids.dim() + 1 or tuple(grad.shape[:-1]) != tuple(ids.shape):
        raise ValueError(f"grad must be [*ids.shape, d], got {tuple(grad.shape)} for ids {tuple(ids.shape)}")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    _on_gpu(grad.device, ids=ids, out=out, workspace=workspace)
    code = _code(grad, "grad")
    flat, bits = _ids_arg(ids)
    t, d = flat.numel(), grad.shape[-1]
    g = _rows_arg(grad.reshape(t, d))
    if out is None:
        out = torch.empty((rows, d), dtype=grad.dtype, device=grad.device)
    elif tuple(out.shape) != (rows, d) or (d > 1 and out.stride(1) != 1) or (rows > 1 and out.stride(0) < d):
        raise ValueError(f"out must be [{rows}, {d}] with contiguous rows, got {tuple(out.shape)}")
    elif out.dtype not in (grad.dtype, torch.float32):
        raise TypeError(f"out must be {grad.dtype} or float32, got {out.dtype}")
    if workspace is None:
        nbytes = lib().mips_embedding_grad_workspace_size(t, rows, d)
        if nbytes == 0:
            raise MipsError(2, "mips_embedding_grad_workspace_size")
        workspace = empty_workspace(nbytes, grad.device)
    _check(lib().mips_embedding_grad(_ptr(g), code, t, d, _row_stride(g), _ptr(flat), bits, rows,
                                     float(scale), int(accumulate), _ptr(out), _code(out, "out"),
                                     _row_stride(out), _ptr(workspace), workspace.numel(),
                                     _stream(grad.device)), "mips_embedding_grad")
    return out


# ------------------------------------------------------------------------- clipping
def _dense(t: torch.Tensor) -> bool:
    """Whether t's elements fill one run of memory, in any order of its axes."""
    want = 1
    for size, stride in sorted(((n, s) for n, s in zip(t.shape, t.stride()) if n != 1), key=lambda x: x[1]):
        if stride != want:
            return False
        want *= size
    return True


def clip_grad_norm(tensors: Sequence[torch.Tensor], max_norm: float,
                   out: Optional[Sequence[torch.Tensor]] = None,
                   workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, List[torch.Tensor]]:
    """The 2-norm over all elements of `tensors` (float32 scalar on the GPU), and the tensors
    scaled by min(1, max_norm / (norm + 1e-6)): in place, or into `out` (tensors of the same
    shapes, types and strides). Nothing waits for the GPU.

    tensors: float32 or bfloat16, mixed as they come, each dense (its elements fill one run of
    memory). max_norm: >= 0; math.inf only takes the norm.
    """
    tensors = list(tensors)
    outs = tensors if out is None else list(out)
    if not tensors:
        raise ValueError("clip_grad_norm needs at least one tensor")
    if len(outs) != len(tensors):
        raise ValueError(f"{len(outs)} out tensors for {len(tensors)}")
    if math.isnan(max_norm) or max_norm < 0:
        raise ValueError(f"max_norm must be at least 0, got {max_norm}")
    device = tensors[0].device
    _on_gpu(device, workspace=workspace)
    n = len(tensors)
    src, dst = (C.c_void_p * n)(), (C.c_void_p * n)()
    counts, codes = (C.c_int64 * n)(), (C.c_int32 * n)()
    for i, (t, o) in enumerate(zip(tensors, outs)):
        if t.device != device or o.device != device:
            raise ValueError(f"tensor {i} is on {t.device} (out {o.device}), expected {device}")
        if o is not t and (o.dtype != t.dtype or o.shape != t.shape or o.stride() != t.stride()):
            raise ValueError(f"out {i} must have its tensor's shape, type and strides")
        if not t.is_contiguous() and not _dense(t):
            raise ValueError(f"tensor {i} is not dense: shape {tuple(t.shape)}, strides {t.stride()}")
        src[i], dst[i], counts[i], codes[i] = t.data_ptr(), o.data_ptr(), t.numel(), _code(t, f"tensor {i}")
    norm = torch.empty((), dtype=torch.float32, device=device)
    if workspace is None:
        workspace = empty_workspace(lib().mips_clip_workspace_size(n), device)
    _check(lib().mips_clip_grad_norm(src, dst, counts, codes, n, float(max_norm), _ptr(norm),
                                     _ptr(workspace), workspace.numel(), _stream(device)),
           "mips_clip_grad_norm")
    return norm, outs
