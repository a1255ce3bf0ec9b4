"""Python binding of libmips' operators over histories of events, the layers of a user tower
between the embedding lookup and the softmax over items: a gated linear recurrence with its
gradient and its form for single events, dropout, and pooled and normalised vectors. Argument
marshalling only, as in the package's other entry points: the work is in the HIP kernels behind
include/mips.h.

Sequences are dense ([b, t, d]), padded (dense, with `lengths` [b]) or packed ([n, d] with
`offsets` [b + 1]); lengths and offsets are int32 or int64 on the GPU, and are not looked at on
the host.
"""
from __future__ import annotations

import ctypes as C
import dataclasses
from typing import Optional, Sequence, Tuple

import torch

from . import MipsError, _check, empty_workspace, lib
from .training import _code, _ids_arg, _on_gpu, _ptr, _row_stride, _rows_arg, _stream

EVENTS_MAX = 65536  # events of one gated_step call
PACKED_STRIDE_MAX = 524288  # elements between packed rows that are used in place


class _Sequences(C.Structure):
    _fields_ = [("b", C.c_int32), ("index_bits", C.c_int32), ("t", C.c_int64), ("n", C.c_int64),
                ("offsets", C.c_void_p), ("lengths", C.c_void_p)]


class _Rows(C.Structure):
    _fields_ = [("data", C.c_void_p), ("row_stride", C.c_int64), ("seq_stride", C.c_int64)]


def _index(x: torch.Tensor, what: str) -> Tuple[torch.Tensor, int]:
    if x.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"{what} must be int32 or int64, got {x.dtype}")
    return x.contiguous(), 32 if x.dtype == torch.int32 else 64


def _int32(what: str, *sizes: int) -> None:
    """Sizes that the C interface takes as 32 bits fit (ctypes would cut them short)."""
    if max(sizes) >= 1 << 31:
        raise MipsError(2, what)


def _sequences(shape: Sequence[int], offsets: Optional[torch.Tensor], lengths: Optional[torch.Tensor]):
    """(structure, b, d, tensors that it points into) of rows laid out as `shape`."""
    if offsets is not None:
        if lengths is not None:
            raise ValueError("offsets (packed rows) and lengths (padded ones) exclude each other")
        if len(shape) != 2 or shape[1] < 1:
            raise ValueError(f"packed rows must be [n, d >= 1], got {tuple(shape)}")
        if offsets.dim() != 1 or offsets.shape[0] < 2:
            raise ValueError(f"offsets must be [b + 1], b >= 1, got {tuple(offsets.shape)}")
        b = offsets.shape[0] - 1
        _int32("sequences", b, shape[1])
        offsets, bits = _index(offsets, "offsets")
        return _Sequences(b, bits, 0, shape[0], offsets.data_ptr(), None), b, shape[1], offsets
    if len(shape) != 3 or shape[0] < 1 or shape[1] < 1 or shape[2] < 1:
        raise ValueError(f"rows must be [b >= 1, t >= 1, d >= 1], or [n, d] with offsets, got {tuple(shape)}")
    b, t, d = shape
    _int32("sequences", b, d)
    bits = 0
    if lengths is not None:
        if tuple(lengths.shape) != (b,):
            raise ValueError(f"lengths must be [{b}], got {tuple(lengths.shape)}")
        lengths, bits = _index(lengths, "lengths")
    return _Sequences(b, bits, t, 0, None, _ptr(lengths)), b, d, lengths


def _rows(x: torch.Tensor) -> Tuple[torch.Tensor, _Rows]:
    """x, or a copy where its rows are not runs of memory that do not overlap, and its description.
    (Strides are asked for once: a tenth of the smallest calls is the time that such questions take.)"""
    shape, stride = x.shape, x.stride()
    if len(shape) == 2:
        x, row = _packed(x, shape, stride)
        if row > PACKED_STRIDE_MAX:
            x, row = x.contiguous(), shape[1]
        return x, _Rows(x.data_ptr(), row, 0)
    b, t, d = shape
    row, seq = stride[1] if t > 1 else d, stride[0] if b > 1 else t * d
    if (stride[2] != 1 and d > 1) or row < d or seq < d:
        x = x.contiguous()
        row, seq = d, t * d
    return x, _Rows(x.data_ptr(), row, seq)


def _packed(x: torch.Tensor, shape, stride) -> Tuple[torch.Tensor, int]:
    """x [n, d], or a copy where its rows are not runs of memory that do not overlap, and its row stride."""
    n, d = shape
    if (stride[1] != 1 and d > 1) or (stride[0] < d and n > 1):
        return x.contiguous(), d
    return x, stride[0] if n > 1 else d


def _like(x: torch.Tensor, **tensors) -> None:
    """The given tensors have x's shape and type."""
    shape, dtype = x.shape, x.dtype
    for name, t in tensors.items():
        if t is not None and (t.shape != shape or t.dtype != dtype):
            raise ValueError(f"{name} must be {x.dtype} {tuple(x.shape)}, got {t.dtype} {tuple(t.shape)}")


def _floats(shape: Tuple[int, int], **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shape):
            raise ValueError(f"{name} must be float32 {list(shape)}, got {t.dtype} {tuple(t.shape)}")


def _workspace(what: str, seq, *sizes, workspace: Optional[torch.Tensor], device) -> Optional[torch.Tensor]:
    """The given workspace, or one of the size that the call needs, None if it needs none."""
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous")
        return workspace
    nbytes = getattr(lib(), what)(C.byref(seq), *sizes)
    return empty_workspace(nbytes, device) if nbytes else None


def _empty(x: torch.Tensor) -> torch.Tensor:
    """A contiguous tensor of x's shape and type (a third less host time than x.new_empty(x.shape), where
    the smallest calls are bound by it)."""
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def _bytes(workspace: Optional[torch.Tensor]) -> int:
    return 0 if workspace is None else workspace.numel()


_F32 = torch.float32


# --------------------------------------------------------------------- recurrence
@dataclasses.dataclass
class GatedScan:
    """What gated_scan returns."""
    states: Optional[torch.Tensor]  # every state, of x's shape and type
    last: torch.Tensor              # float32 [b, d]: the state behind each sequence's last row
    carries: Optional[torch.Tensor]  # float32 [runs, d]: states between runs of rows, for the gradient


def _runs(seq, d: int, code: int) -> int:
    runs = lib().mips_gated_scan_carries(C.byref(seq), d, code)
    if runs < 0:
        raise MipsError(2, "mips_gated_scan_carries")
    return runs


def gated_scan(x: torch.Tensor, forget: torch.Tensor, gate: Optional[torch.Tensor] = None, *,
               offsets: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
               initial: Optional[torch.Tensor] = None, states: bool = True, carries: bool = True,
               workspace: Optional[torch.Tensor] = None) -> GatedScan:
    """A gated linear recurrence along each sequence: h_r = a_r h_{r-1} + b_r x_r per channel, with
    a = sigmoid(forget) and b = sigmoid(gate), or 1 - a without a gate; in binary32.

    x, forget, gate: float32 or bfloat16 [b, t, d] (with `lengths` [b]: padded) or, with
    `offsets` [b + 1], [n, d]; any strides (rows without unit stride along d, or that overlap, are
    copied first). initial: float32 [b, d], the state before each sequence (0 by default). With
    states false only the last states are written; with carries false the result has no gradient (they
    are a quarter of x's bytes where sequences fill their tiles of up to 128 rows or, of few channels, more,
    half where they leave almost half of them empty, and those of one tile at least). Padding is not read and has states of 0; a sequence without rows has
    its initial state as its last one.
    """
    seq, b, d, held = _sequences(x.shape, offsets, lengths)
    code = _code(x, "x")
    _like(x, forget=forget, gate=gate)
    _floats((b, d), initial=initial)
    dev = x.device
    _on_gpu(dev, forget=forget, gate=gate, offsets=offsets, lengths=lengths, initial=initial, workspace=workspace)
    x, xr = _rows(x)
    forget, fr = _rows(forget)
    gate, gr = _rows(gate) if gate is not None else (None, None)
    initial = None if initial is None else initial.contiguous()
    runs = _runs(seq, d, code)
    workspace = _workspace("mips_gated_scan_workspace_size", seq, d, code, workspace=workspace, device=dev)
    out = GatedScan(_empty(x) if states else None, x.new_empty((b, d), dtype=_F32),
                    x.new_empty((runs, d), dtype=_F32) if carries else None)
    _check(lib().mips_gated_scan(C.byref(seq), d, code, C.byref(xr), C.byref(fr), None if gr is None else C.byref(gr),
                                 _ptr(initial), _ptr(out.states), _ptr(out.last), _ptr(out.carries), _ptr(workspace),
                                 _bytes(workspace), _stream(dev)), "mips_gated_scan")
    return out


def gated_scan_backward(grad_states: Optional[torch.Tensor], grad_last: Optional[torch.Tensor], x: torch.Tensor,
                        forget: torch.Tensor, gate: Optional[torch.Tensor], forward: GatedScan, *,
                        offsets: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                        initial: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                        ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """The gradient of gated_scan: (grad_x, grad_forget, grad_gate, grad_initial float32 [b, d]), the
    last two None without a gate and an initial state.

    grad_states: x's shape and type, or None; grad_last: float32 [b, d], or None; one of them at
    least. `forward` is the result of gated_scan on the same arguments (its carries are used).
    """
    seq, b, d, held = _sequences(x.shape, offsets, lengths)
    code = _code(x, "x")
    if grad_states is None and grad_last is None:
        raise ValueError("the gradient of the states or of the last ones is needed")
    _like(x, forget=forget, gate=gate, grad_states=grad_states)
    _floats((b, d), initial=initial, grad_last=grad_last)
    dev = x.device
    if forward.carries is None:
        raise ValueError("the gradient needs the forward pass' carries")
    _floats((_runs(seq, d, code), d), carries=forward.carries)
    _on_gpu(dev, forget=forget, gate=gate, grad_states=grad_states, grad_last=grad_last, offsets=offsets,
            lengths=lengths, initial=initial, carries=forward.carries, workspace=workspace)
    x, xr = _rows(x)
    forget, fr = _rows(forget)
    gate, gr = _rows(gate) if gate is not None else (None, None)
    grad_states, sr = _rows(grad_states) if grad_states is not None else (None, None)
    initial, grad_last, carries = (None if t is None else t.contiguous() for t in (initial, grad_last, forward.carries))
    dx, df = _empty(x), _empty(x)
    dg = _empty(x) if gate is not None else None
    di = x.new_empty((b, d), dtype=_F32) if initial is not None else None
    workspace = _workspace("mips_gated_scan_workspace_size", seq, d, code, workspace=workspace, device=dev)
    _check(lib().mips_gated_scan_backward(
        C.byref(seq), d, code, C.byref(xr), C.byref(fr), None if gr is None else C.byref(gr), _ptr(initial),
        None if sr is None else C.byref(sr), _ptr(grad_last), _ptr(carries), _ptr(dx), _ptr(df),
        _ptr(dg), _ptr(di), _ptr(workspace), _bytes(workspace), _stream(dev)),
        "mips_gated_scan_backward")
    return dx, df, dg, di


def _table(name: str, t: torch.Tensor, d: int):
    """(shape, row stride) of a table of states."""
    shape, stride = t.shape, t.stride()
    if t.dtype != _F32 or len(shape) != 2 or shape[0] < 1 or shape[1] != d:
        raise ValueError(f"{name} must be float32 [rows >= 1, {d}], got {t.dtype} {tuple(shape)}")
    if (d > 1 and stride[1] != 1) or (shape[0] > 1 and stride[0] < d):
        raise ValueError(f"{name} must have contiguous rows that do not overlap, got strides {stride}")
    return shape, stride[0] if shape[0] > 1 else d


def gated_step(x: torch.Tensor, forget: torch.Tensor, state: torch.Tensor, rows: torch.Tensor,
               gate: Optional[torch.Tensor] = None, *, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """gated_scan for single events as they come: state[r] = a state[r] + b x for the events in order,
    r = rows[e]; the state after each event, [b, d] of x's type. Events of one row are applied one
    after another.

    x, forget, gate: float32 or bfloat16 [b, d], b up to EVENTS_MAX. state: float32 [rows, d] with any row
    stride, updated in place; with `out` (the same shape, not overlapping) the changed rows are
    written there instead. rows: int32 or int64 [b]; one outside the table is padding (a state of 0).
    """
    shape = x.shape
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError(f"x must be [b, d >= 1], got {tuple(shape)}")
    b, d = shape
    _int32("mips_gated_step", b, d)
    code = _code(x, "x")
    _like(x, forget=forget, gate=gate)
    if rows.shape != shape[:1]:
        raise ValueError(f"rows must be [{b}], got {tuple(rows.shape)}")
    table, from_stride = _table("state", state, d)
    into, to_stride = state, from_stride
    if out is not None:
        into, to_stride = out, _table("out", out, d)[1]
        if out.shape != table:
            raise ValueError(f"out must be {list(table)}, got {tuple(out.shape)}")
    dev = x.device
    _on_gpu(dev, forget=forget, gate=gate, state=state, rows=rows, out=out)
    ids, bits = _ids_arg(rows)
    x, xs = _packed(x, shape, x.stride())
    forget, fs = _packed(forget, shape, forget.stride())
    gp, gs = None, 0
    if gate is not None:
        gate, gs = _packed(gate, shape, gate.stride())
        gp = gate.data_ptr()
    h = _empty(x)
    _check(lib().mips_gated_step(x.data_ptr(), xs, forget.data_ptr(), fs, gp, gs, code, b, d, state.data_ptr(), from_stride,
                                 into.data_ptr(), to_stride, table[0], ids.data_ptr(), bits, h.data_ptr(), _stream(dev)),
           "mips_gated_step")
    torch.autograd.graph.increment_version(into)
    return h


# ------------------------------------------------------------------------ dropout
def dropout(x: torch.Tensor, p: float, seed: int, offset: int = 0, *, residual: Optional[torch.Tensor] = None,
            counter: Optional[torch.Tensor] = None) -> torch.Tensor:
    """residual + x with each element dropped with probability p and the others scaled by 1 / (1 - p) (as a float32):
    product and sum with one rounding in float32, then x's type. The mask follows from seed, offset (two calls with one seed need different
    ones) and the element's place in x alone; the same call on the gradient is the gradient for x.

    x: float32 or bfloat16 of any shape (copied first unless contiguous); p: taken in steps of
    2^-16; seed, offset: 64 bits. counter: int64 [1] on the GPU, added to the offset when the kernel
    runs: a captured graph that also advances it draws new numbers in every replay.
    """
    code = _code(x, "x")
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be between 0 and 1, got {p}")
    _like(x, residual=residual)
    if counter is not None and (counter.dtype != torch.int64 or counter.numel() != 1):
        raise ValueError(f"counter must be one int64, got {counter.dtype} {tuple(counter.shape)}")
    _on_gpu(x.device, residual=residual, counter=counter)
    x = x.contiguous()
    residual = None if residual is None else residual.contiguous()
    out = _empty(x)
    _check(lib().mips_dropout(_ptr(x), code, x.numel(), float(p), seed % (1 << 64), offset % (1 << 64), _ptr(counter),
                              _ptr(residual), _ptr(out), _stream(x.device)), "mips_dropout")
    return out


# ------------------------------------------------------------------------ pooling
@dataclasses.dataclass
class Pooled:
    """What pool_normalize returns."""
    vectors: torch.Tensor  # [b, d] of x's type
    mean: torch.Tensor     # float32 [b, d]
    norm: torch.Tensor     # float32 [b]: what the mean was divided by
    normalize: bool


def pool_normalize(x: torch.Tensor, *, offsets: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                   normalize: bool = True, workspace: Optional[torch.Tensor] = None) -> Pooled:
    """The mean of each sequence's rows, divided by sqrt(max(sum of its squares, 1e-12)) as
    l2_normalize's rows are (not with normalize false). A sequence without rows has a vector of zeros.

    x: float32 or bfloat16, laid out as gated_scan's; padding is not read.
    """
    seq, b, d, held = _sequences(x.shape, offsets, lengths)
    code = _code(x, "x")
    dev = x.device
    _on_gpu(dev, offsets=offsets, lengths=lengths, workspace=workspace)
    x, xr = _rows(x)
    out = Pooled(x.new_empty((b, d)), x.new_empty((b, d), dtype=_F32), x.new_empty((b,), dtype=_F32), bool(normalize))
    workspace = _workspace("mips_pool_workspace_size", seq, d, workspace=workspace, device=dev)
    _check(lib().mips_pool_normalize(C.byref(seq), d, code, C.byref(xr), int(out.normalize), _ptr(out.vectors),
                                     _ptr(out.mean), _ptr(out.norm), _ptr(workspace), _bytes(workspace), _stream(dev)),
           "mips_pool_normalize")
    return out


def pool_normalize_backward(grad: torch.Tensor, shape: Sequence[int], forward: Pooled, *,
                            offsets: Optional[torch.Tensor] = None,
                            lengths: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of pool_normalize for rows laid out as `shape` (x.shape), given that of the
    vectors (their shape and type) and the forward call's result."""
    seq, b, d, held = _sequences(shape, offsets, lengths)
    code = _code(grad, "grad")
    _like(forward.vectors, grad=grad)
    if tuple(grad.shape) != (b, d):
        raise ValueError(f"grad must be [{b}, {d}], got {tuple(grad.shape)}")
    _floats((b, d), mean=forward.mean)
    if forward.norm.dtype != torch.float32 or tuple(forward.norm.shape) != (b,):
        raise ValueError(f"norm must be float32 [{b}], got {forward.norm.dtype} {tuple(forward.norm.shape)}")
    dev = grad.device
    _on_gpu(dev, offsets=offsets, lengths=lengths, mean=forward.mean, norm=forward.norm)
    grad = _rows_arg(grad)
    mean, norm = forward.mean.contiguous(), forward.norm.contiguous()
    dx = grad.new_empty(tuple(shape))
    _check(lib().mips_pool_normalize_backward(C.byref(seq), d, code, _ptr(grad), _row_stride(grad), int(forward.normalize),
                                              _ptr(mean), _ptr(norm), _ptr(dx), _stream(dev)),
           "mips_pool_normalize_backward")
    return dx
