"""Python binding of libmips' training and evaluation operators: log probabilities over an item
table and their gradient, embedding lookup and its gradient, and gradient-norm clipping.
Argument marshalling only, as in the package's other entry points: the work is in the HIP
kernels behind include/mips.h.
"""
from __future__ import annotations

import ctypes as C
import dataclasses
import math
from typing import List, Optional, Sequence, Tuple, Union

import torch

from . import BF16, F32, Corpus, MipsError, _check, check_version, empty_workspace, lib


_CODES = {torch.float32: F32, torch.bfloat16: BF16}


def _code(t: torch.Tensor, what: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be float32 or bfloat16, got {t.dtype}")
    return code


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device) -> int:
    """The current stream's handle, where torch has a way to it without the stream object that
    torch.cuda.current_stream builds (1.8 of the 11 us of a small lookup)."""
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


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


# ---------------------------------------------------------------- log probabilities
ALTERNATIVES_MAX = 64
TARGETS_MAX = 64  # given ids a query, of item_logprobs_backward
ROWS, PACKED = 0, 1


@dataclasses.dataclass
class ItemLogprobs:
    """What item_logprobs returns; tensors that were not asked for are None."""
    logprobs: Optional[torch.Tensor]      # float32 [b, g]
    logsumexp: torch.Tensor               # float32 [b]
    entropy: Optional[torch.Tensor]       # float32 [b]
    alt_ids: Optional[torch.Tensor]       # int32 [b, k]
    alt_logprobs: Optional[torch.Tensor]  # float32 [b, k]


def _operand(x: torch.Tensor, d: int) -> torch.Tensor:
    """x as [rows, d] with 16-byte aligned rows; d is x's width rounded up to 16 bytes. Rows that
    are so already are used in place, others are copied once (padded with zeros)."""
    e = x.element_size()
    if x.shape[1] == d and x.data_ptr() % 16 == 0 and (x.stride(1) == 1 or d == 1):
        if x.shape[0] == 1 or (x.stride(0) >= d and x.stride(0) * e % 16 == 0 and x.stride(0) * e <= 1 << 25):
            return x
    y = torch.zeros((x.shape[0], d), dtype=x.dtype, device=x.device)
    y[:, :x.shape[1]] = x
    return y


def _exclude_words(exclude: Optional[torch.Tensor], n: int, b: int) -> Tuple[Optional[torch.Tensor], int]:
    """(contiguous bitmap or None, words per query), as topk's exclude."""
    if exclude is None:
        return None, 0
    words = (n + 31) // 32
    if exclude.dtype not in (torch.int32, torch.uint32):
        raise TypeError("exclude must be int32 or uint32")
    if exclude.dim() == 1 and exclude.numel() >= words:
        return exclude.contiguous(), 0
    if exclude.dim() == 2 and exclude.shape[0] == b and exclude.shape[1] >= words:
        return exclude.contiguous(), int(exclude.shape[1])
    raise ValueError(f"exclude must be [>= {words}] or [{b}, >= {words}], got {tuple(exclude.shape)}")


def _softmax_args(queries, items, ids, bias, exclude, workspace, model_version=None):
    """Checked and laid out operands of the softmax entry points: (queries, items pointer,
    layout, item stride, n, d, dtype code, ids, id bits, bias, exclude, exclude words)."""
    if queries.dim() != 2 or queries.shape[0] < 1:
        raise ValueError(f"queries must be [b >= 1, d], got {tuple(queries.shape)}")
    b, width = queries.shape
    if isinstance(items, Corpus):
        check_version(items, model_version)
        if items.dtype not in ("f32", "bf16"):
            raise TypeError(f"log probabilities need an f32 or bf16 index, got {items.dtype}")
        n, code, layout, stride, held = items.n, items.code, PACKED, 0, items.packed
        if items.d != width:
            raise ValueError(f"queries have width {width}, the index {items.d}")
        _code(queries, "queries")
        queries = queries.to(torch.float32 if code == F32 else torch.bfloat16)  # as topk rounds them
        d = width
    else:
        if items.dim() != 2 or items.shape[0] < 1 or items.shape[1] != width:
            raise ValueError(f"items must be [n >= 1, {width}], got {tuple(items.shape)}")
        if items.dtype != queries.dtype:
            raise TypeError(f"queries are {queries.dtype}, items {items.dtype}")
        n, code, layout = items.shape[0], _code(items, "items"), ROWS
        per = 16 // items.element_size()
        d = (width + per - 1) // per * per
        held = _operand(items, d)
        stride = _row_stride(held)
    _on_gpu(queries.device, items=held, ids=ids, bias=bias, exclude=exclude, workspace=workspace)
    queries = _operand(queries, d)
    bits = 32
    if ids is not None:
        if ids.dim() != 2 or ids.shape[0] != b:
            raise ValueError(f"ids must be [{b}, g], got {tuple(ids.shape)}")
        ids, bits = _ids_arg(ids)
    if bias is not None:
        if bias.dtype != torch.float32 or tuple(bias.shape) != (n,):
            raise ValueError(f"bias must be float32 [{n}], got {bias.dtype} {tuple(bias.shape)}")
        bias = bias.contiguous()
    exclude, words = _exclude_words(exclude, n, b)
    return queries, held, layout, stride, n, d, code, ids, bits, bias, exclude, words


def item_logprobs(queries: torch.Tensor, items: Union[torch.Tensor, Corpus], ids: Optional[torch.Tensor] = None, *,
                  scale: float = 1.0, bias: Optional[torch.Tensor] = None,
                  exclude: Optional[torch.Tensor] = None, entropy: bool = True, alternatives: int = 0,
                  workspace: Optional[torch.Tensor] = None, model_version: Optional[str] = None) -> ItemLogprobs:
    """Log probabilities under the softmax of scale * queries @ items.T + bias over all items,
    without the score matrix: of the given ids, with the log-sum-exp, the entropy and the
    `alternatives` most likely items (ties by the lowest id).

    queries: float32 or bfloat16 [b, d]; items: [n, d] of the same type (any strides; rows that
    are not 16-byte aligned are copied first, in every call: a table of 250,000 x 100 bfloat16 takes
    390 us where 104 wide it takes 298), d up to 128 (float32) or 256 (bfloat16), or an
    f32 or bf16 Corpus. ids: int32/int64 [b, g]; an id outside [0, n) is padding (0).
    scale: 1 / temperature, positive. bias: float32 [n], e.g. -log q of a sampled softmax; -inf and
    the lowest float mask an item (p = 0). exclude: bitmap as topk's; excluded items have
    probability 0. A logit of NaN or +inf makes its query's results NaN; one of -inf is no alternative.
    """
    q, held, layout, stride, n, d, code, ids, bits, bias, exclude, words = _softmax_args(
        queries, items, ids, bias, exclude, workspace, model_version)
    b, dev = q.shape[0], q.device
    g = 0 if ids is None else ids.shape[1]
    f32 = dict(dtype=torch.float32, device=dev)
    out = ItemLogprobs(
        logprobs=None if ids is None else torch.empty((b, g), **f32), logsumexp=torch.empty((b,), **f32),
        entropy=torch.empty((b,), **f32) if entropy else None,
        alt_ids=torch.empty((b, alternatives), dtype=torch.int32, device=dev) if alternatives > 0 else None,
        alt_logprobs=torch.empty((b, alternatives), **f32) if alternatives > 0 else None)
    if workspace is None:
        nbytes = lib().mips_logprobs_workspace_size(b, n, d, code, alternatives)
        if nbytes == 0:
            raise MipsError(2, "mips_logprobs_workspace_size")
        workspace = empty_workspace(nbytes, dev)
    _check(lib().mips_logprobs(_ptr(q), _row_stride(q), b, _ptr(held), layout, stride, n, d, code, _ptr(bias),
                               _ptr(exclude), words, float(scale), _ptr(ids), bits, g, alternatives,
                               _ptr(out.logprobs), _ptr(out.logsumexp), _ptr(out.entropy), _ptr(out.alt_ids),
                               _ptr(out.alt_logprobs), _ptr(workspace), workspace.numel(), _stream(dev)),
           "mips_logprobs")
    return out


def item_logprobs_backward(grad_logprobs: Optional[torch.Tensor], queries: torch.Tensor, items: torch.Tensor,
                           ids: Optional[torch.Tensor], forward: ItemLogprobs, *, scale: float = 1.0,
                           bias: Optional[torch.Tensor] = None, exclude: Optional[torch.Tensor] = None,
                           grad_entropy: Optional[torch.Tensor] = None, need_queries: bool = True,
                           need_items: bool = True, need_bias: bool = False,
                           workspace: Optional[torch.Tensor] = None
                           ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """The gradient of item_logprobs over a row table: (grad_queries [b, d], grad_items [n, d],
    grad_bias float32 [n]), the first two of the operands' type; None where not needed.

    grad_logprobs: float32 [b, g], the gradient of each log probability (a loss that is the
    mean of -log p of one target has -1/b); grad_entropy: float32 [b] or None. `forward` is the
    result of item_logprobs on the same arguments (its logsumexp, and its entropy with
    grad_entropy). Up to TARGETS_MAX ids a query. Rows that a shared bitmap excludes may hold
    anything; with one bitmap per query all rows must be finite.
    """
    q, held, _, stride, n, d, code, ids, bits, bias, exclude, words = _softmax_args(
        queries, items, ids, bias, exclude, workspace)
    if isinstance(items, Corpus):
        raise TypeError("the gradient needs a table of rows, not a packed index")
    b, dev, width = q.shape[0], q.device, queries.shape[1]
    g = 0 if ids is None else ids.shape[1]
    lse, ent = forward.logsumexp, forward.entropy if grad_entropy is not None else None
    if grad_entropy is not None and ent is None:
        raise ValueError("grad_entropy needs the forward pass' entropy")
    if (ids is None) != (grad_logprobs is None):
        raise ValueError("grad_logprobs and ids go together")
    for name, t, shape in (("grad_logprobs", grad_logprobs, (b, g)), ("grad_entropy", grad_entropy, (b,)),
                           ("logsumexp", lse, (b,)), ("entropy", ent, (b,))):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shape):
            raise ValueError(f"{name} must be float32 {list(shape)}, got {t.dtype} {tuple(t.shape)}")
    _on_gpu(dev, grad_logprobs=grad_logprobs, grad_entropy=grad_entropy, logsumexp=lse, entropy=ent)
    grad_logprobs, grad_entropy, lse, ent = (None if t is None else t.contiguous()
                                             for t in (grad_logprobs, grad_entropy, lse, ent))
    dq = torch.empty((b, d), dtype=q.dtype, device=dev) if need_queries else None
    di = torch.empty((n, d), dtype=q.dtype, device=dev) if need_items else None
    db = torch.empty((n,), dtype=torch.float32, device=dev) if need_bias else None
    if workspace is None:
        nbytes = lib().mips_logprobs_backward_workspace_size(b, n, d, code, g)
        if nbytes == 0:
            raise MipsError(2, "mips_logprobs_backward_workspace_size")
        workspace = empty_workspace(nbytes, dev)
    _check(lib().mips_logprobs_backward(_ptr(q), _row_stride(q), b, _ptr(held), stride, n, d, code, _ptr(bias),
                                        _ptr(exclude), words, float(scale), _ptr(ids), bits, g, _ptr(lse),
                                        _ptr(ent), _ptr(grad_logprobs), _ptr(grad_entropy), _ptr(dq), _ptr(di),
                                        _ptr(db), _ptr(workspace), workspace.numel(), _stream(dev)),
           "mips_logprobs_backward")
    if d != width:  # rows were padded to 16 bytes
        dq = None if dq is None else dq[:, :width].contiguous()
        di = None if di is None else di[:, :width].contiguous()
    return dq, di, db


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
    sum of grad over the tokens with id v (binary32, in an order that follows from the ids, sizes
    and device: the same call gives the same bits).

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
    given = out is not None
    if not given:
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
    if given:
        torch.autograd.graph.increment_version(out)
    return out


# ------------------------------------------------------------------------- clipping
def _dense(t: torch.Tensor) -> bool:
    """Whether t's elements fill one run of memory, in any order of its axes."""
    if t.numel() == 0:
        return True
    want = 1
    for size, stride in sorted(((n, s) for n, s in zip(t.shape, t.stride()) if n != 1), key=lambda x: x[1]):
        if stride != want:
            return False
        want *= size
    return True


def _same_strides(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether elements of equal indices lie at equal places (a and b have the same shape)."""
    return a.numel() == 0 or all(n == 1 or s == t for n, s, t in zip(a.shape, a.stride(), b.stride()))


def clip_grad_norm(tensors: Sequence[torch.Tensor], max_norm: float,
                   out: Optional[Sequence[torch.Tensor]] = None,
                   workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, List[torch.Tensor]]:
    """The 2-norm over all elements of `tensors` (float32 scalar on the GPU), and the tensors
    scaled by min(1, max_norm / (norm + 1e-6)): in place, or into `out` (tensors of the same
    shapes, types and strides). Nothing waits for the GPU.

    tensors: float32 or bfloat16, mixed as they come, each dense (its elements fill one run of
    memory), none overlapping another. max_norm: >= 0; math.inf only takes the norm, and leaves (or
    copies) the tensors as they are, whatever it is.
    """
    tensors = list(tensors)
    outs = tensors if out is None else list(out)
    n = len(tensors)
    if n == 0:
        raise ValueError("clip_grad_norm needs at least one tensor")
    if len(outs) != n:
        raise ValueError(f"{len(outs)} out tensors for {n}")
    if not max_norm >= 0:
        raise ValueError(f"max_norm must be at least 0, got {max_norm}")
    # one attribute of all tensors at a time: a model has many, and most calls are small
    device = tensors[0].device
    _on_gpu(device, workspace=workspace)
    dtypes = [t.dtype for t in tensors]
    if not set(dtypes) <= _CODES.keys():
        raise TypeError(f"tensors must be float32 or bfloat16, got {set(dtypes)}")
    index = device.index
    if not all([t.get_device() == index for t in tensors]):
        raise ValueError(f"tensors must all be on {device}")
    plain = all([t.is_contiguous() for t in tensors])
    if not plain:
        for i, t in enumerate(tensors):
            if not _dense(t):
                raise ValueError(f"tensor {i} is not dense: shape {tuple(t.shape)}, strides {t.stride()}")
    src = [t.data_ptr() for t in tensors]
    if out is None:
        dst = src
    else:
        if not all([o.get_device() == index for o in outs]) or [o.dtype for o in outs] != dtypes or \
                [o.shape for o in outs] != [t.shape for t in tensors] or \
                (not (plain and all([o.is_contiguous() for o in outs])) and
                 not all(_same_strides(o, t) for o, t in zip(outs, tensors))):
            raise ValueError("out tensors must have their tensors' device, shapes, types and strides")
        dst = [o.data_ptr() for o in outs]
    pointers, sizes, words = C.c_void_p * n, C.c_int64 * n, C.c_int32 * n
    norm = torch.empty((), dtype=torch.float32, device=device)
    if workspace is None:
        workspace = empty_workspace(lib().mips_clip_workspace_size(n), device)
    _check(lib().mips_clip_grad_norm(pointers(*src), pointers(*dst), sizes(*[t.numel() for t in tensors]),
                                     words(*[_CODES[t] for t in dtypes]), n, float(max_norm), _ptr(norm),
                                     _ptr(workspace), workspace.numel(), _stream(device)),
           "mips_clip_grad_norm")
    # written through their addresses: autograd would not notice a saved tensor that changed
    torch.autograd.graph.increment_version(outs)
    return norm, outs
