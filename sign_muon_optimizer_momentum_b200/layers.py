"""Per-worker gradients of a token model around its hidden matrices.

SignMuonStep takes one gradient per (matrix, worker).  The functions here
produce such gradients for the parts of a language model that are not hidden
matrices: the embedding table, the layer norms, and the loss that starts the
backward pass.  Each works on one batch that holds the rows of all workers
(worker m owns rows [splits[m], splits[m + 1]), equal shares by default) and
returns a list of one gradient per worker: grads[i * n_workers + m] of
SignMuonStep.step for that matrix (a norm's weight is a matrix of one row,
`weight.view(1, -1)`).

  embedding_forward     y = scale * table[ids]
  embedding_backward    the table's gradient per worker
  layer_norm_forward    y, and the rows' mean and 1 / std
  layer_norm_backward   dx, and the weight's and bias's gradients per worker
  distill_loss          losses against a teacher's top logits, per worker and row
  distill_loss_and_grad ... and the logits' gradient

PyTorch is used only to allocate device buffers and to pick the stream (the
current one of the tensors' device); all arithmetic runs in libsignmuon.so.
Nothing synchronises, so every call can be captured into a CUDA graph, and
scratch is allocated per call, so calls on different streams (and captured
graphs) share nothing.  Tensors are fp32 or bf16 on one CUDA device; rows may
have any stride, columns must be adjacent.  Wrong arguments raise TypeError or
ValueError, failures in the library SignMuonError.
"""
from __future__ import annotations

import contextlib
import math
from typing import List, Optional, Sequence, Tuple

import torch

from . import _lib as L
from .step import _dtype_code

__all__ = ["embedding_forward", "embedding_backward", "layer_norm_forward", "layer_norm_backward", "distill_loss",
           "distill_loss_and_grad"]

_SAME_DEVICE = contextlib.nullcontext()


def _on(t: torch.Tensor):
    """The context in which t's device is the current one."""
    return _SAME_DEVICE if t.device.index == torch.cuda.current_device() else torch.cuda.device(t.device)


def _stream(t: torch.Tensor) -> int:
    # torch.cuda.current_stream(t.device).cuda_stream without the Stream
    # object, which takes as long to make as a small launch.
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _like(t: torch.Tensor) -> torch.Tensor:
    """A contiguous tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _cuda(t: torch.Tensor, what: str, like: Optional[torch.Tensor] = None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if like is not None and t.device != like.device:
        raise ValueError(f"{what} is on {t.device}, expected {like.device}")


def _rows(t: torch.Tensor, what: str) -> Tuple[int, int, int]:
    """(rows, columns, row stride) of a tensor of rows in its last dimension."""
    if t.dim() < 1:
        raise ValueError(f"{what}: expected rows in the last dimension")
    cols = t.shape[-1]
    if cols == 0:
        raise ValueError(f"{what}: expected at least one column")
    if t.is_contiguous():
        return t.numel() // cols, cols, cols
    if t.dim() != 2:
        try:
            t = t.view(-1, cols)
        except RuntimeError:
            raise ValueError(f"{what}: rows must have one stride") from None
    n, ld = t.shape[0], t.stride(0)
    if (cols > 1 and t.stride(1) != 1) or (n > 1 and ld < cols):
        raise ValueError(f"{what}: columns must be adjacent and rows must not overlap")
    return n, cols, max(ld, cols)


def _matrix(t: torch.Tensor, shape: Tuple[int, ...], dtype: torch.dtype, what: str, like: torch.Tensor) -> int:
    """Row stride of an output of this shape and type."""
    _cuda(t, what, like)
    if t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return _rows(t, what)[2]


def _ids(ids: torch.Tensor, what: str, like: torch.Tensor) -> bool:
    _cuda(ids, what, like)
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"{what}: expected int32 or int64, got {ids.dtype}")
    if not ids.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return ids.dtype == torch.int64


def _shares(rows: int, n_workers: int, splits: Optional[Sequence[int]]):
    """The workers' row offsets as a C array."""
    if not 1 <= n_workers <= L.SIGNMUON_MAX_WORKERS:
        raise ValueError(f"n_workers must be in [1, {L.SIGNMUON_MAX_WORKERS}]")
    if splits is None:
        if rows % n_workers:
            raise ValueError(f"{rows} rows do not divide into {n_workers} workers: give splits")
        splits = range(0, rows + 1, rows // n_workers) if rows else [0] * (n_workers + 1)
    elif len(splits) != n_workers + 1 or splits[0] != 0 or splits[-1] != rows or \
            any(a > b for a, b in zip(splits, splits[1:])):
        raise ValueError(f"splits must be {n_workers + 1} non-decreasing offsets from 0 to {rows}")
    return L._offsets(splits)


def _per_worker(n: int, shape: Tuple[int, ...], dtype: torch.dtype, device) -> Tuple[List[torch.Tensor], List[int]]:
    """n tensors, each 16-byte aligned as the step wants them, and their
    addresses."""
    nbytes = math.prod(shape) * dtype.itemsize
    if n == 1 or nbytes % 16 == 0:
        whole = torch.empty((n, *shape), dtype=dtype, device=device)
        p = whole.data_ptr()
        return list(whole.unbind(0)), [p + i * nbytes for i in range(n)]
    out = [torch.empty(shape, dtype=dtype, device=device) for _ in range(n)]
    return out, [g.data_ptr() for g in out]


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- embedding
def embedding_forward(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, dtype: Optional[torch.dtype] = None,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """scale * table[ids], of shape ids.shape + (columns,) and of `dtype` (the
    table's by default); zero where an id is outside the table (padding).

    table: [vocab, columns]; ids: int32 or int64, contiguous, any shape."""
    _cuda(table, "table")
    if table.dim() != 2:
        raise ValueError("table must have two dimensions")
    wide = _ids(ids, "ids", table)
    vocab, cols, ld = _rows(table, "table")
    if vocab == 0:
        raise ValueError("table must have at least one row")
    dtype = dtype or table.dtype
    code, out_code = _dtype_code(table.dtype), _dtype_code(dtype)
    if out is None:
        out, ld_y = torch.empty((*ids.shape, cols), dtype=dtype, device=table.device), cols
    else:
        ld_y = _matrix(out, (*ids.shape, cols), dtype, "out", table)
    with _on(table):
        L.signmuon_embedding_forward((vocab, cols), code, table.data_ptr(), ld, ids.numel(), wide, ids.data_ptr(), scale,
                                     out_code, out.data_ptr(), ld_y, _stream(table))
    return out


def embedding_backward(ids: torch.Tensor, grad_out: torch.Tensor, vocab: int, n_workers: int = 1,
                       splits: Optional[Sequence[int]] = None, scale: float = 1.0, dtype: Optional[torch.dtype] = None,
                       out: Optional[Sequence[torch.Tensor]] = None, accumulate: bool = False) -> List[torch.Tensor]:
    """The gradient of the table, [vocab, columns] of `dtype` (grad_out's by
    default), for each worker: scale * the sum of grad_out's rows by id.

    ids: as in the forward call, flattened in token order; grad_out: rows of
    the same tokens.  out: the workers' gradient buffers, contiguous; with
    accumulate=True the sums are added to them (a table that the output layer
    shares) and only rows that a token names are touched."""
    _cuda(grad_out, "grad_out")
    wide = _ids(ids, "ids", grad_out)
    rows, cols, ld = _rows(grad_out, "grad_out")
    if ids.numel() != rows:
        raise ValueError(f"{ids.numel()} ids for {rows} rows of grad_out")
    if vocab < 1:
        raise ValueError("vocab must be >= 1")
    dtype = dtype or grad_out.dtype
    code, grad_code = _dtype_code(grad_out.dtype), _dtype_code(dtype)
    shares = _shares(rows, n_workers, splits)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out, ptrs = _per_worker(n_workers, (vocab, cols), dtype, grad_out.device)
    else:
        out = list(out)
        if len(out) != n_workers:
            raise ValueError(f"expected {n_workers} gradient buffers, got {len(out)}")
        for m, g in enumerate(out):
            _matrix(g, (vocab, cols), dtype, f"out[{m}]", grad_out)
            if not g.is_contiguous():
                raise ValueError(f"out[{m}] must be contiguous")
        ptrs = [g.data_ptr() for g in out]
    with _on(grad_out):
        ws = _workspace(L.signmuon_embedding_backward_workspace_bytes((vocab, cols), shares), grad_out.device)
        L.signmuon_embedding_backward((vocab, cols), shares, wide, ids.data_ptr(), code, grad_out.data_ptr(), ld, scale,
                                      accumulate, grad_code, ptrs, ws.data_ptr(), ws.numel(),
                                      _stream(grad_out))
    return out


# --------------------------------------------------------------- layer norm
def _vector(t: torch.Tensor, cols: int, dtype: Optional[torch.dtype], what: str, like: torch.Tensor) -> None:
    _cuda(t, what, like)
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if t.numel() != cols or t.shape[-1:] != (cols,) or not t.is_contiguous():
        raise ValueError(f"{what}: expected {cols} contiguous elements")


def layer_norm_forward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                       out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, mean, rstd): y = (x - mean) * rstd * weight + bias over x's last
    dimension, of x's shape and type; mean and rstd = 1 / sqrt(variance + eps)
    are fp32 of x.shape[:-1].  weight, bias: one type, [columns] or
    [1, columns].  out may be x."""
    _cuda(x, "x")
    rows, cols, ld = _rows(x, "x")
    _vector(weight, cols, None, "weight", x)
    if bias is not None:
        _vector(bias, cols, weight.dtype, "bias", x)
    if not eps >= 0:
        raise ValueError("eps must be >= 0")
    code, w_code = _dtype_code(x.dtype), _dtype_code(weight.dtype)
    if out is None:
        out, ld_y = _like(x), cols
    else:
        ld_y = _matrix(out, x.shape, x.dtype, "out", x)
    mean, rstd = torch.empty((2, *x.shape[:-1]), dtype=torch.float32, device=x.device).unbind(0)
    with _on(x):
        L.signmuon_layer_norm_forward(rows, cols, code, x.data_ptr(), ld, w_code, weight.data_ptr(),
                                      None if bias is None else bias.data_ptr(), eps, out.data_ptr(), ld_y,
                                      mean.data_ptr(), rstd.data_ptr(), _stream(x))
    return out, mean, rstd


def layer_norm_backward(grad_out: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor,
                        rstd: torch.Tensor, n_workers: int = 1, splits: Optional[Sequence[int]] = None, bias: bool = True,
                        out: Optional[torch.Tensor] = None
                        ) -> Tuple[torch.Tensor, List[torch.Tensor], Optional[List[torch.Tensor]]]:
    """(dx, [dweight of each worker], [dbias of each worker] or None), the
    gradients of layer_norm_forward; mean and rstd are what it returned.
    dweight and dbias have the weight's shape and type; out (dx) may be
    grad_out."""
    _cuda(grad_out, "grad_out")
    _cuda(x, "x", grad_out)
    rows, cols, ld_dy = _rows(grad_out, "grad_out")
    if x.shape != grad_out.shape:
        raise ValueError(f"x is {tuple(x.shape)}, grad_out {tuple(grad_out.shape)}")
    if x.dtype != grad_out.dtype:
        raise TypeError(f"x is {x.dtype}, grad_out {grad_out.dtype}")
    ld_x = _rows(x, "x")[2]
    _vector(weight, cols, None, "weight", x)
    for t, what in ((mean, "mean"), (rstd, "rstd")):
        _cuda(t, what, x)
        if t.dtype != torch.float32:
            raise TypeError(f"{what}: expected torch.float32, got {t.dtype}")
        if t.numel() != rows or not t.is_contiguous():
            raise ValueError(f"{what}: expected {rows} contiguous elements")
    code, w_code = _dtype_code(x.dtype), _dtype_code(weight.dtype)
    shares = _shares(rows, n_workers, splits)
    if out is None:
        out, ld_dx = _like(x), cols
    else:
        ld_dx = _matrix(out, x.shape, x.dtype, "out", x)
    grads, ptrs = _per_worker(n_workers * (2 if bias else 1), weight.shape, weight.dtype, x.device)
    dw, db = grads[:n_workers], grads[n_workers:] if bias else None
    with _on(x):
        ws = _workspace(L.signmuon_layer_norm_backward_workspace_bytes(cols, shares), x.device)
        L.signmuon_layer_norm_backward(cols, shares, code, grad_out.data_ptr(), ld_dy, x.data_ptr(), ld_x, w_code,
                                       weight.data_ptr(), mean.data_ptr(), rstd.data_ptr(), out.data_ptr(), ld_dx,
                                       ptrs[:n_workers], ptrs[n_workers:] if bias else None,
                                       ws.data_ptr(), ws.numel(), _stream(x))
    return out, dw, db


# ------------------------------------------------------------- distillation
def _distill(logits, top_ids, top_logits, n_workers, splits, temperature, grad_scale, with_grad, out):
    _cuda(logits, "logits")
    rows, vocab, ld = _rows(logits, "logits")
    wide = _ids(top_ids, "top_ids", logits)
    _cuda(top_logits, "top_logits", logits)
    if top_ids.shape[:-1] != logits.shape[:-1] or top_logits.shape != top_ids.shape:
        raise ValueError("top_ids and top_logits must have one row of entries for each row of logits")
    top = top_ids.shape[-1]
    if not 1 <= top <= 1024:
        raise ValueError("between 1 and 1024 top logits are supported")
    if not top_logits.is_contiguous():
        raise ValueError("top_logits must be contiguous")
    if not 0 < temperature < float("inf"):
        raise ValueError("temperature must be positive and finite")
    code, top_code = _dtype_code(logits.dtype), _dtype_code(top_logits.dtype)
    shares = _shares(rows, n_workers, splits)
    loss = torch.empty(n_workers, dtype=torch.float32, device=logits.device)
    row_loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=logits.device)
    ld_d = 0
    if with_grad:
        if out is None:
            out, ld_d = _like(logits), vocab
        else:
            ld_d = _matrix(out, logits.shape, logits.dtype, "out", logits)
    with _on(logits):
        ws = _workspace(L.signmuon_distill_workspace_bytes(rows, top), logits.device)
        L.signmuon_distill_loss(vocab, shares, code, logits.data_ptr(), ld, top, wide, top_ids.data_ptr(), top_code,
                                top_logits.data_ptr(), temperature, grad_scale, loss.data_ptr(), row_loss.data_ptr(),
                                out.data_ptr() if with_grad else None, ld_d, ws.data_ptr(), ws.numel(), _stream(logits))
    return loss, row_loss, out


def distill_loss(logits: torch.Tensor, top_ids: torch.Tensor, top_logits: torch.Tensor, n_workers: int = 1,
                 splits: Optional[Sequence[int]] = None, temperature: float = 1.0) -> Tuple[torch.Tensor, torch.Tensor]:
    """(loss, row_loss) against the teacher's top logits: row_loss = T^2 *
    KL(softmax(top_logits / T) || softmax(logits / T) at top_ids), fp32 of
    logits.shape[:-1], and loss[m] the mean over worker m's rows, fp32
    [n_workers].

    logits: rows of the vocabulary; top_ids (int32 or int64), top_logits:
    contiguous rows of 1 to 1024 entries; an entry with an id outside the
    vocabulary or a logit of -inf is absent, and a row without entries is
    ignored (loss 0, not counted in the mean)."""
    return _distill(logits, top_ids, top_logits, n_workers, splits, temperature, 1.0, False, None)[:2]


def distill_loss_and_grad(logits: torch.Tensor, top_ids: torch.Tensor, top_logits: torch.Tensor, n_workers: int = 1,
                          splits: Optional[Sequence[int]] = None, temperature: float = 1.0, grad_scale: float = 1.0,
                          out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(loss, row_loss, dlogits) in one pass over the logits: what distill_loss
    returns, and grad_scale * the gradient of each worker's loss by its rows'
    logits, of the logits' shape and type (zero in ignored rows).  out may be
    logits."""
    return _distill(logits, top_ids, top_logits, n_workers, splits, temperature, grad_scale, True, out)
