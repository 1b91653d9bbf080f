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
current one of the tensors' device); all arithmetic runs in libsignmuon.so,
called through a compiled binding (csrc/layers_binding.cpp), which also checks
the arguments.  The functions are not differentiable by autograd: the backward
functions are called for that.
Nothing synchronises, so every call can be captured into a CUDA graph, and
scratch is allocated per call, so calls on different streams (and captured
graphs) share nothing.  The gradients that a call returns for the workers are
views of one allocation; out may not overlap an input unless stated (this is
checked, but for tensors of rows with two different strides), and a write to it
counts in its version as an in-place operation's.  Tensors are fp32 or bf16 on
one CUDA device; rows may have any stride, columns must be adjacent.  Wrong
arguments raise TypeError or ValueError, failures in the library SignMuonError.
"""
from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import torch

from . import _lib as L

__all__ = ["embedding_forward", "embedding_backward", "layer_norm_forward", "layer_norm_backward", "distill_loss",
           "distill_loss_and_grad"]

_native = None


def _load():
    """The compiled binding (raises if it or the library has not been built)."""
    global _native
    if _native is None:
        L.load()
        try:
            from . import _layers_native
        except ImportError as e:
            raise RuntimeError("_layers_native.so is missing or does not load: build it with "
                               "`python -m sign_muon_optimizer_momentum_b200.build`") from e
        _native = _layers_native
    return _native


# ---------------------------------------------------------------- embedding
def embedding_forward(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, dtype: Optional[torch.dtype] = None,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """scale * table[ids], of shape ids.shape + (columns,) and of `dtype` (the
    table's by default); zero where an id is outside the table (padding).

    table: [vocab, columns]; ids: int32 or int64, contiguous, any shape."""
    return _load().embedding_forward(table, ids, scale, dtype, out)


def embedding_backward(ids: torch.Tensor, grad_out: torch.Tensor, vocab: int, n_workers: int = 1,
                       splits: Optional[Sequence[int]] = None, scale: float = 1.0, dtype: Optional[torch.dtype] = None,
                       out: Optional[Sequence[torch.Tensor]] = None, accumulate: bool = False) -> List[torch.Tensor]:
    """The gradient of the table, [vocab, columns] of `dtype` (grad_out's by
    default), for each worker: scale * the sum of grad_out's rows by id.

    ids: as in the forward call, flattened in token order; grad_out: rows of
    the same tokens.  out: the workers' gradient buffers, contiguous; with
    accumulate=True the sums are added to them (a table that the output layer
    shares) and only rows that a token names are touched."""
    return _load().embedding_backward(ids, grad_out, vocab, n_workers, splits, scale, dtype, out, accumulate)


# --------------------------------------------------------------- layer norm
def layer_norm_forward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                       out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, mean, rstd): y = (x - mean) * rstd * weight + bias over x's last
    dimension, of x's shape and type; mean and rstd = 1 / sqrt(variance + eps)
    are fp32 of x.shape[:-1].  weight, bias: one type, [columns] or
    [1, columns].  out may be x."""
    return _load().layer_norm_forward(x, weight, bias, eps, out)


def layer_norm_backward(grad_out: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor,
                        rstd: torch.Tensor, n_workers: int = 1, splits: Optional[Sequence[int]] = None, bias: bool = True,
                        out: Optional[torch.Tensor] = None
                        ) -> Tuple[torch.Tensor, List[torch.Tensor], Optional[List[torch.Tensor]]]:
    """(dx, [dweight of each worker], [dbias of each worker] or None), the
    gradients of layer_norm_forward; mean and rstd are what it returned.
    dweight and dbias have the weight's shape and type; out (dx) may be
    grad_out."""
    return _load().layer_norm_backward(grad_out, x, weight, mean, rstd, n_workers, splits, bias, out)


# ------------------------------------------------------------- distillation
def distill_loss(logits: torch.Tensor, top_ids: torch.Tensor, top_logits: torch.Tensor, n_workers: int = 1,
                 splits: Optional[Sequence[int]] = None, temperature: float = 1.0) -> Tuple[torch.Tensor, torch.Tensor]:
    """(loss, row_loss) against the teacher's top logits: row_loss = T^2 *
    KL(softmax(top_logits / T) || softmax(logits / T) at top_ids), fp32 of
    logits.shape[:-1], and loss[m] the mean over worker m's rows, fp32
    [n_workers].

    logits: rows of the vocabulary; top_ids (int32 or int64), top_logits:
    contiguous rows of 1 to 1024 entries; an entry with an id outside the
    vocabulary or a logit of -inf is absent, and a row without entries is
    ignored (loss 0, not counted in the mean).  temperature: in [1e-6, 1e6],
    and logits / temperature within fp32's range.  Sums are fp32; rows that it
    does not give (logits of millions of temperatures, small divergences at
    temperatures above 8) are computed in fp64, which takes several times as
    long.

    One entry a row at temperature 1 is the cross entropy against next tokens:
    top_ids = targets[:, None], top_logits = zeros."""
    return _load().distill(logits, top_ids, top_logits, n_workers, splits, temperature, 1.0, False, None)[:2]


def distill_loss_and_grad(logits: torch.Tensor, top_ids: torch.Tensor, top_logits: torch.Tensor, n_workers: int = 1,
                          splits: Optional[Sequence[int]] = None, temperature: float = 1.0, grad_scale: float = 1.0,
                          out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(loss, row_loss, dlogits) in one pass over the logits: what distill_loss
    returns, and grad_scale * the gradient of each worker's loss by its rows'
    logits, of the logits' shape and type (zero in ignored rows).  out may be
    logits."""
    return _load().distill(logits, top_ids, top_logits, n_workers, splits, temperature, grad_scale, True, out)
