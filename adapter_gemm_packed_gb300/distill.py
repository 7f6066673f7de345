"""Distillation from a teacher's top logits: loss of every token and the gradient at the logits, in one call."""
from __future__ import annotations

import torch

from . import _mlora as M
from .attention import _int32, _launch_device, _on, _refuse, _vector


def distill_loss(logits, ids, teacher, weight=None, *, temperature=1.0, grad=True, dlogits=None, stream=None):
    """``logits`` [n_tokens, vocab] bf16 or fp32 (rows may be longer than vocab: any row stride),
    ``ids`` int32 and ``teacher`` fp32 [n_tokens, top]: the teacher's largest logits and where they
    are (an id outside of the vocabulary is padding), ``weight`` fp32 [n_tokens] (default 1).

        loss = weight T^2 KL(softmax(teacher / T) || softmax(logits / T))

    over each row's entries.  Returns (loss fp32 [n_tokens], dlogits): the gradient of ``loss.sum()``,
    which ``logits.backward(dlogits)`` hands on; None with ``grad=False``.  Rows of weight zero have loss
    and gradient zero.

    A new ``dlogits`` is dense.  Where the logits' rows are parts of wider ones, a ``dlogits`` given with the same row stride
    and the same offset from a 16-byte boundary is much faster (8192 x 127,993 of 128,000 columns: 0.73 milliseconds
    against 4.6)."""
    where = "distill_loss"
    dev = _launch_device(stream)
    if logits.dim() != 2 or logits.get_device() != dev or (logits.shape[1] > 1 and logits.stride(1) != 1):
        _refuse(where, f"logits must be [n_tokens, vocab] on GPU {dev} with contiguous rows")
    if logits.dtype is torch.bfloat16:
        code = M.MLORA_BF16
    elif logits.dtype is torch.float32:
        code = M.MLORA_F32
    else:
        _refuse(where, f"logits are bf16 or fp32, not {logits.dtype}", M.MLORA_ERR_UNSUPPORTED)
    n, v = logits.shape[0], _int32(where, "vocab", logits.shape[1])
    if ids.dim() != 2:
        _refuse(where, "ids must be [n_tokens, top]")
    top = _int32(where, "top", ids.shape[1])
    a = (_vector(ids, where, "ids", (n, top), torch.int32, dev),
         _vector(teacher, where, "teacher", (n, top), torch.float32, dev),
         None if weight is None else _vector(weight, where, "weight", (n,), torch.float32, dev))
    with _on(stream, dev) as s:
        loss = torch.empty(n, dtype=torch.float32, device=logits.device)
        if not grad:
            dlogits = None
        elif dlogits is None:
            dlogits = torch.empty((n, v), dtype=logits.dtype, device=logits.device)
        elif (dlogits.dtype is not logits.dtype or dlogits.get_device() != dev or dlogits.shape != logits.shape
              or (v > 1 and dlogits.stride(1) != 1)):
            _refuse(where, "dlogits must be of the logits' type, shape and device, with contiguous rows")
        # a single row has no stride to keep to
        p = M.mlora_distill_problem(n, v, top, code, temperature, logits.stride(0) if n > 1 else v,
                                    v if dlogits is None or n == 1 else dlogits.stride(0))
        M.mlora_distill_loss(p, logits.data_ptr(), *a, loss.data_ptr(), None if dlogits is None else dlogits.data_ptr(), s)
    return loss, dlogits
