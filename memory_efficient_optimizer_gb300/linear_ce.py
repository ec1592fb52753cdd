"""PyTorch front end of the cross entropy of a linear output layer
(include/linear_ce.h): the loss from the hidden states and the layer's weight,
with the gradients of both, without the logits.  A training step is::

    hidden = model.body(tokens)                       # [batch, seq, dim]
    out = linear_cross_entropy(hidden.detach(), head.weight, targets)
    hidden.backward(out.grad_hidden)                  # on to the other weights
    head.weight.grad = out.grad_weight
    optimizer.step()

``need_grad=False`` gives the loss and the tokens' log-probabilities alone.

As in losses.py these functions check and marshal arguments, allocate the
outputs and the workspace, and make one call into the library, which does all
of the arithmetic and waits for nothing.  Values of targets are not looked at
on the host; the header says how bad ones show in the results.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple, Optional

import torch

from . import binding as B
from .losses import _DTYPES, _FP32, _INDEX, _NO_ROWS, _context, _raw_stream, _rows, _strides, _written

# The C structs, packed here in one step each, as in losses.py.
_HIDDEN = struct.Struct("@Piqqqqq")
_WEIGHT = struct.Struct("@Piqqi4x")
_TARGETS = struct.Struct("@Pqqiq")
_ARGS = struct.Struct("@Pqqddd")
for _s, _c in ((_HIDDEN, B.linear_ce_hidden), (_WEIGHT, B.linear_ce_weight), (_TARGETS, B.loss_targets),
               (_ARGS, B.linear_ce_args)):
    assert _s.size == ctypes.sizeof(_c), _c.__name__


class LinearCrossEntropy(NamedTuple):
    loss: torch.Tensor                    # fp32 scalar
    grad_hidden: Optional[torch.Tensor]
    grad_weight: Optional[torch.Tensor]
    logp: torch.Tensor                    # fp32, the targets' shape; 0 where ignored
    lse: torch.Tensor                     # fp32, ln sum exp of the scaled logits; 0 where ignored


def _hidden(name, t, shape=None, device=None):
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be a float32 or bfloat16 tensor")
    size, st = t.shape, t.stride()
    if len(size) == 3:
        batch, sb = size[0], st[0]
    elif len(size) == 2:
        batch, sb = 1, 0
    else:
        raise ValueError(f"{name} must be [tokens, dim] or [batch, seq, dim]")
    if shape is not None and (size != shape or t.get_device() != device):
        raise ValueError(f"{name} must have the hidden states' shape and device")
    if st[-1] != 1 and size[-1] != 1:
        raise ValueError(f"{name}: the innermost stride must be 1")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return _HIDDEN.pack(t.data_ptr(), _DTYPES[t.dtype], batch, size[-2], size[-1], sb, st[-2])


def _weight(name, t, dim, device, vocab=None, accumulate=False):
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be a float32 or bfloat16 tensor")
    size, st = t.shape, t.stride()
    if len(size) != 2 or size[1] != dim or t.get_device() != device or (vocab is not None and size[0] != vocab):
        raise ValueError(f"{name} must be [{'vocab' if vocab is None else vocab}, {dim}] on the hidden states' device")
    if st[1] != 1 and dim != 1:
        raise ValueError(f"{name}: the innermost stride must be 1")
    return _WEIGHT.pack(t.data_ptr(), _DTYPES[t.dtype], size[0], st[0], 1 if accumulate else 0)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(tokens, dim, hidden_type, vocab, weight_type, stride, aligned, grad_hidden, grad_weight):
    """Bytes of workspace by what they depend on; grad_hidden, grad_weight: types, or None."""
    h = _HIDDEN.pack(0, hidden_type, 1, tokens, dim, 0, dim)
    w = _WEIGHT.pack(0 if aligned else 8, weight_type, vocab, stride, 0)
    return B.linear_ce_workspace_size(h, w, None if grad_hidden is None else _HIDDEN.pack(0, grad_hidden, 1, tokens, dim, 0, dim),
                                      None if grad_weight is None else _WEIGHT.pack(0, grad_weight, vocab, dim, 0))


def linear_cross_entropy(hidden, weight, targets, *, weights=None, z_loss: float = 0.0, temperature: float = 1.0,
                         ignore_index: int = -100, grad_hidden=None, grad_weight=None, accumulate: bool = False,
                         grad_scale: float = 1.0, need_grad: bool = True, stream=None) -> LinearCrossEntropy:
    """Cross entropy of ``softmax(hidden @ weight.T / temperature)``.

    ``hidden`` [tokens, dim] or [batch, seq, dim] and ``weight`` [vocab, dim]
    are bfloat16, or float32, which is rounded to bfloat16 first; ``targets``
    (int32 or int64) has the tokens' shape, and so has ``weights`` (float32, any
    strides).  With lse = ln sum exp of a token's scaled logits::

        loss = sum(w (z_loss lse^2 - logp))

    with w = weights, or 1 / (number of targets that are not ignore_index).
    The gradients have the hidden states' and the weight's types, or are written
    into ``grad_hidden`` (may be ``hidden`` itself) and ``grad_weight``, float32
    or bfloat16; with ``accumulate`` the weight's is added to what
    ``grad_weight`` holds, as micro-batches do.  ``grad_scale`` multiplies the
    gradients.
    """
    ctx = _context(hidden, stream)
    if ctx is not None:
        with ctx:
            return linear_cross_entropy(hidden, weight, targets, weights=weights, z_loss=z_loss, temperature=temperature,
                                        ignore_index=ignore_index, grad_hidden=grad_hidden, grad_weight=grad_weight,
                                        accumulate=accumulate, grad_scale=grad_scale, need_grad=need_grad)
    h = _hidden("hidden", hidden)
    dev, shape, dim = hidden.get_device(), hidden.shape[:-1], hidden.shape[-1]
    w = _weight("weight", weight, dim, dev)
    code = _INDEX.get(targets.dtype) if isinstance(targets, torch.Tensor) else None
    if code is None:
        raise ValueError("targets must be an int32 or int64 tensor")
    if targets.shape != shape or targets.get_device() != dev:
        raise ValueError(f"targets must have shape {list(shape)} on the hidden states' device")
    y = _TARGETS.pack(targets.data_ptr(), *_strides(targets, shape), code, ignore_index)
    args = _ARGS.pack(*(_NO_ROWS if weights is None else _rows("weights", weights, shape, dev)), temperature, z_loss, grad_scale)
    if accumulate and grad_weight is None:
        raise ValueError("accumulate needs grad_weight")
    device = hidden.device
    gh = gw = None
    given_h, given_w = grad_hidden, grad_weight
    if need_grad:
        if grad_hidden is None:
            grad_hidden = torch.empty(hidden.shape, dtype=hidden.dtype, device=device)
        if grad_weight is None:
            grad_weight = torch.empty(weight.shape, dtype=weight.dtype, device=device)
        gh = _hidden("grad_hidden", grad_hidden, hidden.shape, dev)
        gw = _weight("grad_weight", grad_weight, dim, dev, weight.shape[0], accumulate)
    elif grad_hidden is not None or grad_weight is not None:
        raise ValueError("grad_hidden or grad_weight was given with need_grad=False")
    loss = torch.empty((), dtype=_FP32, device=device)
    logp = torch.empty(shape, dtype=_FP32, device=device)
    lse = torch.empty(shape, dtype=_FP32, device=device)
    n = _workspace_bytes(shape.numel(), dim, _DTYPES[hidden.dtype], weight.shape[0], _DTYPES[weight.dtype], weight.stride(0),
                         weight.data_ptr() % 16 == 0, None if gh is None else _DTYPES[grad_hidden.dtype],
                         None if gw is None else _DTYPES[grad_weight.dtype])
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    B.linear_ce(h, w, y, args, gh, gw, loss.data_ptr(), logp.data_ptr(), lse.data_ptr(),
                ws.data_ptr(), n, _raw_stream(dev))
    _written(given_h)
    _written(given_w)
    return LinearCrossEntropy(loss, grad_hidden, grad_weight, logp, lse)


__all__ = ["LinearCrossEntropy", "linear_cross_entropy"]
