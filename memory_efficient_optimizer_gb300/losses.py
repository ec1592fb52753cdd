"""PyTorch front end of the losses over a vocabulary (include/losses.h).

Each function takes the logits of a language model, ``[tokens, vocab]`` or
``[batch, seq, vocab]``, and answers the loss together with its gradient with
respect to the logits, so that a training step is::

    out = policy_loss(logits.detach(), targets, advantages, old_logp, ref_logp, kl_coef=0.05)
    logits.backward(out.grad)      # on to the weights
    optimizer.step()

``grad=logits.detach()`` writes the gradient over the logits: then the step
holds one tensor of that size where elementary operations hold several in fp32
(autograd must not need the logits' values any more, which a linear layer does
not; where it does, as behind a tanh, ``backward`` raises as after any change
in place).  ``need_grad=False`` gives the loss alone.

As elsewhere in this package PyTorch only provides memory and streams: these
functions check and marshal arguments, allocate the outputs and the workspace,
and make one call into the library, which does all of the arithmetic and waits
for nothing.  Values of targets, ids and offsets are not looked at on the host;
the header says how bad ones show in the results.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple, Optional

import torch

from . import binding as B

_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
# Handle of the current stream of a device (the torch.cuda call that makes a
# Stream object for it takes twenty times as long).
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)

_DTYPES = {torch.float32: B.ADAF_FLOAT32, torch.bfloat16: B.ADAF_BFLOAT16}
_INDEX = {torch.int32: B.LOSS_INT32, torch.int64: B.LOSS_INT64}
_NO_ROWS = (0, 0, 0)
_FP32 = torch.float32

# The C structs, packed here in one step each (a ctypes.Structure costs several
# times that, and for a few tokens the host's part is most of a call).
_LOGITS = struct.Struct("@Piqqqqqd")
_TARGETS = struct.Struct("@Pqqiq")
_GRAD = struct.Struct("@Pqqd")
_ROWS = struct.Struct("@Pqq")
_POLICY = struct.Struct("@PqqPqqPqqPqqddd")
_PREFERENCE = struct.Struct("@PqqqPiiiddd")
_DISTILL = struct.Struct("@PiqqPiqqiPqqPqqPqq")
for _s, _c in ((_LOGITS, B.loss_logits), (_TARGETS, B.loss_targets), (_GRAD, B.loss_grad), (_ROWS, B.loss_rows),
               (_POLICY, B.loss_policy_args), (_PREFERENCE, B.loss_preference_args), (_DISTILL, B.loss_distill_args)):
    assert _s.size == ctypes.sizeof(_c), _c.__name__


class TokenLogprobs(NamedTuple):
    logp: torch.Tensor        # fp32, the targets' shape; 0 where ignored
    stats: torch.Tensor       # fp32 [..., 2], for token_logprobs_backward


class PolicyLoss(NamedTuple):
    loss: torch.Tensor        # fp32 scalar
    grad: Optional[torch.Tensor]
    logp: torch.Tensor        # fp32 per token
    token_loss: torch.Tensor  # fp32 per token, before the weights


class PreferenceLoss(NamedTuple):
    loss: torch.Tensor        # fp32 scalar
    grad: Optional[torch.Tensor]
    pair_loss: torch.Tensor   # fp32 [pairs]
    rewards: torch.Tensor     # fp32 [2 pairs]: beta (logp - ref) summed, chosen then rejected
    logp: torch.Tensor        # fp32 per token


class DistillLoss(NamedTuple):
    loss: torch.Tensor        # fp32 scalar
    grad: Optional[torch.Tensor]
    token_loss: torch.Tensor  # fp32 per token, before the weights


def _context(logits, stream):
    """What to enter so that the logits' device and the call's stream are
    current (the library launches on the current device, and outputs and
    workspace are allocated for the stream that uses them); None if they are."""
    if stream is not None:
        if isinstance(logits, torch.Tensor) and logits.is_cuda and stream.device.index != logits.get_device():
            raise ValueError(f"stream is of {stream.device}, the logits are on {logits.device}")
        return torch.cuda.stream(stream)
    if isinstance(logits, torch.Tensor) and logits.is_cuda and logits.get_device() != _current_device():
        return torch.cuda.device(logits.device)
    return None


def _logits(logits, temperature):
    """The packed logits, the tokens' shape, their device's index."""
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _DTYPES:
        raise ValueError("logits must be a float32 or bfloat16 tensor")
    shape, st = logits.shape, logits.stride()
    if len(shape) == 2:
        batch, sb, ss = 1, 0, st[0]
    elif len(shape) == 3:
        batch, sb, ss = shape[0], st[0], st[1]
    else:
        raise ValueError("logits must be [tokens, vocab] or [batch, seq, vocab]")
    if st[-1] != 1 and shape[-1] != 1:
        raise ValueError("logits: the innermost stride must be 1")
    if not logits.is_cuda:
        raise ValueError("logits must be on a CUDA device")
    return (_LOGITS.pack(logits.data_ptr(), _DTYPES[logits.dtype], batch, shape[-2], shape[-1], sb, ss, temperature),
            shape[:-1], logits.get_device())


def _strides(t, shape):
    st = t.stride()
    return (0, st[0]) if len(shape) == 1 else (st[0], st[1])


def _rows(name, t, shape, device, dtype=_FP32):
    """A per-token argument, with any strides: (pointer, stride_b, stride_s)."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype:
        if t.shape == shape and t.get_device() == device:
            st = t.stride()
            return (t.data_ptr(), 0, st[0]) if len(st) == 1 else (t.data_ptr(), st[0], st[1])
        raise ValueError(f"{name} must have shape {list(shape)} on the logits' device")
    raise ValueError(f"{name} must be a {str(dtype)[6:]} tensor")


def _targets(t, shape, device, ignore_index):
    code = _INDEX.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None:
        raise ValueError("targets must be an int32 or int64 tensor")
    return _TARGETS.pack(*_rows("targets", t, shape, device, t.dtype), code, ignore_index)


def _is_cut(shape, st):
    """Whole rows of sequences that are a few tokens longer: at most 4, and at
    most an eighth, which is what a gradient with the gaps takes in memory."""
    return st[1] == shape[2] and shape[1] * shape[2] < st[0] <= (shape[1] + min(4, shape[1] // 8)) * shape[2]


def _gradient(logits, grad, need_grad, scale, device):
    """(tensor or None, packed or None) of the gradient."""
    if grad is None:
        if not need_grad:
            return None, None
        shape, st = logits.shape, logits.stride()
        if len(shape) == 3 and shape[0] > 1 and shape[2] * logits.element_size() % 16 and _is_cut(shape, st):
            # Views such as logits[:, :-1] of rows that are no multiple of 16
            # bytes: a gradient with the same strides has its rows' 16-byte
            # boundaries where the logits' are (a contiguous one of 999 rows of
            # 50257 fp32 values takes 71 us in the backward pass, this 59).
            whole = torch.empty((shape[0] - 1) * st[0] + shape[1] * shape[2], dtype=logits.dtype, device=logits.device)
            grad = whole.as_strided(shape, st)
        else:
            grad = torch.empty(shape, dtype=logits.dtype, device=logits.device)
    else:
        if not need_grad:
            raise ValueError("grad was given with need_grad=False")
        if not isinstance(grad, torch.Tensor) or grad.dtype != logits.dtype:
            raise ValueError("grad must have the logits' dtype")
        if grad.shape != logits.shape or grad.get_device() != device:
            raise ValueError("grad must have the logits' shape and device")
        if grad.stride(-1) != 1 and grad.shape[-1] != 1:
            raise ValueError("grad: the innermost stride must be 1")
    st = grad.stride()
    return grad, _GRAD.pack(grad.data_ptr(), st[0] if len(st) == 3 else 0, st[-2], scale)


def _written(grad):
    """Tells autograd of a caller's tensor that it has other values now."""
    if grad is not None:
        torch.autograd.graph.increment_version(grad)


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(tokens, pairs):
    return B.loss_workspace_size(tokens, pairs)


def _workspace(shape, device, pairs=0):
    n = _workspace_bytes(shape.numel(), pairs)
    return torch.empty(n, dtype=torch.uint8, device=device), n


def token_logprobs(logits, targets, *, temperature: float = 1.0, ignore_index: int = -100,
                   stream=None) -> TokenLogprobs:
    """Log-probability of each target under softmax(logits / temperature)."""
    ctx = _context(logits, stream)
    if ctx is not None:
        with ctx:
            return token_logprobs(logits, targets, temperature=temperature, ignore_index=ignore_index)
    x, shape, dev = _logits(logits, temperature)
    y = _targets(targets, shape, dev, ignore_index)
    device = logits.device
    logp = torch.empty(shape, dtype=_FP32, device=device)
    stats = torch.empty((*shape, 2), dtype=_FP32, device=device)
    B.loss_token_logprobs(x, y, logp.data_ptr(), stats.data_ptr(), _raw_stream(dev))
    return TokenLogprobs(logp, stats)


def token_logprobs_backward(logits, targets, stats, grad_logp, *, temperature: float = 1.0, ignore_index: int = -100,
                            grad=None, grad_scale: float = 1.0, stream=None) -> torch.Tensor:
    """Gradient of the logits, given that of the log-probabilities: the
    backward pass of token_logprobs under any loss.  ``stats`` is the forward
    pass's; targets, temperature and ignore_index are the same as there."""
    ctx = _context(logits, stream)
    if ctx is not None:
        with ctx:
            return token_logprobs_backward(logits, targets, stats, grad_logp, temperature=temperature,
                                           ignore_index=ignore_index, grad=grad, grad_scale=grad_scale)
    x, shape, dev = _logits(logits, temperature)
    y = _targets(targets, shape, dev, ignore_index)
    if (not isinstance(stats, torch.Tensor) or stats.dtype != _FP32 or stats.get_device() != dev
            or stats.shape != (*shape, 2) or not stats.is_contiguous()):
        raise ValueError(f"stats must be contiguous float32 {[*shape, 2]} on the logits' device")
    d = _ROWS.pack(*_rows("grad_logp", grad_logp, shape, dev))
    out, g = _gradient(logits, grad, True, grad_scale, dev)
    B.loss_token_logprobs_backward(x, y, stats.data_ptr(), d, g, _raw_stream(dev))
    _written(grad)
    return out


def policy_loss(logits, targets, advantages, old_logp=None, ref_logp=None, *, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_coef: float = 0.0, weights=None, temperature: float = 1.0,
                ignore_index: int = -100, grad=None, grad_scale: float = 1.0, need_grad: bool = True,
                stream=None) -> PolicyLoss:
    """Clipped policy loss with a KL term.

    Per token, with r = exp(logp - old_logp) (1 without old_logp) and
    d = ref_logp - logp::

        l = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + kl_coef (exp(d) - d - 1)

    The loss is the mean of l over the tokens whose target is not
    ignore_index, or sum(weights * l).  Per-token arguments have the targets'
    shape and any strides: ``advantages[:, None].expand(batch, seq)`` gives a
    sequence one advantage.
    """
    ctx = _context(logits, stream)
    if ctx is not None:
        with ctx:
            return policy_loss(logits, targets, advantages, old_logp, ref_logp, clip_low=clip_low, clip_high=clip_high,
                               kl_coef=kl_coef, weights=weights, temperature=temperature, ignore_index=ignore_index,
                               grad=grad, grad_scale=grad_scale, need_grad=need_grad)
    x, shape, dev = _logits(logits, temperature)
    y = _targets(targets, shape, dev, ignore_index)
    args = _POLICY.pack(*_rows("advantages", advantages, shape, dev),
                        *(_NO_ROWS if old_logp is None else _rows("old_logp", old_logp, shape, dev)),
                        *(_NO_ROWS if ref_logp is None else _rows("ref_logp", ref_logp, shape, dev)),
                        *(_NO_ROWS if weights is None else _rows("weights", weights, shape, dev)),
                        clip_low, clip_high, kl_coef)
    out, g = _gradient(logits, grad, need_grad, grad_scale, dev)
    device = logits.device
    loss = torch.empty((), dtype=_FP32, device=device)
    logp = torch.empty(shape, dtype=_FP32, device=device)
    token = torch.empty(shape, dtype=_FP32, device=device)
    ws, n = _workspace(shape, device)
    B.loss_policy(x, y, args, g, loss.data_ptr(), logp.data_ptr(), token.data_ptr(), ws.data_ptr(), n,
                  _raw_stream(dev))
    _written(grad)
    return PolicyLoss(loss, out, logp, token)


def preference_loss(logits, targets, ref_logp=None, *, seq_offsets=None, beta: float = 0.1,
                    label_smoothing: float = 0.0, kind: str = "sigmoid", margin: float = 0.0, average: bool = False,
                    temperature: float = 1.0, ignore_index: int = -100, grad=None, grad_scale: float = 1.0,
                    need_grad: bool = True, stream=None) -> PreferenceLoss:
    """Preference loss over pairs of sequences.

    Logits are ``[2 pairs, seq, vocab]``, the chosen sequences before the
    rejected ones (prompts and padding ignored through the targets), or
    ``[tokens, vocab]`` with ``seq_offsets`` (int32 or int64, [2 pairs + 1]) for
    sequences one after another.  With D a sequence's sum (or, with
    ``average``, mean) of logp - ref_logp (ref_logp None: 0) and
    h = D(chosen) - D(rejected), the loss is the mean over the pairs of::

        "sigmoid"   -(1 - e) ln s(beta h - margin) - e ln s(margin - beta h)     e = label_smoothing
        "hinge"     max(0, 1 + margin - beta h)
        "squared"   (h - 1 / (2 beta) - margin)^2
    """
    ctx = _context(logits, stream)
    if ctx is not None:
        with ctx:
            return preference_loss(logits, targets, ref_logp, seq_offsets=seq_offsets, beta=beta,
                                   label_smoothing=label_smoothing, kind=kind, margin=margin, average=average,
                                   temperature=temperature, ignore_index=ignore_index, grad=grad,
                                   grad_scale=grad_scale, need_grad=need_grad)
    x, shape, dev = _logits(logits, temperature)
    y = _targets(targets, shape, dev, ignore_index)
    code = B.LOSS_PREFERENCE_KINDS.get(kind)
    if code is None:
        raise ValueError(f"unknown kind {kind!r}: one of {sorted(B.LOSS_PREFERENCE_KINDS)}")
    if seq_offsets is None:
        if len(shape) != 2 or shape[0] < 2 or shape[0] % 2:
            raise ValueError("without seq_offsets the logits must be [2 pairs, seq, vocab]")
        pairs, at, odt = shape[0] // 2, 0, B.LOSS_INT64
    else:
        odt = _INDEX.get(seq_offsets.dtype) if isinstance(seq_offsets, torch.Tensor) else None
        if odt is None:
            raise ValueError("seq_offsets must be an int32 or int64 tensor")
        n = seq_offsets.numel()
        if (seq_offsets.dim() != 1 or n < 3 or n % 2 == 0 or seq_offsets.get_device() != dev
                or not seq_offsets.is_contiguous()):
            raise ValueError("seq_offsets must be contiguous [2 pairs + 1] on the logits' device")
        if len(shape) != 1:
            raise ValueError("with seq_offsets the logits must be [tokens, vocab]")
        pairs, at = (n - 1) // 2, seq_offsets.data_ptr()
    args = _PREFERENCE.pack(*(_NO_ROWS if ref_logp is None else _rows("ref_logp", ref_logp, shape, dev)), pairs, at,
                            odt, code, 1 if average else 0, beta, label_smoothing, margin)
    out, g = _gradient(logits, grad, need_grad, grad_scale, dev)
    device = logits.device
    loss = torch.empty((), dtype=_FP32, device=device)
    pair = torch.empty(pairs, dtype=_FP32, device=device)
    rewards = torch.empty(2 * pairs, dtype=_FP32, device=device)
    logp = torch.empty(shape, dtype=_FP32, device=device)
    ws, n = _workspace(shape, device, pairs)
    B.loss_preference(x, y, args, g, loss.data_ptr(), pair.data_ptr(), rewards.data_ptr(), logp.data_ptr(),
                      ws.data_ptr(), n, _raw_stream(dev))
    _written(grad)
    return PreferenceLoss(loss, out, pair, rewards, logp)


def distill_loss(logits, teacher_ids, teacher_logits, teacher_lse=None, *, mask=None, weights=None,
                 temperature: float = 1.0, grad=None, grad_scale: float = 1.0, need_grad: bool = True,
                 stream=None) -> DistillLoss:
    """Distillation from the top entries of a teacher's distribution.

    ``teacher_ids`` [..., k] (int32 or int64, distinct in a row, -1 for an entry
    that is not there) and ``teacher_logits`` [..., k] (float32 or bfloat16).
    Without ``teacher_lse`` the teacher is the softmax of its entries at the
    temperature; with it (ln sum exp(t / temperature) over the teacher's whole
    vocabulary) its mass on the words that are not listed is matched as one
    entry.  Per token the loss is temperature^2 KL(teacher || student).
    ``mask`` (bool) leaves tokens out; the loss is the mean over the others, or
    sum(weights * l).
    """
    ctx = _context(logits, stream)
    if ctx is not None:
        with ctx:
            return distill_loss(logits, teacher_ids, teacher_logits, teacher_lse, mask=mask, weights=weights,
                                temperature=temperature, grad=grad, grad_scale=grad_scale, need_grad=need_grad)
    x, shape, dev = _logits(logits, temperature)
    for name, t, types in (("teacher_ids", teacher_ids, _INDEX), ("teacher_logits", teacher_logits, _DTYPES)):
        if not isinstance(t, torch.Tensor) or t.dtype not in types:
            raise ValueError(f"{name} must be a tensor of {' or '.join(str(d)[6:] for d in types)}")
        if t.shape[:-1] != shape or t.get_device() != dev or t.dim() == len(shape):
            raise ValueError(f"{name} must have shape {[*shape, 'k']} on the logits' device")
        if t.stride(-1) != 1 and t.shape[-1] != 1:
            raise ValueError(f"{name}: the innermost stride must be 1")
    k = teacher_ids.shape[-1]
    if teacher_logits.shape[-1] != k:
        raise ValueError("teacher_ids and teacher_logits must have the same shape")
    args = _DISTILL.pack(teacher_ids.data_ptr(), _INDEX[teacher_ids.dtype], *_strides(teacher_ids, shape),
                         teacher_logits.data_ptr(), _DTYPES[teacher_logits.dtype], *_strides(teacher_logits, shape), k,
                         *(_NO_ROWS if teacher_lse is None else _rows("teacher_lse", teacher_lse, shape, dev)),
                         *(_NO_ROWS if mask is None else _rows("mask", mask, shape, dev, torch.bool)),
                         *(_NO_ROWS if weights is None else _rows("weights", weights, shape, dev)))
    out, g = _gradient(logits, grad, need_grad, grad_scale, dev)
    device = logits.device
    loss = torch.empty((), dtype=_FP32, device=device)
    token = torch.empty(shape, dtype=_FP32, device=device)
    ws, n = _workspace(shape, device)
    B.loss_distill(x, args, g, loss.data_ptr(), token.data_ptr(), ws.data_ptr(), n, _raw_stream(dev))
    _written(grad)
    return DistillLoss(loss, out, token)


__all__ = ["TokenLogprobs", "PolicyLoss", "PreferenceLoss", "DistillLoss", "token_logprobs",
           "token_logprobs_backward", "policy_loss", "preference_loss", "distill_loss"]
