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
not).  ``need_grad=False`` gives the loss alone.

As elsewhere in this package PyTorch only provides memory and streams: these
functions check and marshal arguments, allocate the outputs and the workspace,
and make one call into the library, which does all of the arithmetic and waits
for nothing.  Values of targets, ids and offsets are not looked at on the host;
the header says how bad ones show in the results.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import binding as B

_DTYPES = {torch.float32: B.ADAF_FLOAT32, torch.bfloat16: B.ADAF_BFLOAT16}
_INDEX = {torch.int32: B.LOSS_INT32, torch.int64: B.LOSS_INT64}
_NO_ROWS = B.loss_rows(None, 0, 0)


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


class _Call:
    """The logits of one call, its device and stream."""

    def __init__(self, logits, temperature, stream):
        if not isinstance(logits, torch.Tensor) or logits.dtype not in _DTYPES:
            raise ValueError("logits must be a float32 or bfloat16 tensor")
        dim = logits.dim()
        if dim not in (2, 3):
            raise ValueError("logits must be [tokens, vocab] or [batch, seq, vocab]")
        shape, st = logits.shape, logits.stride()
        if st[-1] != 1 and shape[-1] != 1:
            raise ValueError("logits: the innermost stride must be 1")
        if logits.device.type != "cuda":
            raise ValueError("logits must be on a CUDA device")
        self.logits, self.device, self.shape = logits, logits.device, shape[:-1]
        if dim == 2:
            self.x = B.loss_logits(logits.data_ptr() or None, _DTYPES[logits.dtype], 1, shape[0], shape[1], 0, st[0],
                                   temperature)
        else:
            self.x = B.loss_logits(logits.data_ptr() or None, _DTYPES[logits.dtype], shape[0], shape[1], shape[2],
                                   st[0], st[1], temperature)
        self.tokens = self.x.batch * self.x.seq
        self._given = stream

    def _strides(self, t):
        st = t.stride()
        return (0, st[0]) if len(self.shape) == 1 else (st[0], st[1])

    def rows(self, name, t, dtype=torch.float32):
        """A per-token argument, with any strides."""
        if not isinstance(t, torch.Tensor) or t.dtype != dtype:
            raise ValueError(f"{name} must be a {str(dtype)[6:]} tensor")
        if t.device != self.device or t.shape != self.shape:
            raise ValueError(f"{name} must have shape {list(self.shape)} on the logits' device")
        return B.loss_rows(t.data_ptr() or None, *self._strides(t))

    def optional(self, name, t, dtype=torch.float32):
        return _NO_ROWS if t is None else self.rows(name, t, dtype)

    def targets(self, t, ignore_index):
        if not isinstance(t, torch.Tensor) or t.dtype not in _INDEX:
            raise ValueError("targets must be an int32 or int64 tensor")
        return B.loss_targets(self.rows("targets", t, t.dtype), _INDEX[t.dtype], ignore_index)

    def grad(self, grad, need_grad, scale):
        """(tensor or None, descriptor or None) of the gradient."""
        if grad is None:
            if not need_grad:
                return None, None
            grad = torch.empty(self.logits.shape, dtype=self.logits.dtype, device=self.device)
        else:
            if not need_grad:
                raise ValueError("grad was given with need_grad=False")
            if not isinstance(grad, torch.Tensor) or grad.dtype != self.logits.dtype:
                raise ValueError("grad must have the logits' dtype")
            if grad.device != self.device or grad.shape != self.logits.shape:
                raise ValueError("grad must have the logits' shape and device")
            if grad.stride(-1) != 1 and grad.shape[-1] != 1:
                raise ValueError("grad: the innermost stride must be 1")
        return grad, B.loss_grad(grad.data_ptr() or None, *self._strides(grad), scale)

    def empty(self, *shape):
        return torch.empty(shape, dtype=torch.float32, device=self.device)

    def workspace(self, pairs=0):
        n = B.loss_workspace_size(self.tokens, pairs)
        return torch.empty(n, dtype=torch.uint8, device=self.device), n

    def __enter__(self):
        """Makes the logits' device and the call's stream current: the library
        launches on the current device, and outputs and workspace are allocated
        for the stream that uses them."""
        self._before = None
        if self._given is not None:
            self._before = torch.cuda.stream(self._given)
        elif torch.cuda.current_device() != self.device.index:
            self._before = torch.cuda.device(self.device)
        if self._before is not None:
            self._before.__enter__()
        self.stream = torch.cuda.current_stream(self.device).cuda_stream
        return self

    def __exit__(self, *exc):
        if self._before is not None:
            self._before.__exit__(*exc)


def token_logprobs(logits, targets, *, temperature: float = 1.0, ignore_index: int = -100,
                   stream=None) -> TokenLogprobs:
    """Log-probability of each target under softmax(logits / temperature)."""
    c = _Call(logits, temperature, stream)
    y = c.targets(targets, ignore_index)
    with c:
        logp, stats = c.empty(*c.shape), c.empty(*c.shape, 2)
        B.loss_token_logprobs(c.x, y, logp.data_ptr(), stats.data_ptr(), c.stream)
    return TokenLogprobs(logp, stats)


def token_logprobs_backward(logits, targets, stats, grad_logp, *, temperature: float = 1.0, ignore_index: int = -100,
                            grad=None, grad_scale: float = 1.0, stream=None) -> torch.Tensor:
    """Gradient of the logits, given that of the log-probabilities: the
    backward pass of token_logprobs under any loss.  ``stats`` is the forward
    pass's; targets, temperature and ignore_index are the same as there."""
    c = _Call(logits, temperature, stream)
    y = c.targets(targets, ignore_index)
    if (not isinstance(stats, torch.Tensor) or stats.dtype != torch.float32 or stats.device != c.device
            or stats.shape != (*c.shape, 2) or not stats.is_contiguous()):
        raise ValueError(f"stats must be contiguous float32 {[*c.shape, 2]} on the logits' device")
    d = c.rows("grad_logp", grad_logp)
    with c:
        out, g = c.grad(grad, True, grad_scale)
        B.loss_token_logprobs_backward(c.x, y, stats.data_ptr(), d, g, c.stream)
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
    c = _Call(logits, temperature, stream)
    y = c.targets(targets, ignore_index)
    args = B.loss_policy_args(c.rows("advantages", advantages), c.optional("old_logp", old_logp),
                              c.optional("ref_logp", ref_logp), c.optional("weights", weights),
                              clip_low, clip_high, kl_coef)
    with c:
        out, g = c.grad(grad, need_grad, grad_scale)
        loss, logp, token = c.empty(), c.empty(*c.shape), c.empty(*c.shape)
        ws, n = c.workspace()
        B.loss_policy(c.x, y, args, g, loss.data_ptr(), logp.data_ptr() or None, token.data_ptr() or None,
                      ws.data_ptr(), n, c.stream)
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
    c = _Call(logits, temperature, stream)
    y = c.targets(targets, ignore_index)
    code = B.LOSS_PREFERENCE_KINDS.get(kind)
    if code is None:
        raise ValueError(f"unknown kind {kind!r}: one of {sorted(B.LOSS_PREFERENCE_KINDS)}")
    if seq_offsets is None:
        if len(c.shape) != 2 or c.shape[0] < 2 or c.shape[0] % 2:
            raise ValueError("without seq_offsets the logits must be [2 pairs, seq, vocab]")
        pairs, at, odt = c.shape[0] // 2, None, B.LOSS_INT64
    else:
        if not isinstance(seq_offsets, torch.Tensor) or seq_offsets.dtype not in _INDEX:
            raise ValueError("seq_offsets must be an int32 or int64 tensor")
        n = seq_offsets.numel()
        if (seq_offsets.dim() != 1 or n < 3 or n % 2 == 0 or seq_offsets.device != c.device
                or not seq_offsets.is_contiguous()):
            raise ValueError("seq_offsets must be contiguous [2 pairs + 1] on the logits' device")
        if len(c.shape) != 1:
            raise ValueError("with seq_offsets the logits must be [tokens, vocab]")
        pairs, at, odt = (n - 1) // 2, seq_offsets.data_ptr(), _INDEX[seq_offsets.dtype]
    args = B.loss_preference_args(c.optional("ref_logp", ref_logp), pairs, at, odt, code, 1 if average else 0,
                                  beta, label_smoothing, margin)
    with c:
        out, g = c.grad(grad, need_grad, grad_scale)
        loss, pair, rewards, logp = c.empty(), c.empty(pairs), c.empty(2 * pairs), c.empty(*c.shape)
        ws, n = c.workspace(pairs)
        B.loss_preference(c.x, y, args, g, loss.data_ptr(), pair.data_ptr(), rewards.data_ptr(),
                          logp.data_ptr() or None, ws.data_ptr(), n, c.stream)
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
    c = _Call(logits, temperature, stream)
    for name, t, types in (("teacher_ids", teacher_ids, _INDEX), ("teacher_logits", teacher_logits, _DTYPES)):
        if not isinstance(t, torch.Tensor) or t.dtype not in types:
            raise ValueError(f"{name} must be a tensor of {' or '.join(str(d)[6:] for d in types)}")
        if t.device != c.device or t.dim() != len(c.shape) + 1 or t.shape[:-1] != c.shape:
            raise ValueError(f"{name} must have shape {[*c.shape, 'k']} on the logits' device")
        if t.stride(-1) != 1 and t.shape[-1] != 1:
            raise ValueError(f"{name}: the innermost stride must be 1")
    k = teacher_ids.shape[-1]
    if teacher_logits.shape[-1] != k:
        raise ValueError("teacher_ids and teacher_logits must have the same shape")
    if mask is not None and isinstance(mask, torch.Tensor) and mask.dtype == torch.bool:
        mask = mask.view(torch.uint8)
    elif mask is not None:
        raise ValueError("mask must be a bool tensor")
    args = B.loss_distill_args(teacher_ids.data_ptr() or None, _INDEX[teacher_ids.dtype], *c._strides(teacher_ids),
                               teacher_logits.data_ptr() or None, _DTYPES[teacher_logits.dtype],
                               *c._strides(teacher_logits), k, c.optional("teacher_lse", teacher_lse),
                               c.optional("mask", mask, torch.uint8), c.optional("weights", weights))
    with c:
        out, g = c.grad(grad, need_grad, grad_scale)
        loss, token = c.empty(), c.empty(*c.shape)
        ws, n = c.workspace()
        B.loss_distill(c.x, args, g, loss.data_ptr(), token.data_ptr() or None, ws.data_ptr(), n, c.stream)
    return DistillLoss(loss, out, token)


__all__ = ["TokenLogprobs", "PolicyLoss", "PreferenceLoss", "DistillLoss", "token_logprobs",
           "token_logprobs_backward", "policy_loss", "preference_loss", "distill_loss"]
