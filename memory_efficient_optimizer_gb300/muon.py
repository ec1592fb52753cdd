"""PyTorch front end of the CUDA Muon step and its orthogonalisation
(include/muon.h).

As for the other steps, PyTorch only provides device memory and streams: these
functions check and marshal arguments, allocate zeroed state and the workspace,
and make one call into the C library per step.

Muon is a step for weight matrices; embeddings, output layers, vectors and
scalars go to another of this package's steps (Adafactor, LAMB, CAME).  A
tensor with more than two dimensions is a stack of matrices, one for each
leading index, as it is for the factored steps: the experts of a layer.
"""
from __future__ import annotations

import functools
from operator import is_
from typing import Iterable, Optional, Sequence

import torch

from . import binding as B
from .losses import _written

_DTYPES = {torch.float32: B.ADAF_FLOAT32, torch.bfloat16: B.ADAF_BFLOAT16}

#: a, b, c of the default Newton-Schulz step.
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def make_iteration(steps: int = 5, coefficients=COEFFICIENTS, eps: float = 1e-7) -> B.muon_iteration:
    """Validated muon_iteration: `steps` times one triple (a, b, c), or a triple for each of the steps."""
    try:
        rows = [tuple(float(v) for v in c) for c in coefficients] if hasattr(coefficients[0], "__len__") else (
            [tuple(float(v) for v in coefficients)] * int(steps))
    except (TypeError, IndexError, ValueError):
        raise ValueError("coefficients must be (a, b, c), or such a triple for each step") from None
    if any(len(r) != 3 for r in rows):
        raise ValueError("coefficients must be (a, b, c), or such a triple for each step")
    if len(rows) != int(steps) or not 1 <= len(rows) <= B.MUON_MAX_STEPS:
        raise ValueError(f"steps must be 1 to {B.MUON_MAX_STEPS}, with as many coefficients")
    it = B.muon_iteration()
    it.steps = len(rows)
    for k, r in enumerate(rows):
        it.coef[k][0], it.coef[k][1], it.coef[k][2] = r
    it.eps = float(eps)
    B.muon_validate_iteration(it)
    return it


def make_muon_hparams(lr=1e-3, momentum=0.95, nesterov=True, weight_decay=0.0, adjust_lr="original", steps=5,
                      coefficients=COEFFICIENTS, eps=1e-7) -> B.muon_hparams:
    """Validated muon_hparams (the library's checks; a bad value raises ValueError)."""
    code = B.MUON_ADJUST.get(adjust_lr)
    if code is None:
        raise ValueError(f"unknown adjust_lr {adjust_lr!r}: one of {sorted(B.MUON_ADJUST)}")
    hp = B.muon_hparams(float(lr), float(momentum), float(weight_decay), 1 if nesterov else 0, code,
                        make_iteration(steps, coefficients, eps))
    B.muon_validate(hp)
    return hp


def init_muon_state(params: Sequence[torch.Tensor]) -> list:
    """Zeroed fp32 momentum for each parameter."""
    return [{"momentum": torch.zeros_like(p, dtype=torch.float32, memory_format=torch.contiguous_format)}
            for p in params]


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _matrices(shape):
    """(batch, rows, cols) of a tensor as a stack of matrices."""
    batch = 1
    for n in shape[:-2]:
        batch *= n
    return batch, shape[-2], shape[-1]


class MuonStep:
    """A marshalled multi-tensor Muon step: the descriptor array and the
    workspace are built once; every call is one C-library call.  Parameters
    have two dimensions or more (leading ones: a stack).  ``workspace``: uint8
    memory to use in place of an own one, if it is large enough; steps that
    share it must not run at the same time."""

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], states: Sequence[dict], lr=1e-3,
                 momentum=0.95, nesterov=True, weight_decay=0.0, adjust_lr="original", steps=5,
                 coefficients=COEFFICIENTS, eps=1e-7, workspace: Optional[torch.Tensor] = None):
        self._hp = make_muon_hparams(lr, momentum, nesterov, weight_decay, adjust_lr, steps, coefficients, eps)
        self._shapes = None
        self._take(params, grads, states)
        if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()
                                      or workspace.device != self.device or workspace.numel() < self.workspace_bytes):
            workspace = None
        if workspace is None and self.n:
            workspace = torch.empty(max(self.workspace_bytes, 256), dtype=torch.uint8, device=self.device)
        self.workspace = workspace

    def _take(self, params, grads, states) -> None:
        """Checks the tensors and puts them into the descriptor array."""
        params, grads, states = list(params), list(grads), list(states)
        if len(params) != len(grads) or len(params) != len(states):
            raise ValueError("params, grads and states must have the same length")
        n = len(params)
        device = params[0].device if n else None
        tensors = (B.muon_tensor * max(1, n))()
        for k, (p, g, st) in enumerate(zip(params, grads, states)):
            if not isinstance(p, torch.Tensor) or p.dtype != torch.float32:
                raise ValueError(f"tensor {k}: params must be float32 tensors")
            if p.dim() < 2:
                raise ValueError(f"tensor {k}: Muon steps matrices (two dimensions or more); give this one to another step")
            if p.device.type != "cuda" or g.device != p.device or p.device != device:
                raise ValueError(f"tensor {k}: params and grads must be CUDA tensors on one device")
            if g.dtype not in _DTYPES:
                raise ValueError(f"tensor {k}: grad dtype must be float32 or bfloat16")
            if g.shape != p.shape:
                raise ValueError(f"tensor {k}: grad shape {tuple(g.shape)} != param shape {tuple(p.shape)}")
            if not p.is_contiguous() or not g.is_contiguous():
                raise ValueError(f"tensor {k}: params and grads must be contiguous")
            m = st.get("momentum")
            if not (isinstance(m, torch.Tensor) and m.dtype == torch.float32 and m.device == p.device
                    and m.is_contiguous() and m.numel() == p.numel()):
                raise ValueError(f"tensor {k}: state 'momentum' must be contiguous float32 with {p.numel()} elements on "
                                 "the param's device")
            tensors[k] = B.muon_tensor(_ptr(p), _ptr(g), _DTYPES[g.dtype], *_matrices(p.shape), _ptr(m))
        self.params, self.grads, self.states = params, grads, states
        self.n, self.device, self._tensors = n, device, tensors
        shapes = [p.shape for p in params]
        if shapes != self._shapes:
            self.workspace_bytes = B.muon_workspace_size(tensors, n) if n else 0
            self._shapes = shapes

    def __call__(self, stream: Optional[torch.cuda.Stream] = None) -> None:
        if self.n == 0:
            return
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        elif stream.device != self.device:
            raise ValueError(f"stream is of {stream.device}, the parameters are on {self.device}")
        with torch.cuda.device(self.device):
            B.muon_step(self._tensors, self.n, self._hp, _ptr(self.workspace), self.workspace_bytes,
                        int(stream.cuda_stream))
            self.workspace.record_stream(stream)   # (its memory is not given away while this stream works on it)

    def device_status(self, stream: Optional[torch.cuda.Stream] = None) -> int:
        """0, or 1 if a bounded wait inside a kernel of the last call ran out (synchronises the stream)."""
        if self.n == 0 or self.workspace_bytes == 0:
            return 0
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        return B.muon_device_status(_ptr(self.workspace), int(stream.cuda_stream))


def muon_step(params, grads, states, lr=1e-3, momentum=0.95, nesterov=True, weight_decay=0.0, adjust_lr="original",
              steps=5, coefficients=COEFFICIENTS, eps=1e-7, stream=None) -> None:
    """One Muon step over a list of matrices (functional form); states come
    from init_muon_state().  Use MuonStep to marshal once."""
    with (torch.cuda.stream(stream) if stream is not None else _Nothing()):
        MuonStep(params, grads, states, lr=lr, momentum=momentum, nesterov=nesterov, weight_decay=weight_decay,
                 adjust_lr=adjust_lr, steps=steps, coefficients=coefficients, eps=eps)(stream)


class _Nothing:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


def orthogonalize(x: torch.Tensor, *, steps: int = 5, coefficients=COEFFICIENTS, eps: float = 1e-7,
                  dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The matrix with x's singular vectors and singular values near 1, by
    Newton-Schulz steps (include/muon.h).

    ``x`` [..., rows, cols], float32 or bfloat16, with innermost stride 1 (rows
    may have gaps; leading dimensions are a stack).  The result is bfloat16, or
    ``dtype`` float32; either way it is good to about 1e-3 of its norm (the header
    has the bounds).  ``out``: a contiguous tensor for it, of x's shape; it may
    be x itself.
    """
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPES:
        raise ValueError("x must be a float32 or bfloat16 tensor")
    if x.dim() < 2:
        raise ValueError("x must have two dimensions or more")
    if out is not None:
        dtype = out.dtype if isinstance(out, torch.Tensor) else None
    if dtype not in _DTYPES:
        raise ValueError("the result must be float32 or bfloat16")
    if not x.is_cuda:
        raise ValueError("x must be on a CUDA device")
    if stream is not None and stream.device != x.device:
        raise ValueError(f"stream is of {stream.device}, x is on {x.device}")
    if x.shape[-1] > 1 and x.stride(-1) != 1:
        raise ValueError("x: the innermost stride must be 1")
    it = _iteration(steps, coefficients, eps)
    batch, rows, cols = _matrices(x.shape)
    if x.dim() > 3:
        try:
            flat = x.view(batch, rows, cols)
        except RuntimeError:
            raise ValueError("x: the leading dimensions must lie one after another") from None
    else:
        flat = x
    stride_b = flat.stride(0) if flat.dim() == 3 and batch > 1 else 0
    given = out
    with torch.cuda.device(x.device) if stream is None else torch.cuda.stream(stream):
        if out is None:
            out = torch.empty(x.shape, dtype=dtype, device=x.device)
        elif out.shape != x.shape or out.device != x.device or not out.is_contiguous():
            raise ValueError("out must be contiguous, with x's shape and device")
        n = _workspace_bytes(batch, rows, cols)
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device=x.device)
        B.muon_orthogonalize(B.muon_matrices(_ptr(x), _DTYPES[x.dtype], batch, rows, cols, stride_b, flat.stride(-2)), it,
                             _ptr(out), _DTYPES[dtype], _ptr(ws), n, int(torch.cuda.current_stream(x.device).cuda_stream))
    _written(given)
    return out


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(batch, rows, cols):
    return B.muon_orthogonalize_workspace_size(batch, rows, cols)


_iterations: dict = {}


def _iteration(steps, coefficients, eps):
    """make_iteration, kept for the arguments that were checked before."""
    try:
        key = (steps, tuple(coefficients), eps)
        it = _iterations.get(key)
    except TypeError:
        return make_iteration(steps, coefficients, eps)
    if it is None:
        it = make_iteration(steps, coefficients, eps)
        if len(_iterations) >= 64:
            _iterations.clear()
        _iterations[key] = it
    return it


class Muon(torch.optim.Optimizer):
    """torch.optim.Optimizer wrapper; each parameter group is one call into
    the library.  Parameters have two dimensions or more."""

    def __init__(self, params: Iterable, lr=1e-3, momentum=0.95, nesterov=True, weight_decay=0.0,
                 adjust_lr="original", steps=5, coefficients=COEFFICIENTS, eps=1e-7):
        make_muon_hparams(lr, momentum, nesterov, weight_decay, adjust_lr, steps, coefficients, eps)
        super().__init__(params, dict(lr=lr, momentum=momentum, nesterov=nesterov, weight_decay=weight_decay,
                                      adjust_lr=adjust_lr, steps=steps, coefficients=coefficients, eps=eps))
        for group in self.param_groups:
            for p in group["params"]:
                if p.dim() < 2:
                    raise ValueError("Muon steps matrices (two dimensions or more): give the others to another optimizer")
        self._plans = {}
        self._workspaces = {}       # by device: gigabytes for large layers, so one for all plans

    def __setstate__(self, state):
        super().__setstate__(state)
        self._plans = {}            # (not part of what is copied, pickled or loaded)
        self._workspaces = {}

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for gi, group in enumerate(self.param_groups):
            hp = {k: group[k] for k in ("lr", "momentum", "nesterov", "weight_decay", "adjust_lr", "steps", "coefficients",
                                        "eps")}
            ps = [p for p in group["params"] if p.grad is not None]
            if not ps:
                continue
            capturing = False
            if ps[0].is_cuda:
                with torch.cuda.device(ps[0].device):
                    capturing = torch.cuda.is_current_stream_capturing()
            for p in ps:
                if not self.state[p]:
                    if capturing:
                        # its zeros would be part of the graph: every replay would forget the momentum
                        raise RuntimeError("a first step cannot be captured: the momentum has to be there before (call "
                                           "step() once, or load a state)")
                    self.state[p].update(init_muon_state([p])[0])
            grads = [p.grad for p in ps]
            states = [self.state[p] for p in ps]
            if capturing:
                # memory of a graph's own pool is not kept for calls outside it
                MuonStep(ps, grads, states, **hp)()
                continue
            # A group's plan stays; the tensors are looked at in every step and put into it where they are others
            # (gradients come and go, on other memory or in another form), and it does not keep them.
            plan, values = self._plans.get(gi), repr(sorted(hp.items()))
            momenta = [st.get("momentum") for st in states]
            seen = [(p.data_ptr(), p.shape, p.is_contiguous(), g.data_ptr(), g.shape, g.is_contiguous(), g.dtype)
                    for p, g in zip(ps, grads)]
            if plan is None:
                plan = MuonStep(ps, grads, states, workspace=self._workspaces.get(ps[0].device), **hp)
                self._plans[gi] = plan
            else:
                if seen != plan.seen or not all(map(is_, momenta, plan.momenta)):
                    plan.seen = None
                    plan._take(ps, grads, states)
                if values != plan.values:
                    plan.values = None
                    plan._hp = make_muon_hparams(**hp)
            plan.seen, plan.momenta, plan.values = seen, momenta, values
            self._share_workspace(plan)
            try:
                plan()
            finally:
                plan.params, plan.grads, plan.states = [], [], []
        return loss

    def _share_workspace(self, plan) -> None:
        """One workspace for all plans of a device, as large as the largest of them needs."""
        kept = self._workspaces.get(plan.device)
        if kept is None or kept.numel() < plan.workspace_bytes:
            kept = plan.workspace
            if kept is None or kept.numel() < plan.workspace_bytes:
                kept = torch.empty(max(plan.workspace_bytes, 256), dtype=torch.uint8, device=plan.device)
            self._workspaces[plan.device] = kept
        for other in self._plans.values():
            if other.device == plan.device:
                other.workspace = kept


__all__ = ["Muon", "MuonStep", "muon_step", "init_muon_state", "make_muon_hparams", "orthogonalize"]
