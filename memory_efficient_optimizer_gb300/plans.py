"""What the optimizer classes keep from step to step: one marshalled plan for
each list of tensors that they step together."""
from __future__ import annotations

from operator import is_


def check_grad(k: int, p, g, dtypes) -> None:
    """What a step takes as the gradient of parameter k."""
    if g.device != p.device:
        raise ValueError(f"tensor {k}: params and grads must be CUDA tensors on one device")
    if g.dtype not in dtypes:
        raise ValueError(f"tensor {k}: grad dtype must be float32 or bfloat16")
    if g.shape != p.shape:
        raise ValueError(f"tensor {k}: grad shape {tuple(g.shape)} != param shape {tuple(p.shape)}")
    if not g.is_contiguous():
        raise ValueError(f"tensor {k}: params and grads must be contiguous")


def _same(state: dict, tensors: list) -> bool:
    """Whether a state has these tensors, and "step" behind them."""
    return len(state) == len(tensors) + 1 and all(map(is_, state.values(), tensors))


def plan_for(plans: dict, slot, ps: list, states: list, hp: dict, make):
    """The plan of a slot for parameters, with the gradients that they have now
    and their states (dicts with a "step" beside the tensors).  It is made anew
    where the parameters, states or hyperparameters are others than the last
    time.  Gradients come and go, on other memory or in another form: they are
    looked at in every step, put in where they are others, and taken out by the
    caller after it (``plan.grads = []``), so that a plan keeps none of them alive."""
    grads = [p.grad for p in ps]
    at = [g.data_ptr() for g in grads]
    seen = ([(p.data_ptr(), p.shape, p.is_contiguous(), g.shape, g.is_contiguous(), g.dtype) for p, g in zip(ps, grads)],
            repr(sorted(hp.items())))
    kept = plans.get(slot)
    if kept is not None and kept[0] == seen and all(map(_same, states, kept[3])):
        plan, before = kept[1:3]
        if at != before:
            # (how a gradient is read may go by its alignment)
            if any((x ^ y) % 16 for x, y in zip(at, before)):
                kept = None
            else:
                plan.take_grads(grads)
                plans[slot] = (seen, plan, at, kept[3])
    else:
        kept = None
    if kept is None:
        plans.pop(slot, None)
        for st in states:
            st["step"] = st.pop("step")               # (last: see _same)
        tensors = [{k: v for k, v in st.items() if k != "step"} for st in states]
        plan = make(ps, grads, tensors, **hp)
        plans[slot] = (seen, plan, at, [list(t.values()) for t in tensors])
    return plan
