"""What the optimizer classes keep from step to step: one marshalled plan for
each list of tensors that they step together."""
from __future__ import annotations


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


def plan_for(plans: dict, slot, ps: list, grads: list, states: list, hp: dict, make):
    """The plan of a slot, made anew where its parameters, states or
    hyperparameters are others than the last time.  Gradients come and go, on
    other memory or in another form: they are checked and put in at every step,
    and taken out by the caller after it (``plan.grads = []``), so that a plan
    keeps none of them alive."""
    key = ([(p.data_ptr(), p.shape, p.dtype, p.is_contiguous()) for p in ps],
           [{k: v.data_ptr() for k, v in st.items()} for st in states],
           [(g.dtype, g.data_ptr() % 16) for g in grads],      # (how a gradient is read may go by its alignment)
           repr(sorted(hp.items())))
    kept = plans.get(slot)
    if kept is not None and kept[0] == key:
        kept[1].take_grads(grads)
        return kept[1]
    plans.pop(slot, None)
    plan = make(ps, grads, states, **hp)
    plans[slot] = (key, plan)
    return plan
