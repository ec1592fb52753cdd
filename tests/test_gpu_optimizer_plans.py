"""What the optimizer classes keep and check from step to step."""
import gc
import weakref

import pytest
import torch

import memory_efficient_optimizer_gb300 as meo
from memory_efficient_optimizer_gb300 import binding as B

pytestmark = pytest.mark.gpu

KINDS = {
    "lamb": (lambda ps, **kw: meo.Lamb(ps, **kw), "lamb_step", lambda t: (t.p, t.g)),
    "came": (lambda ps, **kw: meo.Came(ps, **{"lr": 1e-3, **kw}), "came_step", lambda t: (t.p, t.g)),
    "adafactor": (lambda ps, **kw: meo.Adafactor(ps, **kw), "adafactor_step", lambda t: (t.param, t.grad)),
}


@pytest.fixture(params=sorted(KINDS))
def kind(request, monkeypatch):
    """(make an optimizer, what the library was called with)."""
    make, name, pointers = KINDS[request.param]
    seen, real = [], getattr(B, name)

    def call(tensors, *rest):
        n = next(r for r in rest if isinstance(r, int))
        seen.append([pointers(t) for t in tensors[:n]])
        real(tensors, *rest)

    monkeypatch.setattr(B, name, call)
    return make, seen


def parameters(*shapes):
    return [torch.nn.Parameter(torch.ones(s, device="cuda")) for s in shapes]


def value(t, k, shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(100 * t + k)).cuda()


def test_old_gradients_are_not_kept(kind):
    make, seen = kind
    params = parameters((40, 60), (7,), (3, 5, 4))
    opt, gone = make(params), []
    for t in range(20):
        grads = [value(t, k, p.shape) for k, p in enumerate(params)]
        for p, g in zip(params, grads):
            p.grad = g
        opt.step()
        assert seen[-1] == [(p.data_ptr(), g.data_ptr()) for p, g in zip(params, grads)]
        gone += [weakref.ref(g) for g in grads]
        del grads, g
        opt.zero_grad()
        gc.collect()
        assert not [r for r in gone if r() is not None], f"step {t}"


def test_new_gradients_step_as_kept_ones_do(kind):
    """Tensors that come anew at every step, on memory of any alignment, against one kept gradient with the same values."""
    make, _ = kind
    shapes = [(40, 64), (300,), (3, 8, 16)]
    a, b = parameters(*shapes), parameters(*shapes)
    opt, other = make(a), make(b)
    for p in b:
        p.grad = torch.zeros_like(p)
    for t in range(6):
        for k, (p, q) in enumerate(zip(a, b)):
            g = value(t, k, p.shape)
            room = torch.empty(g.numel() + 1, device="cuda")
            p.grad = room[t % 2:t % 2 + g.numel()].view(g.shape).copy_(g)
            q.grad.copy_(g)
        opt.step()
        other.step()
        opt.zero_grad()
        for p, q in zip(a, b):
            # (sums of squares in another order, or taken over from the step before: in double precision)
            assert (p - q).abs().max() <= 2.0 ** -22 * q.abs().max()


def test_gradients_are_checked_at_every_step(kind):
    """On the same memory, but in another order."""
    make, seen = kind
    p, = parameters((8, 8))
    opt = make([p])
    g = value(0, 0, (8, 8))
    p.grad = g
    opt.step()
    p.grad = g.t()
    with pytest.raises(ValueError, match="contiguous"):
        opt.step()
    assert len(seen) == 1


def test_a_loaded_state_is_stepped_with(kind):
    """With the gradients where they were."""
    make, _ = kind
    a, b = parameters((40, 64), (30,)), parameters((40, 64), (30,))
    opt, other = make(a), make(b)
    for k, (p, q) in enumerate(zip(a, b)):
        p.grad, q.grad = value(0, k, p.shape), value(0, k, p.shape)
    opt.step()
    other.step()
    saved = {"state": {k: {n: v.clone() if torch.is_tensor(v) else v for n, v in st.items()} for k, st in opt.state_dict()["state"].items()},
             "param_groups": opt.state_dict()["param_groups"]}
    before = [p.detach().clone() for p in a]
    for k, p in enumerate(a):
        p.grad.copy_(value(1, k, p.shape))
    opt.step()                                        # a step that is taken back
    opt.load_state_dict(saved)
    with torch.no_grad():
        for p, b0 in zip(a, before):
            p.copy_(b0)
    for k, (p, q) in enumerate(zip(a, b)):
        p.grad.copy_(value(2, k, p.shape))
        q.grad.copy_(value(2, k, p.shape))
    opt.step()
    other.step()
    for p, q in zip(a, b):
        assert (p - q).abs().max() <= 2.0 ** -22 * q.abs().max()
        for n, v in other.state[q].items():
            if torch.is_tensor(v):
                assert torch.allclose(opt.state[p][n].double(), v.double(), rtol=1e-6, atol=0)
            else:
                assert opt.state[p][n] == v
