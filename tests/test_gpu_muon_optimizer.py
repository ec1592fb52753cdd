"""What the Muon optimizer keeps and checks from step to step: the descriptors
that the library is given are looked at on their way."""
import gc
import weakref

import pytest
import torch

import memory_efficient_optimizer_gb300 as meo
from memory_efficient_optimizer_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture
def calls(monkeypatch):
    """(p, g, dtype, momentum) of every tensor of a call, and the learning rate."""
    seen, real = [], B.muon_step

    def step(tensors, n, hp, *rest):
        seen.append(([(t.p, t.g, t.grad_dtype, t.momentum) for t in tensors[:n]], hp.lr))
        real(tensors, n, hp, *rest)

    monkeypatch.setattr(B, "muon_step", step)
    return seen


def parameters(*shapes):
    return [torch.nn.Parameter(torch.ones(s, device="cuda")) for s in shapes]


def step(opt, params):
    """A step with new gradients; what the call has to be given, and references to the gradients."""
    grads = [torch.ones_like(p) for p in params]
    for p, g in zip(params, grads):
        p.grad = g
    opt.step()
    want = [(p.data_ptr(), g.data_ptr(), B.ADAF_FLOAT32, opt.state[p]["momentum"].data_ptr()) for p, g in zip(params, grads)]
    opt.zero_grad()
    return want, [weakref.ref(g) for g in grads]


def test_old_gradients_are_not_kept(calls):
    params = parameters((4, 6), (8, 3))
    opt = meo.Muon([{"params": params[:1]}, {"params": params[1:], "lr": 0.2}], lr=0.1)
    gone = []
    for t in range(20):
        want, refs = step(opt, params)
        gone += refs
        gc.collect()
        assert calls[-2:] == [(want[:1], 0.1), (want[1:], 0.2)]
        assert not [r for r in gone if r() is not None], f"step {t}"
    assert len({plan.workspace.data_ptr() for plan in opt._plans.values()}) == 1


def test_a_schedule_makes_no_new_plans(calls):
    params = parameters((4, 6))
    opt = meo.Muon(params, lr=0.1, coefficients=[(1.875, -1.25, 0.375)] * 5)
    plans = set()
    for t in range(20):
        opt.param_groups[0]["lr"] = 0.1 / (t + 1)
        want, _ = step(opt, params)
        assert calls[-1] == (want, 0.1 / (t + 1))
        plans |= {id(plan) for plan in opt._plans.values()}
    assert len(opt._plans) == len(plans) == 1
    opt.param_groups[0]["coefficients"][0] = (5.0, 0.0, 0.0)      # (the same list)
    with pytest.raises(ValueError, match="coefficients"):
        step(opt, params)
    opt.param_groups[0]["coefficients"][0] = (1.875, -1.25, 0.375)
    opt.param_groups[0]["lr"] = -1.0
    with pytest.raises(ValueError, match="learning rate"):
        step(opt, params)
    assert len(calls) == 20


def test_gradients_are_checked_at_every_step(calls):
    """On the same memory, but in another order."""
    p, = parameters((6, 6))
    opt = meo.Muon([p], lr=0.1)
    g = torch.ones(6, 6, device="cuda")
    p.grad = g
    opt.step()
    p.grad = g.t()
    with pytest.raises(ValueError, match="contiguous"):
        opt.step()
    p.grad = g
    opt.step()
    assert len(calls) == 2


def test_new_memory_of_a_parameter_or_its_momentum(calls):
    p, = parameters((4, 6))
    opt = meo.Muon([p], lr=0.1)
    for shape in ((4, 6), (4, 6), (300, 200), (20, 10)):
        p.data = torch.zeros(shape, device="cuda")
        opt.state[p]["momentum"] = torch.zeros(shape, device="cuda")
        want, _ = step(opt, [p])
        assert calls[-1][0] == want and p.isfinite().all() and not p.eq(0).any()
        plan, = opt._plans.values()
        assert plan.workspace.numel() >= B.muon_orthogonalize_workspace_size(1, *shape)
    opt.state[p]["momentum"] = torch.zeros(20, 11, device="cuda")
    with pytest.raises(ValueError, match="momentum"):
        step(opt, [p])


def test_parameters_without_a_gradient_are_left_out(calls):
    params = parameters((4, 6), (3, 5), (2, 7))
    opt = meo.Muon(params, lr=0.1)
    for some in (params, params[1:], params[:1], params):
        before = [p.detach().clone() for p in params]
        want, _ = step(opt, some)
        assert calls[-1][0] == want
        for p, b in zip(params, before):
            assert torch.equal(p, b) == all(p is not q for q in some)


def test_a_first_step_is_not_captured():
    """Its momentum would be zeroed by every replay.  Captured after a step, replays go on where it was."""
    def grad(t):
        return torch.randn(12, 20, generator=torch.Generator().manual_seed(t)).cuda()

    p, twin = parameters((12, 20), (12, 20))
    opt, other = meo.Muon([p], lr=0.1), meo.Muon([twin], lr=0.1)
    p.grad, twin.grad = grad(0), grad(0)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="momentum"):
        with torch.cuda.graph(graph):
            opt.step()
    assert p.eq(1).all() and not opt.state[p]
    opt.step()
    other.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    for t in range(1, 4):
        p.grad.copy_(grad(t))
        twin.grad.copy_(grad(t))
        graph.replay()
        other.step()
        assert torch.equal(p, twin) and torch.equal(opt.state[p]["momentum"], other.state[twin]["momentum"])


def test_a_workspace_outlives_the_work_on_another_stream():
    """A step on a stream that is not the one its plan was made on: the plan may go before the work has begun, but not
    its memory."""
    p = torch.randn(200, 300, generator=torch.Generator().manual_seed(1)).cuda()
    g = torch.randn(200, 300, generator=torch.Generator().manual_seed(2)).cuda()
    want = p.clone()
    meo.muon_step([want], [g], meo.init_muon_state([p]), lr=0.1)
    state, other = meo.init_muon_state([p]), torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    plan = meo.MuonStep([p], [g], state, lr=0.1)
    size, at = plan.workspace.numel(), plan.workspace.data_ptr()
    with torch.cuda.stream(other):
        torch.cuda._sleep(200_000_000)
    plan(other)
    del plan
    taken = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert at not in [t.data_ptr() for t in taken]
    torch.cuda.synchronize()
    assert torch.equal(p, want)
