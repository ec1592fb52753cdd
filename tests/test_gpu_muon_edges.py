"""The orthogonalisation and the Muon step at the ends of their ranges."""
import numpy as np
import pytest
import torch

import memory_efficient_optimizer_gb300 as meo
from oracle import muon as O

pytestmark = pytest.mark.gpu

# As in the other tests of these operators: four roundings to fp16 a step, 2^-12 each, and those of the last
# three steps, which grow by 2 a step: 4 (1 + 2 + 4) / 2 2^-12 = 3.4e-3.
TOL = 4e-3
FLT_MIN = 2.0 ** -126


def normal(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def far(got, want):
    got = got.double().cpu().numpy()
    return np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("eps", [FLT_MIN, 1e-36, 1e-30, 1e-20, 1e-15, 1e-7])
def test_zeros_stay_zero_at_every_eps(eps):
    for shape in ((50, 70), (2, 33, 7), (1, 1)):
        assert meo.orthogonalize(torch.zeros(shape, device="cuda"), eps=eps, dtype=torch.float32).eq(0).all()
    p = normal((40, 60), 1).cuda()
    before = p.clone()
    meo.muon_step([p], [torch.zeros_like(p)], meo.init_muon_state([p]), lr=0.1, eps=eps)
    assert torch.equal(p, before)


@pytest.mark.parametrize("scale", [1e-7, 1e-8, 3e-19, 1e-22, 1e-30, 1e-36])
@pytest.mark.parametrize("shape", [(60, 90), (90, 61)])
def test_small_matrices_are_scaled_by_their_norm(shape, scale):
    """Their squares are not normal fp32 numbers, or none at all."""
    x = (normal(shape, 2) * scale).cuda()
    wide = torch.zeros(shape[0], shape[1] + 3, device="cuda")
    wide[:, :shape[1]] = x
    for eps in (FLT_MIN, scale * 1e-2) if scale > 1e-36 else (FLT_MIN,):
        want = O.orthogonalize(x.double().cpu().numpy(), eps=eps)
        for t in (x, wide[:, :shape[1]]):
            assert far(meo.orthogonalize(t, eps=eps, dtype=torch.float32), want) < TOL


@pytest.mark.parametrize("eps", [1e-20, 1e-10, 1e-7, 9e-7, 1e-6, 1e-3, 1e10])
def test_an_eps_above_the_norm(eps):
    """The matrix is divided by eps, with a norm on both sides of where the squares are taken another way."""
    for norm in (eps * 0.9, eps * 1e-3, 0.99 * 2.0 ** -20, 1.01 * 2.0 ** -20):
        x = normal((64, 80), 3)
        x = (x * (norm / x.double().norm())).cuda()
        want = O.orthogonalize(x.double().cpu().numpy(), eps=eps)
        assert far(meo.orthogonalize(x, eps=eps, dtype=torch.float32), want) < TOL


def test_autograd_learns_of_a_result_over_a_tensor():
    """A matrix that a backward pass needs, and that holds the orthogonalisation by then, is an error."""
    w, a = (torch.nn.Parameter(normal(s, 4).cuda()) for s in ((40, 60), (60, 30)))     # (each other's gradients need both)
    for out in (a.detach(), w.detach()):
        y = (w @ a).square().sum()
        meo.orthogonalize(out, out=out)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    version = a._version
    meo.orthogonalize(a)
    assert a._version == version


@pytest.mark.parametrize("shapes", [[(1, 300, 300)], [(1, 40, 64)], [(2, 1500, 1500)], [(1, 64, 9000)], [(7, 1024, 2048)], [(1, 4096, 4400)],
                                    [(7, 1024, 2048), (2, 1100, 1200), (50, 30, 20)], [(1, 2048, 4096), (1, 2049, 4100)]])
def test_the_workspace_is_not_left(shapes):
    """A step within the bytes that it asked for, on memory of any contents, against the oracle's formula."""
    params = [normal(s, k).cuda() for k, s in enumerate(shapes)]
    grads = [normal(s, 10 + k).cuda() for k, s in enumerate(shapes)]
    before = [p.clone() for p in params]
    states = meo.init_muon_state(params)
    need = meo.MuonStep(params, grads, states).workspace_bytes
    ws = torch.full((need + (1 << 20),), 255, dtype=torch.uint8, device="cuda")
    step = meo.MuonStep(params, grads, states, lr=1.0, momentum=0.0, adjust_lr="match_rms", workspace=ws)
    assert step.workspace is ws
    step()
    assert step.device_status() == 0 and ws[need:].eq(255).all()
    for p, b, g in zip(params, before, grads):
        x = g.double() / g.double().flatten(-2).norm(dim=-1)[..., None, None]
        x = x if x.shape[-2] <= x.shape[-1] else x.mT
        for c0, c1, c2 in O.COEFFICIENTS:
            a = x @ x.mT
            x = c0 * x + (c1 * a + c2 * (a @ a)) @ x
        want = (x if g.shape[-2] <= g.shape[-1] else x.mT) * 0.2 * max(g.shape[-2:]) ** 0.5
        # p's own rounding, 2^-24 of a normal value, beside an update of 0.2
        assert far(b - p, want.cpu().numpy()) < TOL + 2.0 ** -20
