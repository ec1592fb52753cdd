"""The bounds that include/muon.h gives for the orthogonalisation's error, on spectra of each kind."""
import pytest
import torch

import memory_efficient_optimizer_gb300 as meo
from oracle import muon as O

pytestmark = pytest.mark.gpu


def formula(x):
    """In 64 bits, on the GPU."""
    x = x.double() / x.double().flatten(-2).norm(dim=-1)[..., None, None]
    turn = x.shape[-2] > x.shape[-1]
    x = x.mT if turn else x
    for a, b, c in O.COEFFICIENTS:
        g = x @ x.mT
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.mT if turn else x


def far(x):
    want = formula(x)
    return ((meo.orthogonalize(x, dtype=torch.float32) - want).flatten(-2).norm(dim=-1) / want.flatten(-2).norm(dim=-1)).max().item()


def with_values(shape, s, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q1, q2 = (torch.linalg.qr(torch.randn(*shape[:-2], n, len(s), device="cuda", generator=g, dtype=torch.float64))[0] for n in shape[-2:])
    return ((q1 * s.cuda().double()) @ q2.mT).float()


def falling(shape, power, seed):
    if power == 0:
        return torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))
    return with_values(shape, torch.arange(1, min(shape[-2:]) + 1) ** -float(power), seed)


@pytest.mark.parametrize("power", [0, 0.5, 1.0, 2.0])
@pytest.mark.parametrize("shape", [(128, 128), (128, 700), (640, 200), (256, 512), (500, 500), (130, 9000), (1030, 1024), (2000, 1500),
                                   (7, 1024, 2048), (3, 1100, 2304)])
def test_usual_spectra(shape, power):
    assert max(far(falling(shape, power, seed)) for seed in range(3)) <= 1.5e-3


@pytest.mark.parametrize("shape", [(128, 128), (400, 128), (200, 200), (256, 512), (1024, 1024)])
def test_any_spectrum(shape):
    n = min(shape)
    k = torch.arange(1, n + 1).double()
    spectra = [k ** -4, k ** -8, 0.5 ** k, 0.97 ** k, torch.where(k <= n // 2, 1.0, 0.01), torch.where(k < 2, 1.0, 1e-3)]
    spectra += [torch.ones(r) for r in (1, 2, 3, 4, 7, 15, 20, 30, 45, 60, 90, n)]
    for s in spectra:
        assert max(far(with_values(shape, s, seed)) for seed in range(2)) <= 6e-3


@pytest.mark.parametrize("shape", [(1, 1), (1, 300), (2, 3), (3, 3), (4, 4), (5, 9), (8, 8), (100, 8), (12, 12), (15, 17), (16, 64), (24, 40),
                                   (32, 32), (64, 48), (64, 5000), (96, 96), (127, 300)])
def test_small_matrices(shape):
    for power in (0, 0.5, 1.0, 2.0):
        assert far(torch.stack([falling(shape, power, seed) for seed in range(20)])) <= 1.5e-2
