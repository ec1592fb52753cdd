"""The Muon step and its orthogonalisation on the GPU against the float64 oracle.

Tolerance of the result, 2-norm of the difference over 2-norm: a step of the
iteration rounds four factors to fp16 (x twice in x x^T, then F and E; at most
2^-12 relative each), a step's derivative lets errors of the steps before grow
by about 2 where singular values lie between 0.7 and 1.2, and those of the last
three steps count: 4 (1 + 2 + 4) / 2 2^-12 = 3.4e-3 if all of them lined up.
4e-3 is taken; a bf16 result is off by up to 2^-8 of itself more.
"""
import numpy as np
import pytest
import torch

import memory_efficient_optimizer_gb300 as meo
from memory_efficient_optimizer_gb300 import binding as B
from oracle import muon as O

pytestmark = pytest.mark.gpu
TOL = 4e-3


def decaying(shape, power, seed):
    """Singular values that fall as 1 / k^power."""
    g = torch.Generator().manual_seed(seed)
    r = min(shape[-2:])
    q1, _ = torch.linalg.qr(torch.randn(*shape[:-2], shape[-2], r, generator=g, dtype=torch.float64))
    q2, _ = torch.linalg.qr(torch.randn(*shape[:-2], shape[-1], r, generator=g, dtype=torch.float64))
    s = torch.arange(1, r + 1, dtype=torch.float64) ** -power
    return ((q1 * s) @ q2.mT).float()


def normal(shape, seed, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def far(got, want):
    got, want = got.double().cpu().numpy(), np.asarray(want)
    assert got.shape == want.shape
    return np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-300)


def reference(x, **kw):
    x = x.double().cpu().numpy()
    flat = x.reshape(-1, *x.shape[-2:])
    return np.stack([O.orthogonalize(m, **kw) for m in flat]).reshape(x.shape)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1, 1), (1, 300), (300, 1), (2, 3), (8, 8), (15, 17), (64, 64), (65, 200), (128, 128),
                                   (129, 127), (1, 130, 70), (5, 24, 40), (256, 512), (511, 300), (2, 3, 31, 66)])
def test_matches_the_oracle(shape, dtype):
    x = normal(shape, 1, dtype)
    want = reference(x)
    x = x.cuda()
    assert far(meo.orthogonalize(x, dtype=torch.float32), want) < TOL
    out = meo.orthogonalize(x)
    assert out.dtype == torch.bfloat16 and far(out, want) < TOL + 2 ** -8


@pytest.mark.parametrize("power", [0.5, 1.0, 2.0])
@pytest.mark.parametrize("shape", [(96, 96), (200, 640), (300, 100)])
def test_small_singular_values_are_kept(shape, power):
    """The directions of small singular values come out as exactly as the others: iterates that were
    rounded to 16 bits would be 1e-2 to 1e-1 off here."""
    x = decaying(shape, power, 3)
    want = reference(x)
    got = meo.orthogonalize(x.cuda(), dtype=torch.float32).double().cpu().numpy()
    assert np.linalg.norm(got - want) < TOL * np.linalg.norm(want)
    left, s, right = np.linalg.svd(x.double().numpy(), full_matrices=False)
    a, b = (np.einsum("ik,ij,kj->k", left, m, right) for m in (got, want))
    # along every singular direction: relative to what is there
    assert np.all(np.abs(a - b) < 4 * TOL * np.abs(b) + 1e-6)


def on_gpu(x, coefficients=O.COEFFICIENTS):
    """The formula in fp64 on the GPU, for matrices too large for the oracle."""
    want = x.double()
    want = want / want.flatten(-2).norm(dim=-1)[..., None, None]
    turn = x.shape[-2] > x.shape[-1]
    want = want.mT if turn else want
    for a, b, c in coefficients:
        g = want @ want.mT
        want = a * want + (b * g + c * (g @ g)) @ want
    return (want.mT if turn else want).cpu().numpy()


@pytest.mark.parametrize("shape", [(2000, 1500), (3, 1100, 2304), (4608, 520)])
def test_large_tiles(shape):
    """Many tiles a matrix and a CTA, in pairs of CTAs and apart."""
    x = normal(shape, 5).cuda()
    assert far(meo.orthogonalize(x, dtype=torch.float32), on_gpu(x)) < TOL


@pytest.mark.parametrize("shape", [(7, 1024, 2048), (7, 2101, 1030), (12, 1025, 2056)])
@pytest.mark.parametrize("spectrum", ["flat", "falling"])
def test_two_steps_at_once(shape, spectrum):
    """Wide matrices, enough of them: the first two steps come from one x x^T."""
    x = normal(shape, 6).cuda()
    if spectrum == "falling":
        r = min(shape[-2:])
        s = torch.arange(1, r + 1, device="cuda") ** -1.0
        x = (normal((shape[0], shape[1], r), 7).cuda() * s) @ normal((shape[0], r, shape[2]), 8).cuda()
    assert far(meo.orthogonalize(x, dtype=torch.float32), on_gpu(x)) < TOL
    for co in ([O.COEFFICIENTS[0]] * 2, [O.COEFFICIENTS[0]] * 3, [(1.875, -1.25, 0.375)] * 4, [O.COEFFICIENTS[0]]):
        got = meo.orthogonalize(x[:7], steps=len(co), coefficients=co, dtype=torch.float32)
        assert far(got, on_gpu(x[:7], co)) < TOL


def test_a_list_of_wide_and_square_matrices():
    """Both kinds of group in one call."""
    shapes = [(7, 1024, 2048), (300, 300), (2, 2100, 1024), (64, 200), (1100, 1200)]
    params = [normal(s, k).cuda() for k, s in enumerate(shapes)]
    grads = [normal(s, 10 + k).cuda() for k, s in enumerate(shapes)]
    before = [p.clone() for p in params]
    step = meo.MuonStep(params, grads, meo.init_muon_state(params), lr=0.1, adjust_lr="match_rms", nesterov=False)
    step()
    assert step.device_status() == 0
    for p, b, g, s in zip(params, before, grads, shapes):
        moved = (b - p).double() / (0.1 * 0.2 * max(s[-2:]) ** 0.5)
        want = on_gpu(g)
        # an fp32 rounding of p is 2^-24 of it, the update's elements are 1 / sqrt(max side) or so
        assert far(moved, want) < TOL + 1e-3


@pytest.mark.parametrize("shape", [(1, 1279), (1, 1280), (1, 10301), (16, 2688), (6400, 63), (64, 20000), (65, 1281), (129, 2600),
                                   (2, 200, 7001), (13, 16, 3584), (300, 16001), (1024, 1920), (1025, 4100), (72, 40, 1300),
                                   (73, 40, 1300)])
def test_long_sums_in_parts(shape):
    """x x^T of few wide matrices is summed in parts, which are joined in their order: equal bits."""
    x = normal(shape, 4).cuda()
    out = meo.orthogonalize(x, dtype=torch.float32)
    assert far(out, on_gpu(x)) < TOL
    for _ in range(3):
        assert torch.equal(out, meo.orthogonalize(x, dtype=torch.float32))


def test_a_list_with_sums_in_parts_and_in_one():
    shapes = [(64, 9000), (40, 60), (3, 16, 1400), (700, 130), (2000, 100), (256, 256), (1, 5000)]
    params = [normal(s, k).cuda() for k, s in enumerate(shapes)]
    grads = [normal(s, 20 + k).cuda() for k, s in enumerate(shapes)]
    before = [p.clone() for p in params]
    meo.muon_step(params, grads, meo.init_muon_state(params), lr=1.0, momentum=0.0)
    for p, b, g in zip(params, before, grads):
        want = on_gpu(g) * max(1.0, g.shape[-2] / g.shape[-1]) ** 0.5
        # (the difference has p's own rounding too: 2^-24 of a normal value, and the update is 1 / sqrt(n) or more)
        assert far(b - p, want) < TOL + 2e-5
    many = [normal((64, 9000), k).cuda() for k in range(50)]   # two launches, with one workspace
    apart = [meo.orthogonalize(m, dtype=torch.float32) for m in many]
    zero = [torch.zeros_like(m) for m in many]
    meo.muon_step(zero, many, meo.init_muon_state(zero), lr=1.0, momentum=0.0)
    for z, o in zip(zero, apart):
        assert far(-z, o.double().cpu().numpy()) < 2 * TOL


def test_values_of_sums_in_parts():
    x = normal((3, 32, 4000), 1).cuda()
    want = on_gpu(x)
    x[1, 3, 3999] = float("nan")
    out = meo.orthogonalize(x, dtype=torch.float32)
    assert out[1].isnan().all() and far(out[::2], want[::2]) < TOL
    x[1] = 0
    out = meo.orthogonalize(x, dtype=torch.float32)
    assert out[1].eq(0).all() and far(out[::2], want[::2]) < TOL


def test_rows_with_gaps_and_views():
    base = normal((3, 70, 100), 7).cuda()
    for x in (base[:, :, :90], base[:, 3:40], base[1:], base[:, :1], base[:, ::2, 10:63]):
        assert far(meo.orthogonalize(x, dtype=torch.float32), reference(x)) < TOL
    with pytest.raises(ValueError, match="innermost"):
        meo.orthogonalize(base.mT)
    with pytest.raises(ValueError, match="leading"):
        meo.orthogonalize(normal((4, 4, 6, 6), 1).cuda().transpose(0, 1))
    odd = torch.empty(70 * 100 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(70, 100)
    odd.copy_(base[0])
    assert far(meo.orthogonalize(odd, dtype=torch.float32), reference(odd)) < TOL
    out = torch.empty(70 * 100 + 1, device="cuda")[1:].view(70, 100)
    assert meo.orthogonalize(base[0], out=out) is out and far(out, reference(base[0])) < TOL


def test_in_place_and_refusals():
    x = normal((40, 60), 8).cuda()
    want = reference(x)
    assert meo.orthogonalize(x, out=x) is x and far(x, want) < TOL
    with pytest.raises(ValueError, match="out"):
        meo.orthogonalize(x, out=torch.empty(60, 40, device="cuda"))
    with pytest.raises(ValueError, match="out"):
        meo.orthogonalize(x, out=torch.empty(60, 40, device="cuda").mT)
    with pytest.raises(ValueError, match="overlaps"):
        meo.orthogonalize(x[:30], out=x[10:])


def test_values():
    z = torch.zeros(50, 70, device="cuda")
    assert meo.orthogonalize(z).eq(0).all()
    one = z.clone()
    one[3, 5] = 1e-30                       # a norm below eps
    assert far(meo.orthogonalize(one, dtype=torch.float32) + 1, reference(one) + 1) < 1e-6
    for bad in (float("nan"), float("inf"), -float("inf"), 1e25):
        x = normal((2, 50, 70), 2).cuda()
        want = reference(x[:1])
        x[1, 7, 9] = bad
        out = meo.orthogonalize(x, dtype=torch.float32)
        assert out[1].isnan().all() and far(out[:1], want) < TOL
    for scale in (1e-4, 1e15):              # scale-free
        x = normal((50, 70), 2)
        assert far(meo.orthogonalize((x * scale).cuda(), dtype=torch.float32), reference(x)) < TOL
    assert meo.orthogonalize(torch.zeros(0, 4, device="cuda")).shape == (0, 4)
    assert meo.orthogonalize(torch.zeros(2, 4, 0, device="cuda")).shape == (2, 4, 0)


def test_other_iterations():
    x = normal((90, 120), 4)
    cubic = [(1.875, -1.25, 0.375)] * 8
    for co in (cubic, [(3.4445, -4.7750, 2.0315)] * 3 + cubic[:3], cubic[:1], [(1.5, -0.5, 0.0)] * 16):
        got = meo.orthogonalize(x.cuda(), steps=len(co), coefficients=co, dtype=torch.float32)
        assert far(got, reference(x, coefficients=co)) < TOL


def run_step(shapes, gdtype, hp, steps=3, seed=0):
    params = [normal(s, seed + k) * 0.1 for k, s in enumerate(shapes)]
    ref = [p.double().numpy() for p in params]
    mom = [np.zeros(s) for s in shapes]
    params = [p.cuda() for p in params]
    grads = [torch.empty(s, device="cuda", dtype=gdtype) for s in shapes]
    states = meo.init_muon_state(params)
    step = meo.MuonStep(params, grads, states, **hp)
    ohp = {("adjust" if k == "adjust_lr" else k): v for k, v in hp.items()}
    moved = [0.0] * len(shapes)
    for t in range(steps):
        for k, s in enumerate(shapes):
            g = normal(s, 100 * t + k + 17, gdtype) * 1e-3
            grads[k].copy_(g)
            g = grads[k].double().cpu().numpy()
            old, flat = ref[k], ref[k].reshape(-1, *s[-2:])
            new = [O.step(p, gg, m, **ohp) for p, gg, m in zip(flat, g.reshape(flat.shape), mom[k].reshape(flat.shape))]
            ref[k] = np.stack([n[0] for n in new]).reshape(s)
            mom[k] = np.stack([n[1] for n in new]).reshape(s)
            moved[k] += np.linalg.norm(ref[k] - old)
        step()
    torch.cuda.synchronize()
    assert step.device_status() == 0
    for k in range(len(shapes)):
        p, m = params[k].double().cpu().numpy(), states[k]["momentum"].double().cpu().numpy()
        # 3 roundings of fp32 a step and value, and the update's own tolerance
        assert np.linalg.norm(p - ref[k]) < TOL * moved[k] + 3 * steps * 2 ** -24 * np.linalg.norm(ref[k])
        assert np.all(np.abs(m - mom[k]) <= 3 * steps * 2 ** -24 * np.abs(mom[k]).max())


SHAPES = [(40, 64), (64, 40), (128, 128), (3, 20, 33), (40, 64), (1, 7), (256, 100), (7, 1), (2, 2, 64, 40), (130, 515)]


@pytest.mark.parametrize("gdtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hp", [dict(), dict(lr=0.02, nesterov=False, weight_decay=0.1),
                                dict(lr=0.01, adjust_lr="match_rms", momentum=0.5, weight_decay=0.01), dict(momentum=0.0)])
def test_step_matches_the_oracle(gdtype, hp):
    run_step(SHAPES, gdtype, hp)


def test_step_of_a_large_group():
    """More matrices of one shape than a launch takes."""
    run_step([(70, 16, 24), (24, 16)], torch.bfloat16, dict(lr=0.01), steps=2)


def test_unaligned_tensors():
    def odd(t):
        return torch.empty(t.numel() + 1, device="cuda", dtype=t.dtype)[1:].view(t.shape).copy_(t)
    p, g, m = normal((30, 44), 1), normal((30, 44), 2).bfloat16(), normal((30, 44), 3)
    want, wm = O.step(p.double().numpy(), g.double().numpy(), m.double().numpy(), lr=0.1)
    p, g, m = odd(p), odd(g), odd(m)
    meo.muon_step([p], [g], [{"momentum": m}], lr=0.1)
    assert far(p, want) < 1e-3 and far(m, wm) < 1e-6


def test_equal_bits_and_other_streams():
    x = normal((3, 300, 200), 9).cuda()
    a = meo.orthogonalize(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = meo.orthogonalize(x, stream=s)
    c = meo.orthogonalize(x * 1)            # at the same time
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)


def test_beside_other_work():
    """Several calls and other kernels at once: whichever SMs a call gets, and however few at first, its bits are the same."""
    x, x2 = normal((5, 700, 1500), 1).cuda(), normal((200, 3000), 2).cuda().bfloat16()
    h, w = normal((3000, 256), 3).cuda().bfloat16(), normal((9000, 256), 4).cuda().bfloat16() / 16
    y = torch.randint(0, 9000, (3000,), device="cuda")
    big = normal((4096, 4096), 5).cuda()
    alone = meo.orthogonalize(x), meo.orthogonalize(x2), meo.linear_cross_entropy(h, w, y)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(streams[3]):
            other = big @ big
        a = meo.orthogonalize(x, stream=streams[0])
        c = meo.linear_cross_entropy(h, w, y, stream=streams[2])
        b = meo.orthogonalize(x2, stream=streams[1])
        torch.cuda.synchronize()
        assert torch.equal(a, alone[0]) and torch.equal(b, alone[1]) and all(torch.equal(p, q) for p, q in zip(c, alone[2]))
        del other


def test_captured_and_replayed():
    shapes = [(40, 64), (64, 40), (3, 200, 150)]
    params = [normal(s, k).cuda() for k, s in enumerate(shapes)]
    grads = [normal(s, 9 + k).cuda() for k, s in enumerate(shapes)]
    twin = [p.clone() for p in params]
    st, st2 = meo.init_muon_state(params), meo.init_muon_state(params)
    step, step2 = meo.MuonStep(params, grads, st, lr=0.1), meo.MuonStep(twin, grads, st2, lr=0.1)
    x = normal((70, 90), 3).cuda()
    first = meo.orthogonalize(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        o = meo.orthogonalize(x)
    for _ in range(3):
        graph.replay()
        step2()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(params, twin))
    assert all(torch.equal(a["momentum"], b["momentum"]) for a, b in zip(st, st2))
    assert torch.equal(o, first)


def test_nothing_beside_the_tensors_is_written():
    big = torch.full((3, 64, 80), 7.0, device="cuda")
    p, m = big[1], torch.full((3, 64, 80), 5.0, device="cuda")
    ws = meo.MuonStep([p], [normal((64, 80), 1).cuda()], [{"momentum": m[1]}], lr=0.1)
    ws()
    assert big[0].eq(7).all() and big[2].eq(7).all() and m[0].eq(5).all() and m[2].eq(5).all()
    assert not big[1].eq(7).any()


def test_optimizer_with_the_loss_of_a_model():
    torch.manual_seed(0)
    model = torch.nn.Sequential(torch.nn.Linear(24, 48, bias=False), torch.nn.Tanh(), torch.nn.Linear(48, 16, bias=False)).cuda()
    opt = meo.Muon(model.parameters(), lr=0.02, weight_decay=0.01)
    ref = [p.detach().double().cpu().numpy() for p in model.parameters()]
    mom = [np.zeros_like(r) for r in ref]
    x, y = normal((64, 24), 1).cuda(), normal((64, 16), 2).cuda()
    for _ in range(3):
        torch.nn.functional.mse_loss(model(x), y).backward()
        for k, p in enumerate(model.parameters()):
            # from where the parameter is: the gradients are those of the model as it has moved
            ref[k], mom[k] = O.step(p.detach().double().cpu().numpy(), p.grad.double().cpu().numpy(), mom[k], lr=0.02, weight_decay=0.01)
        opt.step()
        opt.zero_grad(set_to_none=False)
        for k, p in enumerate(model.parameters()):
            assert far(p.detach(), ref[k]) < 1e-3
    state = opt.state_dict()
    again = meo.Muon(model.parameters(), lr=0.02)
    again.load_state_dict(state)
    assert all(torch.equal(opt.state[p]["momentum"], again.state[p]["momentum"]) for p in model.parameters())


def test_optimizer_keeps_one_workspace():
    """New gradient tensors every step make new plans, not new workspaces."""
    ps = [torch.nn.Parameter(normal((40, 30), k).cuda()) for k in range(2)]
    opt = meo.Muon([{"params": ps[:1]}, {"params": ps[1:], "lr": 0.1}], lr=0.02)
    keep = []
    for t in range(4):
        for k, p in enumerate(ps):
            p.grad = normal((40, 30), 10 * t + k).cuda()
            keep.append(p.grad)
        opt.step()
    assert len({plan.workspace.data_ptr() for plan in opt._plans.values()}) == 1
    graph = torch.cuda.CUDAGraph()
    before = [p.detach().clone() for p in ps]
    with torch.cuda.graph(graph):
        opt.step()
    assert all(torch.equal(p, b) for p, b in zip(ps, before))
    graph.replay()
    torch.cuda.synchronize()
    assert not any(torch.equal(p, b) for p, b in zip(ps, before)) and all(p.isfinite().all() for p in ps)


def test_optimizer_after_a_change_of_shape():
    """The same memory as a matrix of another shape: another step."""
    p, g = torch.nn.Parameter(normal((40, 60), 1).cuda()), normal((40, 60), 2).cuda()
    opt = meo.Muon([p], lr=0.1, momentum=0.0)
    p.grad = g
    opt.step()
    p.grad = None
    p.data = p.data.view(30, 80)
    p.grad = g.view(30, 80)
    twin = p.detach().clone()
    meo.muon_step([twin], [p.grad], meo.init_muon_state([twin]), lr=0.1, momentum=0.0)
    opt.step()
    assert torch.equal(p.detach(), twin)


def test_a_copy_that_never_lands_ends_the_call():
    """A wait runs out: the call ends by itself, the status says so, the parameters stay."""
    p = normal((100, 300), 1).cuda()
    before = p.clone()
    step = meo.MuonStep([p], [normal((100, 300), 2).cuda()], meo.init_muon_state([p]), lr=0.1, steps=1)
    B.muon_debug_stall_copies(True)
    try:
        step()
        out = meo.orthogonalize(before, steps=1)
        torch.cuda.synchronize()
    finally:
        B.muon_debug_stall_copies(False)
    assert step.device_status() == B.ADAF_DEVICE_WAIT_TIMEOUT
    assert torch.equal(p, before) and out.isnan().all()
    step()
    torch.cuda.synchronize()
    assert step.device_status() == 0 and not torch.equal(p, before) and p.isfinite().all()


def test_a_copy_that_never_lands_in_a_sum_in_parts():
    x = normal((70, 3000), 1).cuda()
    B.muon_debug_stall_copies(True)
    try:
        out = meo.orthogonalize(x, steps=1)
        torch.cuda.synchronize()
    finally:
        B.muon_debug_stall_copies(False)
    assert out.isnan().all()
    assert far(meo.orthogonalize(x, dtype=torch.float32), on_gpu(x)) < TOL
