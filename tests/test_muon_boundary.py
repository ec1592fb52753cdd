"""The Muon C ABI (include/muon.h) and its front end without a GPU: every
refusal is decided on the host before any CUDA call."""
import ctypes

import pytest
import torch

from memory_efficient_optimizer_gb300 import binding as B
from memory_efficient_optimizer_gb300 import build as libbuild
from memory_efficient_optimizer_gb300 import muon as M

P, G, MO, WS = 1 << 32, 1 << 36, 1 << 40, 1 << 41


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return B.load()


def hp(lr=1e-3, momentum=0.95, wd=0.0, adjust=0, **it):
    h = B.muon_hparams(lr, momentum, wd, 1, adjust, B.muon_default_iteration())
    for k, v in it.items():
        setattr(h.iteration, k, v)
    return h


def tensors(*shapes, dtype=B.ADAF_BFLOAT16, p=P, g=G, m=MO):
    return (B.muon_tensor * len(shapes))(*[B.muon_tensor(p, g, dtype, *s, m) for s in shapes])


def matrices(**kw):
    d = dict(x=P, dtype=B.ADAF_FLOAT32, batch=2, rows=6, cols=10, stride_b=60, stride_r=10)
    d.update(kw)
    return B.muon_matrices(*d.values())


def test_defaults(lib):
    B.muon_validate(hp())
    it = B.muon_default_iteration()
    assert it.steps == 5 and it.eps == 1e-7
    assert [tuple(it.coef[k]) for k in range(5)] == [(3.4445, -4.7750, 2.0315)] * 5


@pytest.mark.parametrize("kw,msg", [
    (dict(lr=-1.0), "learning rate"), (dict(lr=float("nan")), "learning rate"), (dict(momentum=1.0), "momentum"),
    (dict(momentum=-0.1), "momentum"), (dict(wd=-0.1), "weight_decay"), (dict(adjust=2), "adjust_lr"),
    (dict(steps=0), "steps"), (dict(steps=17), "steps"), (dict(eps=0.0), "eps"), (dict(eps=float("inf")), "eps"),
    (dict(eps=1e-60), "eps")])
def test_hparams_refused(lib, kw, msg):
    with pytest.raises(ValueError, match=msg):
        B.muon_validate(hp(**kw))
    with pytest.raises(ValueError, match=msg):
        B.muon_step(tensors((1, 4, 4)), 1, hp(**kw), WS, 1 << 20, 0)


@pytest.mark.parametrize("coef", [(3.4445, -4.7750, 3.5), (1.0, 0.0, float("nan")), (2.0, 0.0, 0.0), (2000.0, 0.0, 0.0),
                                  (0.0, 0.0, 0.0)])
def test_coefficients_that_leave_the_range_are_refused(lib, coef):
    with pytest.raises(ValueError, match="coefficients"):
        M.make_iteration(5, coef)


def test_other_coefficients_are_taken(lib):
    M.make_iteration(8, (1.875, -1.25, 0.375))             # the convergent quintic
    M.make_iteration(2, [(3.4445, -4.7750, 2.0315), (1.875, -1.25, 0.375)])
    for bad in [(1.0, 2.0), [(1.875, -1.25, 0.375)], "abc", None, 3]:
        with pytest.raises(ValueError):
            M.make_iteration(2, bad)


@pytest.mark.parametrize("t,msg", [
    (tensors((1, -4, 4)), "negative"), (tensors((-1, 4, 4)), "negative"), (tensors((1, 4, 4), dtype=7), "grad_dtype"),
    (tensors((1, 4, 4), p=None), "NULL"), (tensors((1, 4, 4), g=None), "NULL"), (tensors((1, 4, 4), m=None), "NULL"),
    (tensors((1, 4, 4), p=P + 2), "aligned"), (tensors((1, 4, 4), g=G + 1), "aligned"),
    (tensors((1, 4, 4), m=MO + 1), "aligned")])
def test_lists_refused(lib, t, msg):
    with pytest.raises(ValueError, match=msg):
        B.muon_step(t, 1, hp(), WS, 1 << 30, 0)


@pytest.mark.parametrize("shape", [(1, 1 << 21, 1), (1, 1, 1 << 21), (1, 1 << 16, 1 << 15), (1 << 25, 1, 1)])
def test_sizes_out_of_range_are_unsupported(lib, shape):
    with pytest.raises(B.AdafactorError) as e:
        B.muon_workspace_size(tensors(shape), 1)
    assert e.value.status == B.ADAF_ERR_UNSUPPORTED
    with pytest.raises(B.AdafactorError):
        B.muon_orthogonalize_workspace_size(*shape)


def test_workspace(lib):
    t = tensors((1, 64, 100))
    need = B.muon_workspace_size(t, 1)
    assert need % 256 == 0 and need == B.muon_orthogonalize_workspace_size(1, 64, 100)
    assert need == B.muon_workspace_size(tensors((1, 100, 64)), 1)      # worked on transposed
    assert need < B.muon_workspace_size(tensors((1, 100, 64), (1, 64, 100)), 2)
    # groups are bounded: a long list needs no more than the largest of them
    many = B.muon_workspace_size(tensors((64, 1024, 4096)), 1)
    assert many == B.muon_workspace_size(tensors((64, 1024, 4096), (300, 1024, 4096)), 2)
    with pytest.raises(B.AdafactorError, match="workspace") as e:
        B.muon_step(t, 1, hp(), WS, need - 1, 0)
    assert e.value.status == B.ADAF_ERR_WORKSPACE_TOO_SMALL
    for ws in (None, WS + 128):
        with pytest.raises(ValueError, match="workspace"):
            B.muon_step(t, 1, hp(), ws, need, 0)


@pytest.mark.parametrize("kw,msg", [
    (dict(dtype=4), "dtype"), (dict(x=None), "NULL"), (dict(x=P + 2), "aligned"), (dict(stride_r=-1), "strides"),
    (dict(stride_b=1 << 50), "strides"), (dict(batch=-1), "negative")])
def test_matrices_refused(lib, kw, msg):
    with pytest.raises(ValueError, match=msg):
        B.muon_orthogonalize(matrices(**kw), B.muon_default_iteration(), G, B.ADAF_FLOAT32, WS, 1 << 30, 0)


@pytest.mark.parametrize("x,out", [(dict(), P + 40), (dict(stride_r=12, stride_b=72), P), (dict(dtype=B.ADAF_BFLOAT16), P),
                                   (dict(), P - 40)])
def test_overlap_refused(lib, x, out):
    with pytest.raises(ValueError, match="overlaps"):
        B.muon_orthogonalize(matrices(**x), B.muon_default_iteration(), out, B.ADAF_FLOAT32, WS, 1 << 30, 0)


def test_empty_needs_no_pointers(lib):
    B.muon_step(tensors((0, 4, 4), (1, 0, 4), p=None, g=None, m=None), 2, hp(), None, 0, 0)
    B.muon_step(None, 0, hp(), None, 0, 0)
    B.muon_orthogonalize(matrices(x=None, rows=0), B.muon_default_iteration(), None, B.ADAF_FLOAT32, None, 0, 0)


def test_null_structs_refused(lib):
    for st in (lib.muon_validate(None), lib.muon_validate_iteration(None), lib.muon_step(None, 0, None, None, 0, None),
               lib.muon_step(None, 1, ctypes.byref(hp()), None, 0, None), lib.muon_workspace_size(None, 1, None),
               lib.muon_orthogonalize(None, ctypes.byref(B.muon_default_iteration()), None, 0, None, 0, None),
               lib.muon_device_status(None, None, None)):
        assert st == B.ADAF_ERR_INVALID_ARGUMENT


def test_every_entry_point_is_exported(lib):
    for name in B.MUON_EXPORTS:
        assert isinstance(getattr(lib, name), ctypes._CFuncPtr)
    assert all(B.muon_kernel_name(k).startswith("k_muon_") for k in range(B.muon_num_kernels()))
    assert B.muon_kernel_name(99) == ""


def test_front_end_refuses_on_the_host(lib):
    w, v = torch.zeros(4, 6), torch.zeros(6)
    st = M.init_muon_state([w])
    with pytest.raises(ValueError, match="CUDA"):
        M.MuonStep([w], [w], st)
    with pytest.raises(ValueError, match="two dimensions"):
        M.MuonStep([v], [v], M.init_muon_state([v]))
    with pytest.raises(ValueError, match="two dimensions"):
        M.Muon([torch.nn.Parameter(v)])
    with pytest.raises(ValueError, match="adjust_lr"):
        M.Muon([torch.nn.Parameter(w)], adjust_lr="rms")
    with pytest.raises(ValueError, match="same length"):
        M.MuonStep([w], [], st)
    for x, msg in ((w, "CUDA"), (v, "two dimensions"), (w.half(), "float32 or bfloat16"), (None, "float32 or bfloat16")):
        with pytest.raises(ValueError, match=msg):
            M.orthogonalize(x)
    with pytest.raises(ValueError, match="result"):
        M.orthogonalize(w, dtype=torch.float16)
    with pytest.raises(ValueError, match="result"):
        M.orthogonalize(w, out=v.half())


def test_optimizer_refuses_tensors_of_the_host(lib):
    p = torch.nn.Parameter(torch.zeros(4, 6))
    p.grad = torch.zeros(4, 6)
    with pytest.raises(ValueError, match="CUDA"):
        M.Muon([p]).step()


@pytest.mark.parametrize("at,msg", [
    (dict(), "tensors 0 and 1 overlap"),                                             # one tensor listed twice
    (dict(p=P + (1 << 20)), "tensors 0 and 1 overlap"),                              # its momentum alone
    (dict(m=MO + (1 << 20)), "tensors 0 and 1 overlap"),                             # the parameter alone
    (dict(p=P + 4 * (4 * 6 - 1), m=MO + (1 << 20)), "tensors 0 and 1 overlap"),      # by one value
    (dict(p=MO, m=MO + (1 << 20)), "tensors 0 and 1 overlap"),                       # a parameter on a momentum
    (dict(p=P + (1 << 20), m=MO + (1 << 20), g=P), "tensors 0 and 1 overlap"),       # a gradient on another's parameter
    (dict(p=P + (1 << 20), m=P + (1 << 20) + 64), "tensor 1: p, g and momentum overlap"),
    (dict(p=P + (1 << 20), m=MO + (1 << 20), g=P + (1 << 20)), "tensor 1: p, g and momentum overlap")])
def test_shared_memory_in_a_list_is_refused(lib, at, msg):
    one, other = dict(p=P, g=G, m=MO), dict(p=P, g=G, m=MO)
    other.update(at)
    t = (B.muon_tensor * 2)(*[B.muon_tensor(d["p"], d["g"], B.ADAF_FLOAT32, 1, 4, 6, d["m"]) for d in (one, other)])
    with pytest.raises(ValueError, match=msg):
        B.muon_step(t, 2, hp(), WS, 1 << 30, 0)


def test_gradients_may_be_shared_and_tensors_may_touch(lib):
    """Then the next check is the workspace's."""
    t = (B.muon_tensor * 3)(*[B.muon_tensor(P + 96 * k, G, B.ADAF_FLOAT32, 1, 4, 6, P + 96 * (k + 3)) for k in (1, 0, 2)])
    with pytest.raises(B.AdafactorError, match="workspace needs"):
        B.muon_step(t, 3, hp(), WS, 0, 0)
    # an empty tensor has no memory to share
    t = (B.muon_tensor * 2)(*[B.muon_tensor(P, G, B.ADAF_FLOAT32, b, 4, 6, MO) for b in (1, 0)])
    with pytest.raises(B.AdafactorError, match="workspace needs"):
        B.muon_step(t, 2, hp(), WS, 0, 0)


def test_overlaps_are_found_in_long_lists(lib):
    """Against every pair looked at, with one overlap or none in lists in any order."""
    import random
    rng = random.Random(5)
    for trial in range(60):
        n, places = 12, list(range(40))
        rng.shuffle(places)
        rows = [rng.randint(1, 6) for _ in range(n)]
        ts = [[P + 4096 * places[2 * k], G, P + 4096 * places[2 * k + 1]] for k in range(n)]
        if trial % 2:
            k = rng.randrange(n)
            ts[k][rng.randrange(3)] = ts[(k + 1 + rng.randrange(n - 1)) % n][rng.choice((0, 2))] + 4 * rng.randint(0, 3)
        ext = [(i, j, a, a + 4 * 8 * rows[i]) for i, t in enumerate(ts) for j, a in enumerate(t)]
        meets = any(x[2] < y[3] and y[2] < x[3] and not (x[1] == y[1] == 1) for a, x in enumerate(ext) for y in ext[:a])
        t = (B.muon_tensor * n)(*[B.muon_tensor(p, g, B.ADAF_FLOAT32, 1, r, 8, m) for (p, g, m), r in zip(ts, rows)])
        with pytest.raises(Exception, match="overlap" if meets else "workspace needs"):
            B.muon_step(t, n, hp(), WS, 0, 0)


@pytest.mark.parametrize("shape,per_value", [
    ((1, 4096, 4096), 16), ((1, 512, 512), 16), ((7, 1000, 1000), 16),   # x twice in fp16 and in fp32; A and its polynomial, twice
    ((1, 4096, 14336), 8 + 16 * 4096 / 14336),                           # wide: four symmetric matrices, for two steps at once
    ((1, 1024, 4096), 8 + 8 / 4)])                                       # too few of them for that
def test_workspace_by_value(lib, shape, per_value):
    """Bytes for each value, but for the sums, the diagonals and the sums of x x^T in parts."""
    values = shape[0] * shape[1] * shape[2]
    have = B.muon_orthogonalize_workspace_size(*shape)
    assert per_value * values <= have <= 1.05 * per_value * values + (12 << 20)
