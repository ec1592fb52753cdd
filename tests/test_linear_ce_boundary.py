"""The C ABI of the linear output layer's cross entropy (include/linear_ce.h)
and its front end without a GPU: every refusal is decided on the host before
any CUDA call."""
import ctypes

import pytest
import torch

from memory_efficient_optimizer_gb300 import binding as B
from memory_efficient_optimizer_gb300 import build as libbuild
from memory_efficient_optimizer_gb300 import linear_ce as L

H, W, GH, GW, Y, WS, F = 1 << 32, 1 << 36, 1 << 40, 1 << 41, 1 << 42, 1 << 43, 1 << 44
BF, FP = B.ADAF_BFLOAT16, B.ADAF_FLOAT32


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return B.load()


def hidden(**kw):
    d = dict(p=H, dtype=BF, batch=2, seq=6, dim=16, sb=96, ss=16)
    d.update(kw)
    return B.linear_ce_hidden(*d.values())


def weight(**kw):
    d = dict(p=W, dtype=BF, vocab=100, sv=16, acc=0)
    d.update(kw)
    return B.linear_ce_weight(*d.values())


def call(h=None, w=None, y=None, gh=None, gw=None, loss=F, logp=F, lse=F, ws=WS, n=None, rows=(None, 0, 0), t=1.0, z=0.0,
         scale=1.0, ydt=B.LOSS_INT64):
    h, w = h or hidden(), w or weight()
    gh, gw = gh or hidden(p=GH), gw or weight(p=GW)
    y = B.loss_targets(B.loss_rows(*(y or (Y, 6, 1))), ydt, -100)
    args = B.linear_ce_args(B.loss_rows(*rows), t, z, scale)
    B.linear_ce(h, w, y, args, gh, gw, loss, logp, lse, ws,
                B.linear_ce_workspace_size(h, w, gh, gw) if n is None else n, 0)


@pytest.mark.parametrize("kw,msg", [
    (dict(h=hidden(dtype=5)), "hidden: unknown dtype"), (dict(w=weight(dtype=5)), "weight: unknown dtype"),
    (dict(h=hidden(batch=-1)), "negative"), (dict(h=hidden(dim=0)), "dim"), (dict(w=weight(vocab=0)), "vocab"),
    (dict(h=hidden(p=None)), "hidden is NULL"), (dict(w=weight(p=None)), "weight is NULL"),
    (dict(h=hidden(p=H + 1)), "hidden is not element"), (dict(w=weight(p=W + 1)), "weight is not element"),
    (dict(h=hidden(ss=-1)), "strides"), (dict(gh=hidden(p=GH, sb=1 << 47)), "strides"), (dict(w=weight(sv=1 << 39)), "strides"), (dict(w=weight(sv=15)), "rows overlap"), (dict(ydt=4), "targets: unknown"),
    (dict(y=(None, 0, 0)), "targets is NULL"), (dict(y=(Y + 4, 6, 1)), "targets is not element"), (dict(y=(Y, -6, 1)), "strides"),
    (dict(rows=(F + 2, 0, 0)), "weights is not"), (dict(rows=(F, -1, 0)), "weights: strides"), (dict(t=0.0), "temperature"),
    (dict(t=-1.0), "temperature"), (dict(t=float("nan")), "temperature"), (dict(t=float("inf")), "temperature"),
    (dict(t=1e-40), "temperature"), (dict(z=-1.0), "z_loss"), (dict(z=float("inf")), "z_loss"),
    (dict(scale=float("nan")), "grad_scale"), (dict(loss=None), "loss is NULL"), (dict(logp=F + 2), "element-aligned"),
    (dict(gh=hidden(p=GH, dtype=9)), "grad_hidden: unknown"), (dict(gh=hidden(p=GH, dim=8)), "size"),
    (dict(gh=hidden(p=GH, ss=15)), "rows overlap"), (dict(gh=hidden(p=GH, sb=90)), "rows overlap"),
    (dict(gh=hidden(p=GH + 1)), "grad_hidden is not"), (dict(gh=hidden(p=H + 32)), "overlaps the hidden"),
    (dict(gh=hidden(p=H, dtype=FP)), "overlaps the hidden"), (dict(gh=hidden(p=W)), "overlaps the weight"),
    (dict(gw=weight(p=GW, dtype=9)), "grad_weight: unknown"), (dict(gw=weight(p=GW, vocab=99)), "size"),
    (dict(gw=weight(p=GW, sv=8)), "rows overlap"), (dict(gw=weight(p=W)), "overlaps the weight"),
    (dict(gw=weight(p=H)), "overlaps the hidden"), (dict(gw=weight(p=GH)), "overlaps grad_hidden"),
    (dict(gw=weight(p=GW + 1)), "grad_weight is not"), (dict(ws=None), "workspace"), (dict(ws=WS + 64), "workspace")])
def test_refused(lib, kw, msg):
    with pytest.raises(ValueError, match=msg):
        call(**kw)


@pytest.mark.parametrize("h,w", [(hidden(dim=1 << 17), weight(sv=1 << 17)), (hidden(batch=1 << 14, seq=1 << 13), weight()),
                                 (hidden(), weight(vocab=1 << 22))])
def test_sizes_out_of_range_are_unsupported(lib, h, w):
    with pytest.raises(B.AdafactorError) as e:
        B.linear_ce_workspace_size(h, w)
    assert e.value.status == B.ADAF_ERR_UNSUPPORTED


def test_workspace(lib):
    alone = B.linear_ce_workspace_size(hidden(), weight())
    grads = B.linear_ce_workspace_size(hidden(), weight(), hidden(p=GH), weight(p=GW))
    assert alone % 256 == 0 and grads > alone
    # a weight that has to be laid out anew takes room for it
    for w in (weight(p=W + 2), weight(sv=17), weight(dtype=FP)):
        assert B.linear_ce_workspace_size(hidden(), w) >= alone + 2 * 100 * 16
    with pytest.raises(B.AdafactorError, match="workspace") as e:
        call(n=grads - 1)
    assert e.value.status == B.ADAF_ERR_WORKSPACE_TOO_SMALL
    # many tokens: pieces, whose exponentials take 2 GB, the weight gradient's fp32 sums, and 256 MB of parts
    big = hidden(batch=1, seq=1 << 20, dim=64, ss=64)
    n = B.linear_ce_workspace_size(big, weight(vocab=32000, sv=64), big, weight(vocab=32000, sv=64))
    assert n < (1 << 31) + (1 << 28) + (1 << 20) * (64 * 2 + 12) + 32000 * 64 * 4 + 33600 * (250 * 8 + 4) + (1 << 20)
    with pytest.raises(ValueError, match="bytes"):
        B._check(lib.linear_ce_workspace_size(hidden(), weight(), None, None, None))


def test_rows_that_reach_too_far_are_refused(lib):
    h, args = hidden(ss=1 << 38, seq=1 << 20, batch=1), B.linear_ce_args(B.loss_rows(None, 0, 0), 1.0, 0.0, 1.0)
    y = B.loss_targets(B.loss_rows(Y, 0, 1), B.LOSS_INT64, -100)
    with pytest.raises(ValueError, match="reach"):
        B.linear_ce(h, weight(), y, args, None, None, F, None, None, WS, 1 << 40, 0)


def test_null_structs_refused(lib):
    y = B.loss_targets(B.loss_rows(Y, 6, 1), B.LOSS_INT64, -100)
    for st in (lib.linear_ce(None, None, None, None, None, None, None, None, None, None, 0, None),
               lib.linear_ce(hidden(), None, None, None, None, None, None, None, None, None, 0, None),
               lib.linear_ce(hidden(), weight(), None, None, None, None, F, None, None, WS, 0, None),
               lib.linear_ce(hidden(), weight(), ctypes.byref(y), None, None, None, F, None, None, WS, 0, None)):
        assert st == B.ADAF_ERR_INVALID_ARGUMENT


def test_every_entry_point_is_exported(lib):
    for name in B.LINEAR_CE_EXPORTS:
        assert isinstance(getattr(lib, name), ctypes._CFuncPtr)
    assert all(B.linear_ce_kernel_name(k).startswith("k_lce_") for k in range(B.linear_ce_num_kernels()))
    assert B.linear_ce_kernel_name(99) == ""


def test_front_end_refuses_on_the_host():
    h, w, y = torch.zeros(4, 8), torch.zeros(9, 8), torch.zeros(4, dtype=torch.int64)
    for args, msg in (((h, w, y), "CUDA"), ((h.half(), w, y), "float32 or bfloat16"), ((h[0], w, y), "tokens, dim"),
                      ((torch.zeros(8, 4).t(), w, y), "innermost"), ((None, w, y), "float32 or bfloat16")):
        with pytest.raises(ValueError, match=msg):
            L.linear_cross_entropy(*args)


@pytest.mark.parametrize("empty", [dict(batch=0), dict(seq=0)])
@pytest.mark.parametrize("gh,gw", [(False, False), (True, False), (False, True), (True, True)])
def test_without_tokens(lib, empty, gh, gw):
    """A batch without tokens has a workspace too, and is refused one that is too small."""
    h, w = hidden(**empty), weight()
    gh, gw = hidden(p=GH, **empty) if gh else None, weight(p=GW) if gw else None
    n = B.linear_ce_workspace_size(h, w, gh, gw)
    assert 256 <= n < B.linear_ce_workspace_size(hidden(), w, gh and hidden(p=GH), gw)
    y, args = B.loss_targets(B.loss_rows(Y, 6, 1), B.LOSS_INT64, -100), B.linear_ce_args(B.loss_rows(None, 0, 0), 1.0, 0.0, 1.0)
    with pytest.raises(B.AdafactorError, match="workspace"):
        B.linear_ce(h, w, y, args, gh, gw, F, F, F, WS, n - 1, 0)
