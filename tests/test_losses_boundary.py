"""The C ABI of the losses (include/losses.h) without a GPU: every refusal is
decided on the host before any CUDA call.  The pointers are made up; a call
that passes its checks would fail at its first launch here."""
import ctypes

import pytest
import torch

from memory_efficient_optimizer_gb300 import binding as B
from memory_efficient_optimizer_gb300 import build as libbuild
from memory_efficient_optimizer_gb300 import losses as L

X, G, Y, WS, F = 1 << 32, 1 << 36, 1 << 40, 1 << 41, 1 << 42


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return B.load()


def logits(**kw):
    d = dict(p=X, dtype=B.ADAF_BFLOAT16, batch=2, seq=6, vocab=100, stride_b=600, stride_s=100, temperature=1.0)
    d.update(kw)
    return B.loss_logits(*[d[k] for k in ("p", "dtype", "batch", "seq", "vocab", "stride_b", "stride_s",
                                          "temperature")])


def targets(p=Y, dtype=B.LOSS_INT64, sb=6, ss=1):
    return B.loss_targets(B.loss_rows(p, sb, ss), dtype, -100)


def rows(p=F, sb=6, ss=1):
    return B.loss_rows(p, sb, ss)


def grad(p=G, sb=600, ss=100, scale=1.0):
    return B.loss_grad(p, sb, ss, scale)


def policy(x=None, y=None, g=None, loss=F, ws=WS, n=None, **kw):
    d = dict(adv=rows(), old=rows(), ref=rows(), w=rows(None), lo=0.2, hi=0.2, kl=0.0)
    d.update(kw)
    args = B.loss_policy_args(*d.values())
    B.loss_policy(x or logits(), y or targets(), args, g or grad(), loss, F, F, ws,
                  B.loss_workspace_size(12) if n is None else n, 0)


def preference(x=None, **kw):
    d = dict(ref=rows(), pairs=1, offsets=None, odt=B.LOSS_INT64, kind=0, average=0, beta=0.1, smooth=0.0, margin=0.0)
    d.update(kw)
    B.loss_preference(x or logits(), targets(), B.loss_preference_args(*d.values()), grad(), F, F, F, F, WS,
                      B.loss_workspace_size(12, 1), 0)


def distill(**kw):
    d = dict(ids=F, idt=B.LOSS_INT64, isb=24, iss=4, v=F, vdt=B.ADAF_FLOAT32, vsb=24, vss=4, k=4, lse=rows(None),
             mask=rows(None), w=rows(None))
    d.update(kw)
    B.loss_distill(logits(), B.loss_distill_args(*d.values()), grad(), F, F, WS, B.loss_workspace_size(12), 0)


@pytest.mark.parametrize("bad,msg", [
    (dict(dtype=5), "dtype"), (dict(vocab=0), "vocab"), (dict(batch=-1), "batch"), (dict(seq=-1), "seq"),
    (dict(p=None), "NULL"), (dict(p=X + 1), "aligned"), (dict(dtype=B.ADAF_FLOAT32, p=X + 2), "aligned"),
    (dict(stride_s=-100), "strides"), (dict(stride_b=1 << 60), "strides"), (dict(temperature=0.0), "temperature"),
    (dict(temperature=-1.0), "temperature"), (dict(temperature=float("nan")), "temperature"),
    (dict(temperature=float("inf")), "temperature"), (dict(temperature=1e-40), "temperature")])
def test_logits_refused(lib, bad, msg):
    with pytest.raises(ValueError, match=msg):
        B.loss_token_logprobs(logits(**bad), targets(), F, None, 0)
    with pytest.raises(ValueError, match=msg):
        policy(x=logits(**bad))


@pytest.mark.parametrize("bad", [dict(vocab=1 << 30), dict(batch=1 << 16, seq=1 << 15, stride_b=1, stride_s=1)])
def test_sizes_out_of_range_are_unsupported(lib, bad):
    with pytest.raises(B.AdafactorError) as e:
        B.loss_token_logprobs(logits(**bad), targets(sb=0, ss=0), F, None, 0)
    assert e.value.status == B.ADAF_ERR_UNSUPPORTED


@pytest.mark.parametrize("y,msg", [(targets(dtype=3), "dtype"), (targets(p=None), "NULL"), (targets(p=Y + 4), "aligned"),
                                   (targets(sb=-6), "strides")])
def test_targets_refused(lib, y, msg):
    with pytest.raises(ValueError, match=msg):
        B.loss_token_logprobs(logits(), y, F, None, 0)


@pytest.mark.parametrize("g,msg", [
    (grad(p=G + 1), "aligned"), (grad(ss=99), "rows overlap"), (grad(sb=599), "rows overlap"), (grad(sb=0), "rows overlap"),
    (grad(scale=float("inf")), "scale"), (grad(p=X + 200), "overlaps the logits"), (grad(p=X, sb=700, ss=100), "overlaps"),
    (grad(p=X - 200), "overlaps the logits"), (grad(sb=-600), "strides")])
def test_gradient_refused(lib, g, msg):
    with pytest.raises(ValueError, match=msg):
        policy(g=g)
    with pytest.raises(ValueError, match=msg):
        B.loss_token_logprobs_backward(logits(), targets(), F, rows(), g, 0)


@pytest.mark.parametrize("kw,msg", [
    (dict(adv=rows(None)), "advantages"), (dict(adv=rows(F + 2)), "advantages"), (dict(old=rows(F, -1, 0)), "old_logp"),
    (dict(kl=0.1, ref=rows(None)), "ref_logp"), (dict(kl=-0.1), "kl_coef"), (dict(lo=-0.1), "clip_low"),
    (dict(lo=1.5), "clip_low"), (dict(hi=-0.1), "clip_high"), (dict(hi=float("nan")), "clip_high"),
    (dict(loss=None), "loss"), (dict(ws=None), "workspace"), (dict(ws=WS + 128), "workspace")])
def test_policy_refused(lib, kw, msg):
    with pytest.raises(ValueError, match=msg):
        policy(**kw)


def test_short_workspace_refused(lib):
    need = B.loss_workspace_size(12)
    with pytest.raises(B.AdafactorError, match="workspace") as e:
        policy(n=need - 1)
    assert e.value.status == B.ADAF_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("kw,msg", [
    (dict(pairs=0), "pairs"), (dict(pairs=2), "2 \\* pairs"), (dict(kind=3), "kind"), (dict(beta=0.0), "beta"),
    (dict(beta=float("inf")), "beta"), (dict(smooth=0.5), "label_smoothing"), (dict(smooth=0.1, kind=1), "label_smoothing"),
    (dict(margin=float("nan")), "margin"), (dict(offsets=F, odt=7), "seq_offsets"), (dict(offsets=F + 4), "seq_offsets"),
    (dict(offsets=F), "batch = 1"), (dict(ref=rows(F + 1)), "ref_logp")])
def test_preference_refused(lib, kw, msg):
    with pytest.raises(ValueError, match=msg):
        preference(**kw)


@pytest.mark.parametrize("kw,msg", [
    (dict(k=0), "top_k"), (dict(k=1025), "top_k"), (dict(idt=2), "ids"), (dict(vdt=2), "values"), (dict(ids=None), "ids"),
    (dict(ids=F + 4), "ids"), (dict(v=F + 2), "values"), (dict(isb=-1), "ids"), (dict(lse=rows(F + 2)), "lse"),
    (dict(mask=rows(F, -1, 1)), "mask"), (dict(w=rows(F + 2)), "weights")])
def test_distill_refused(lib, kw, msg):
    with pytest.raises(ValueError, match=msg):
        distill(**kw)


def test_workspace_sizes(lib):
    assert B.loss_workspace_size(0) % 256 == 0
    assert B.loss_workspace_size(1000) < B.loss_workspace_size(100000) < B.loss_workspace_size(100000, 8)
    with pytest.raises(ValueError):
        B.loss_workspace_size(-1)
    with pytest.raises(B.AdafactorError):
        B.loss_workspace_size(1 << 31)
    with pytest.raises(ValueError, match="bytes"):
        B._check(lib.loss_workspace_size(1, 0, None))


def test_null_structs_refused(lib):
    for st in (lib.loss_token_logprobs(None, None, None, None, None),
               lib.loss_token_logprobs(logits(), None, None, None, None),
               lib.loss_policy(logits(), targets(), None, None, None, None, None, None, 0, None),
               lib.loss_preference(logits(), targets(), None, None, None, None, None, None, None, 0, None),
               lib.loss_distill(logits(), None, None, None, None, None, 0, None),
               lib.loss_token_logprobs_backward(logits(), targets(), None, None, None, None)):
        assert st == B.ADAF_ERR_INVALID_ARGUMENT


def test_no_tokens_need_no_pointers(lib):
    none = logits(p=None, batch=0)
    B.loss_token_logprobs(none, targets(p=None), None, None, 0)
    B.loss_token_logprobs_backward(none, targets(p=None), None, rows(None), grad(p=None), 0)


def test_every_entry_point_is_exported(lib):
    for name in B.LOSS_EXPORTS:
        assert isinstance(getattr(lib, name), ctypes._CFuncPtr)
    assert all(B.loss_kernel_name(k).startswith("k_loss_") for k in range(B.loss_num_kernels()))
    assert B.loss_kernel_name(99) == ""


def test_front_end_refuses_on_the_host():
    """What the PyTorch layer looks at before the library: types, shapes, devices."""
    x = torch.zeros(4, 10)
    y = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        L.token_logprobs(x, y)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        L.token_logprobs(x.half(), y)
    with pytest.raises(ValueError, match="vocab"):
        L.token_logprobs(x[0], y)
    with pytest.raises(ValueError, match="innermost stride"):
        L.token_logprobs(torch.zeros(10, 4).t(), y)
