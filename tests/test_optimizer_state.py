"""States of the optimizer classes through a checkpoint, without a GPU."""
import copy
import io
import pickle

import pytest
import torch

import memory_efficient_optimizer_gb300 as meo
from memory_efficient_optimizer_gb300.optim import init_state


@pytest.mark.parametrize("kw", [dict(), dict(beta1=0.9), dict(beta1=0.9, exp_avg_int8=True)])
def test_adafactor_states_keep_their_types(kw):
    """torch casts what it loads to the parameter's type: the carried sum of squares is double precision, and a
    momentum's codes are 8 bits."""
    params = [torch.nn.Parameter(torch.randn(20, 30)), torch.nn.Parameter(torch.randn(7))]
    opt, again = meo.Adafactor(params, **kw), meo.Adafactor(params, **kw)
    for p, st in zip(params, init_state(params, beta1=kw.get("beta1"), exp_avg_int8=kw.get("exp_avg_int8", False))):
        for name, v in st.items():
            v.copy_(torch.randint(-128, 128, v.shape) if v.dtype == torch.int8 else torch.randn(v.shape, dtype=v.dtype))
        opt.state[p].update(st, step=3)
    file = io.BytesIO()
    torch.save(opt.state_dict(), file)
    file.seek(0)
    again.load_state_dict(torch.load(file))
    for p in params:
        assert set(again.state[p]) == set(opt.state[p]) and again.state[p]["step"] == 3
        for name, v in opt.state[p].items():
            if torch.is_tensor(v):
                got = again.state[p][name]
                assert got.dtype == v.dtype and got.is_contiguous() and got.shape == v.shape
                if name != "param_sq_sum":             # (of the parameters as they are at the next step)
                    assert torch.equal(got, v)


@pytest.mark.parametrize("make", [meo.Adafactor, meo.Lamb, lambda ps: meo.Came(ps, lr=1e-3), meo.Muon])
def test_optimizers_can_be_copied_and_pickled(make):
    """A copy steps its own parameters with its own states: here as far as the first check of a device."""
    p = torch.nn.Parameter(torch.randn(4, 6))
    opt = make([p])
    for again in (copy.deepcopy(opt), pickle.loads(pickle.dumps(opt))):
        q, = again.param_groups[0]["params"]
        assert torch.equal(p, q) and q is not p
        q.grad = torch.zeros(4, 6)
        with pytest.raises(ValueError, match="CUDA"):
            again.step()
        again.load_state_dict(again.state_dict())
        with pytest.raises(ValueError, match="CUDA"):
            again.step()
