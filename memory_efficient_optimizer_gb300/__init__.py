"""GB300-native Adafactor step (factored second moment) as a C-ABI CUDA library,
with the multi-tensor LAMB, CAME and Muon steps beside it, and losses over a
vocabulary that give the gradients such a step takes.

The CUDA kernels and the C entry points live in ``csrc/`` (declared in
``include/adafactor.h``, ``include/lamb.h``, ``include/came.h``,
``include/muon.h``, ``include/losses.h`` and ``include/linear_ce.h``); ``binding`` is the ctypes marshalling layer with the
same names as the C entry points; ``optim`` holds the list-of-tensors step and
a ``torch.optim.Optimizer`` wrapper, ``lamb``, ``came`` and ``muon`` the same for LAMB, CAME
and Muon (with its orthogonalisation); ``linear_ce`` holds the cross entropy of an
output layer from its hidden states and weight; ``losses`` holds the policy, preference and distillation losses and token
log-probabilities.  There is no CPU fallback: without the
built library every entry point raises.
"""
from .binding import AdafactorError, library_path  # noqa: F401
from .came import Came, CameStep, came_step, init_came_state, make_came_hparams  # noqa: F401
from .lamb import Lamb, LambStep, init_lamb_state, lamb_step, make_lamb_hparams  # noqa: F401
from .linear_ce import LinearCrossEntropy, linear_cross_entropy  # noqa: F401
from .losses import (DistillLoss, PolicyLoss, PreferenceLoss, TokenLogprobs, distill_loss,  # noqa: F401
                     policy_loss, preference_loss, token_logprobs, token_logprobs_backward)
from .muon import Muon, MuonStep, init_muon_state, make_muon_hparams, muon_step, orthogonalize  # noqa: F401
from .optim import (Adafactor, AdafactorShardStep, AdafactorStep, adafactor_step,  # noqa: F401
                    init_state, make_hparams)

__all__ = ["Adafactor", "AdafactorStep", "AdafactorShardStep", "AdafactorError", "adafactor_step", "init_state",
           "make_hparams", "library_path", "Lamb", "LambStep", "lamb_step", "init_lamb_state",
           "make_lamb_hparams", "Came", "CameStep", "came_step", "init_came_state", "make_came_hparams",
           "Muon", "MuonStep", "muon_step", "init_muon_state", "make_muon_hparams", "orthogonalize",
           "LinearCrossEntropy", "linear_cross_entropy",
           "TokenLogprobs", "PolicyLoss", "PreferenceLoss", "DistillLoss", "token_logprobs",
           "token_logprobs_backward", "policy_loss", "preference_loss", "distill_loss"]
