"""ctypes binding of the C ABI in include/adafactor.h, include/lamb.h,
include/came.h, include/losses.h, include/muon.h and include/linear_ce.h
(argument marshalling only).

Every function here has the name of the C entry point it calls and does no
arithmetic of the method: all of the step runs in the CUDA library.  Loading
fails loudly when the library has not been built; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

ADAF_OK = 0
ADAF_ERR_INVALID_ARGUMENT = 1
ADAF_ERR_UNSUPPORTED = 2
ADAF_ERR_WORKSPACE_TOO_SMALL = 3
ADAF_ERR_CUDA = 4
ADAF_FLOAT32 = 0
ADAF_BFLOAT16 = 1
ADAF_MAX_NDIM = 8
ADAF_DEVICE_WAIT_TIMEOUT = 1

# Entry points declared in include/adafactor.h.
EXPORTS = (
    "adafactor_default_hparams", "adafactor_validate", "adafactor_workspace_size",
    "adafactor_step", "adafactor_device_status", "adafactor_last_error", "adafactor_release_cache",
    "adafactor_profile_enable", "adafactor_profile_read", "adafactor_num_kernels",
    "adafactor_kernel_name", "adafactor_step_noalloc", "adafactor_noalloc_device_status",
    "adafactor_debug_stall_copies",
    "adafactor_shard_sizes", "adafactor_shard_begin", "adafactor_shard_middle", "adafactor_shard_end",
)
# Entry points declared in include/came.h.
CAME_EXPORTS = (
    "came_default_hparams", "came_validate", "came_workspace_size", "came_step", "came_profile_enable",
    "came_profile_read", "came_num_kernels", "came_kernel_name",
)
# Entry points declared in include/lamb.h.
LAMB_EXPORTS = (
    "lamb_validate", "lamb_workspace_size", "lamb_step", "lamb_trust_ratios", "lamb_profile_enable",
    "lamb_profile_read", "lamb_num_kernels", "lamb_kernel_name",
)

# Entry points declared in include/losses.h.
LOSS_EXPORTS = (
    "loss_workspace_size", "loss_token_logprobs", "loss_token_logprobs_backward", "loss_policy", "loss_preference",
    "loss_distill", "loss_debug_stall_copies", "loss_profile_enable", "loss_profile_read", "loss_num_kernels",
    "loss_kernel_name",
)
# Entry points declared in include/muon.h.
MUON_EXPORTS = (
    "muon_default_iteration", "muon_validate", "muon_validate_iteration", "muon_workspace_size",
    "muon_orthogonalize_workspace_size", "muon_step", "muon_orthogonalize", "muon_device_status",
    "muon_debug_stall_copies", "muon_profile_enable", "muon_profile_read", "muon_num_kernels", "muon_kernel_name",
)
# Entry points declared in include/linear_ce.h.
LINEAR_CE_EXPORTS = (
    "linear_ce_workspace_size", "linear_ce", "linear_ce_debug_stall_copies", "linear_ce_profile_enable",
    "linear_ce_profile_read", "linear_ce_num_kernels", "linear_ce_kernel_name",
)
MUON_MAX_STEPS = 16
MUON_ADJUST = {"original": 0, "match_rms": 1}
LOSS_INT32 = 0
LOSS_INT64 = 1
LOSS_MAX_TOP_K = 1024
LOSS_PREFERENCE_KINDS = {"sigmoid": 0, "hinge": 1, "squared": 2}


class adaf_tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("grad_dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * ADAF_MAX_NDIM)]


class adaf_state(ctypes.Structure):
    _fields_ = [("exp_avg_sq_row", ctypes.c_void_p), ("exp_avg_sq_col", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("param_sq_sum", ctypes.c_void_p),
                ("exp_avg_codes", ctypes.c_void_p), ("exp_avg_scales", ctypes.c_void_p)]


class adaf_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("has_lr", ctypes.c_int32),
                ("eps1", ctypes.c_double), ("eps2", ctypes.c_double),
                ("clip_threshold", ctypes.c_double), ("decay_rate", ctypes.c_double),
                ("beta1", ctypes.c_double), ("has_beta1", ctypes.c_int32),
                ("weight_decay", ctypes.c_double), ("scale_parameter", ctypes.c_int32),
                ("relative_step", ctypes.c_int32), ("warmup_init", ctypes.c_int32),
                ("param_sq_sum_valid", ctypes.c_int32), ("exp_avg_int8", ctypes.c_int32)]


class adaf_shard(ctypes.Structure):
    _fields_ = [("global_rows", ctypes.c_int64)]


class lamb_tensor(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("grad_dtype", ctypes.c_int32),
                ("numel", ctypes.c_int64), ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p)]


class lamb_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("bias_correction", ctypes.c_int32)]


class came_tensor(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("grad_dtype", ctypes.c_int32),
                ("ndim", ctypes.c_int32), ("shape", ctypes.c_int64 * ADAF_MAX_NDIM)]


class came_state(ctypes.Structure):
    _fields_ = [("exp_avg", ctypes.c_void_p), ("exp_avg_sq_row", ctypes.c_void_p),
                ("exp_avg_sq_col", ctypes.c_void_p), ("exp_avg_res_row", ctypes.c_void_p),
                ("exp_avg_res_col", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("exp_avg_res", ctypes.c_void_p)]


class came_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("eps1", ctypes.c_double), ("eps2", ctypes.c_double),
                ("clip_threshold", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("beta3", ctypes.c_double), ("weight_decay", ctypes.c_double)]


class loss_logits(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("batch", ctypes.c_int64), ("seq", ctypes.c_int64),
                ("vocab", ctypes.c_int64), ("stride_b", ctypes.c_int64), ("stride_s", ctypes.c_int64),
                ("temperature", ctypes.c_double)]


class loss_rows(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_s", ctypes.c_int64)]


class loss_targets(ctypes.Structure):
    _fields_ = [("rows", loss_rows), ("dtype", ctypes.c_int32), ("ignore_index", ctypes.c_int64)]


class loss_grad(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_s", ctypes.c_int64),
                ("scale", ctypes.c_double)]


class loss_policy_args(ctypes.Structure):
    _fields_ = [("advantages", loss_rows), ("old_logp", loss_rows), ("ref_logp", loss_rows), ("weights", loss_rows),
                ("clip_low", ctypes.c_double), ("clip_high", ctypes.c_double), ("kl_coef", ctypes.c_double)]


class loss_preference_args(ctypes.Structure):
    _fields_ = [("ref_logp", loss_rows), ("pairs", ctypes.c_int64), ("seq_offsets", ctypes.c_void_p),
                ("offsets_dtype", ctypes.c_int32), ("kind", ctypes.c_int32), ("average", ctypes.c_int32),
                ("beta", ctypes.c_double), ("label_smoothing", ctypes.c_double), ("margin", ctypes.c_double)]


class loss_distill_args(ctypes.Structure):
    _fields_ = [("ids", ctypes.c_void_p), ("ids_dtype", ctypes.c_int32), ("ids_stride_b", ctypes.c_int64),
                ("ids_stride_s", ctypes.c_int64), ("values", ctypes.c_void_p), ("values_dtype", ctypes.c_int32),
                ("values_stride_b", ctypes.c_int64), ("values_stride_s", ctypes.c_int64), ("top_k", ctypes.c_int32),
                ("lse", loss_rows), ("mask", loss_rows), ("weights", loss_rows)]


class muon_tensor(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("grad_dtype", ctypes.c_int32),
                ("batch", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("momentum", ctypes.c_void_p)]


class muon_iteration(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int32), ("coef", (ctypes.c_double * 3) * MUON_MAX_STEPS), ("eps", ctypes.c_double)]


class muon_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("momentum", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("nesterov", ctypes.c_int32), ("adjust_lr", ctypes.c_int32), ("iteration", muon_iteration)]


class muon_matrices(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("batch", ctypes.c_int64), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("stride_b", ctypes.c_int64), ("stride_r", ctypes.c_int64)]


class linear_ce_hidden(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("batch", ctypes.c_int64), ("seq", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("stride_b", ctypes.c_int64), ("stride_s", ctypes.c_int64)]


class linear_ce_weight(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("vocab", ctypes.c_int64),
                ("stride_v", ctypes.c_int64), ("accumulate", ctypes.c_int32)]


class linear_ce_args(ctypes.Structure):
    _fields_ = [("weights", loss_rows), ("temperature", ctypes.c_double), ("z_loss", ctypes.c_double),
                ("grad_scale", ctypes.c_double)]


class AdafactorError(RuntimeError):
    """A non-zero adaf_status other than an argument error."""

    def __init__(self, status: int, message: str):
        super().__init__(f"adafactor status {status}: {message}")
        self.status = status


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False) -> ctypes.CDLL:
    """Loads libmeo_adafactor.so; raises if it is missing (no CPU fallback)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            if not build_if_missing:
                raise RuntimeError(
                    f"{path} is missing: build it with `python -m memory_efficient_optimizer_gb300.build` "
                    "(there is no fallback implementation)")
            _build.build()
        lib = ctypes.CDLL(path)
        P = ctypes.POINTER
        lib.adafactor_default_hparams.restype = None
        lib.adafactor_default_hparams.argtypes = [P(adaf_hparams)]
        lib.adafactor_validate.restype = ctypes.c_int
        lib.adafactor_validate.argtypes = [P(adaf_hparams)]
        lib.adafactor_workspace_size.restype = ctypes.c_int
        lib.adafactor_workspace_size.argtypes = [P(adaf_tensor), ctypes.c_int32, P(ctypes.c_size_t)]
        lib.adafactor_step.restype = ctypes.c_int
        lib.adafactor_step.argtypes = [P(adaf_tensor), P(adaf_state), ctypes.c_int32, ctypes.c_int64,
                                       P(adaf_hparams), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        lib.adafactor_step_noalloc.restype = ctypes.c_int
        lib.adafactor_step_noalloc.argtypes = [P(adaf_tensor), P(adaf_state), ctypes.c_int32, ctypes.c_int64,
                                               P(adaf_hparams), ctypes.c_void_p]
        lib.adafactor_noalloc_device_status.restype = ctypes.c_int
        lib.adafactor_noalloc_device_status.argtypes = [ctypes.c_void_p, P(ctypes.c_int32)]
        lib.adafactor_device_status.restype = ctypes.c_int
        lib.adafactor_device_status.argtypes = [ctypes.c_void_p, ctypes.c_void_p, P(ctypes.c_int32)]
        lib.adafactor_debug_stall_copies.restype = None
        lib.adafactor_debug_stall_copies.argtypes = [ctypes.c_int32]
        lib.adafactor_last_error.restype = ctypes.c_char_p
        lib.adafactor_last_error.argtypes = []
        lib.adafactor_release_cache.restype = None
        lib.adafactor_release_cache.argtypes = []
        lib.adafactor_profile_enable.restype = ctypes.c_int
        lib.adafactor_profile_enable.argtypes = [ctypes.c_int32]
        lib.adafactor_profile_read.restype = ctypes.c_int
        lib.adafactor_profile_read.argtypes = [P(ctypes.c_double), P(ctypes.c_int64), ctypes.c_int32]
        lib.adafactor_num_kernels.restype = ctypes.c_int32
        lib.adafactor_num_kernels.argtypes = []
        lib.adafactor_kernel_name.restype = ctypes.c_char_p
        lib.adafactor_kernel_name.argtypes = [ctypes.c_int32]
        lib.adafactor_shard_sizes.restype = ctypes.c_int
        lib.adafactor_shard_sizes.argtypes = [P(adaf_tensor), P(adaf_shard), ctypes.c_int32, P(ctypes.c_size_t),
                                              P(ctypes.c_size_t), P(ctypes.c_size_t)]
        shard_head = [P(adaf_tensor), P(adaf_state), P(adaf_shard), ctypes.c_int32, ctypes.c_int64,
                      P(adaf_hparams), ctypes.c_void_p, ctypes.c_size_t]
        lib.adafactor_shard_begin.restype = ctypes.c_int
        lib.adafactor_shard_begin.argtypes = shard_head + [ctypes.c_void_p, ctypes.c_void_p]
        lib.adafactor_shard_middle.restype = ctypes.c_int
        lib.adafactor_shard_middle.argtypes = shard_head + [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
        lib.adafactor_shard_end.restype = ctypes.c_int
        lib.adafactor_shard_end.argtypes = shard_head + [ctypes.c_void_p, ctypes.c_void_p]
        lib.came_default_hparams.restype = None
        lib.came_default_hparams.argtypes = [P(came_hparams)]
        lib.came_validate.restype = ctypes.c_int
        lib.came_validate.argtypes = [P(came_hparams)]
        lib.came_workspace_size.restype = ctypes.c_int
        lib.came_workspace_size.argtypes = [P(came_tensor), ctypes.c_int32, P(ctypes.c_size_t)]
        lib.came_step.restype = ctypes.c_int
        lib.came_step.argtypes = [P(came_tensor), P(came_state), ctypes.c_int32, ctypes.c_int64, P(came_hparams),
                                  ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        lib.came_profile_enable.restype = ctypes.c_int
        lib.came_profile_enable.argtypes = [ctypes.c_int32]
        lib.came_profile_read.restype = ctypes.c_int
        lib.came_profile_read.argtypes = [P(ctypes.c_double), P(ctypes.c_int64), ctypes.c_int32]
        lib.came_num_kernels.restype = ctypes.c_int32
        lib.came_num_kernels.argtypes = []
        lib.came_kernel_name.restype = ctypes.c_char_p
        lib.came_kernel_name.argtypes = [ctypes.c_int32]
        lib.lamb_validate.restype = ctypes.c_int
        lib.lamb_validate.argtypes = [P(lamb_hparams)]
        lib.lamb_workspace_size.restype = ctypes.c_int
        lib.lamb_workspace_size.argtypes = [P(lamb_tensor), ctypes.c_int32, P(ctypes.c_size_t)]
        lib.lamb_step.restype = ctypes.c_int
        lib.lamb_step.argtypes = [P(lamb_tensor), ctypes.c_int32, ctypes.c_int64, P(lamb_hparams),
                                  ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        lib.lamb_trust_ratios.restype = ctypes.c_int
        lib.lamb_trust_ratios.argtypes = [ctypes.c_void_p, ctypes.c_int32, P(ctypes.c_double), ctypes.c_void_p]
        lib.lamb_profile_enable.restype = ctypes.c_int
        lib.lamb_profile_enable.argtypes = [ctypes.c_int32]
        lib.lamb_profile_read.restype = ctypes.c_int
        lib.lamb_profile_read.argtypes = [P(ctypes.c_double), P(ctypes.c_int64), ctypes.c_int32]
        lib.lamb_num_kernels.restype = ctypes.c_int32
        lib.lamb_num_kernels.argtypes = []
        lib.lamb_kernel_name.restype = ctypes.c_char_p
        lib.lamb_kernel_name.argtypes = [ctypes.c_int32]
        lib.loss_workspace_size.restype = ctypes.c_int
        lib.loss_workspace_size.argtypes = [ctypes.c_int64, ctypes.c_int64, P(ctypes.c_size_t)]
        lib.loss_token_logprobs.restype = ctypes.c_int
        lib.loss_token_logprobs.argtypes = [P(loss_logits), P(loss_targets), ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_void_p]
        lib.loss_token_logprobs_backward.restype = ctypes.c_int
        lib.loss_token_logprobs_backward.argtypes = [P(loss_logits), P(loss_targets), ctypes.c_void_p, P(loss_rows),
                                                     P(loss_grad), ctypes.c_void_p]
        lib.loss_policy.restype = ctypes.c_int
        lib.loss_policy.argtypes = [P(loss_logits), P(loss_targets), P(loss_policy_args), P(loss_grad),
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_size_t, ctypes.c_void_p]
        lib.loss_preference.restype = ctypes.c_int
        lib.loss_preference.argtypes = [P(loss_logits), P(loss_targets), P(loss_preference_args), P(loss_grad),
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        lib.loss_distill.restype = ctypes.c_int
        lib.loss_distill.argtypes = [P(loss_logits), P(loss_distill_args), P(loss_grad), ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        lib.loss_debug_stall_copies.restype = None
        lib.loss_debug_stall_copies.argtypes = [ctypes.c_int32]
        lib.loss_profile_enable.restype = ctypes.c_int
        lib.loss_profile_enable.argtypes = [ctypes.c_int32]
        lib.loss_profile_read.restype = ctypes.c_int
        lib.loss_profile_read.argtypes = [P(ctypes.c_double), P(ctypes.c_int64), ctypes.c_int32]
        lib.loss_num_kernels.restype = ctypes.c_int32
        lib.loss_num_kernels.argtypes = []
        lib.loss_kernel_name.restype = ctypes.c_char_p
        lib.loss_kernel_name.argtypes = [ctypes.c_int32]
        lib.muon_default_iteration.restype = None
        lib.muon_default_iteration.argtypes = [P(muon_iteration)]
        lib.muon_validate.restype = ctypes.c_int
        lib.muon_validate.argtypes = [P(muon_hparams)]
        lib.muon_validate_iteration.restype = ctypes.c_int
        lib.muon_validate_iteration.argtypes = [P(muon_iteration)]
        lib.muon_workspace_size.restype = ctypes.c_int
        lib.muon_workspace_size.argtypes = [P(muon_tensor), ctypes.c_int32, P(ctypes.c_size_t)]
        lib.muon_orthogonalize_workspace_size.restype = ctypes.c_int
        lib.muon_orthogonalize_workspace_size.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                                          P(ctypes.c_size_t)]
        lib.muon_step.restype = ctypes.c_int
        lib.muon_step.argtypes = [P(muon_tensor), ctypes.c_int32, P(muon_hparams), ctypes.c_void_p, ctypes.c_size_t,
                                  ctypes.c_void_p]
        lib.muon_orthogonalize.restype = ctypes.c_int
        lib.muon_orthogonalize.argtypes = [P(muon_matrices), P(muon_iteration), ctypes.c_void_p, ctypes.c_int32,
                                           ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        lib.muon_device_status.restype = ctypes.c_int
        lib.muon_device_status.argtypes = [ctypes.c_void_p, ctypes.c_void_p, P(ctypes.c_int32)]
        lib.muon_debug_stall_copies.restype = None
        lib.muon_debug_stall_copies.argtypes = [ctypes.c_int32]
        lib.muon_profile_enable.restype = ctypes.c_int
        lib.muon_profile_enable.argtypes = [ctypes.c_int32]
        lib.muon_profile_read.restype = ctypes.c_int
        lib.muon_profile_read.argtypes = [P(ctypes.c_double), P(ctypes.c_int64), ctypes.c_int32]
        lib.muon_num_kernels.restype = ctypes.c_int32
        lib.muon_num_kernels.argtypes = []
        lib.muon_kernel_name.restype = ctypes.c_char_p
        lib.muon_kernel_name.argtypes = [ctypes.c_int32]
        lib.linear_ce_workspace_size.restype = ctypes.c_int
        lib.linear_ce_workspace_size.argtypes = [P(linear_ce_hidden), P(linear_ce_weight), P(linear_ce_hidden),
                                                 P(linear_ce_weight), P(ctypes.c_size_t)]
        lib.linear_ce.restype = ctypes.c_int
        lib.linear_ce.argtypes = [P(linear_ce_hidden), P(linear_ce_weight), P(loss_targets), P(linear_ce_args),
                                  P(linear_ce_hidden), P(linear_ce_weight), ctypes.c_void_p, ctypes.c_void_p,
                                  ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        lib.linear_ce_debug_stall_copies.restype = None
        lib.linear_ce_debug_stall_copies.argtypes = [ctypes.c_int32]
        lib.linear_ce_profile_enable.restype = ctypes.c_int
        lib.linear_ce_profile_enable.argtypes = [ctypes.c_int32]
        lib.linear_ce_profile_read.restype = ctypes.c_int
        lib.linear_ce_profile_read.argtypes = [P(ctypes.c_double), P(ctypes.c_int64), ctypes.c_int32]
        lib.linear_ce_num_kernels.restype = ctypes.c_int32
        lib.linear_ce_num_kernels.argtypes = []
        lib.linear_ce_kernel_name.restype = ctypes.c_char_p
        lib.linear_ce_kernel_name.argtypes = [ctypes.c_int32]
        _lib = lib
        return lib


def _check(status: int) -> None:
    if status == ADAF_OK:
        return
    msg = adafactor_last_error()
    if status == ADAF_ERR_INVALID_ARGUMENT:
        raise ValueError(msg)
    raise AdafactorError(status, msg)


def adafactor_default_hparams() -> adaf_hparams:
    hp = adaf_hparams()
    load().adafactor_default_hparams(ctypes.byref(hp))
    return hp


def adafactor_validate(hp: adaf_hparams) -> None:
    _check(load().adafactor_validate(ctypes.byref(hp)))


def adafactor_workspace_size(tensors, n: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().adafactor_workspace_size(tensors, int(n), ctypes.byref(out)))
    return int(out.value)


def adafactor_step(tensors, states, n: int, step: int, hp: adaf_hparams, workspace: int,
                   workspace_bytes: int, stream: int) -> None:
    _check(load().adafactor_step(tensors, states, int(n), int(step), ctypes.byref(hp),
                                 ctypes.c_void_p(workspace), ctypes.c_size_t(workspace_bytes),
                                 ctypes.c_void_p(stream)))


def adafactor_step_noalloc(tensors, states, n: int, step: int, hp: adaf_hparams, stream: int) -> None:
    """The step with the library's fixed scratch area (no workspace argument)."""
    _check(load().adafactor_step_noalloc(tensors, states, int(n), int(step), ctypes.byref(hp),
                                         ctypes.c_void_p(stream)))


def adafactor_shard_sizes(tensors, shards, n: int):
    """(workspace bytes, round-1 bytes, round-2 bytes) of a row-sharded step."""
    ws, r1, r2 = ctypes.c_size_t(0), ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(load().adafactor_shard_sizes(tensors, shards, int(n), ctypes.byref(ws), ctypes.byref(r1),
                                        ctypes.byref(r2)))
    return int(ws.value), int(r1.value), int(r2.value)


def adafactor_shard_begin(tensors, states, shards, n: int, step: int, hp: adaf_hparams, workspace: int,
                          workspace_bytes: int, round1: int, stream: int) -> None:
    _check(load().adafactor_shard_begin(tensors, states, shards, int(n), int(step), ctypes.byref(hp),
                                        ctypes.c_void_p(workspace), ctypes.c_size_t(workspace_bytes),
                                        ctypes.c_void_p(round1), ctypes.c_void_p(stream)))


def adafactor_shard_middle(tensors, states, shards, n: int, step: int, hp: adaf_hparams, workspace: int,
                           workspace_bytes: int, round1: int, round2: int, stream: int) -> None:
    _check(load().adafactor_shard_middle(tensors, states, shards, int(n), int(step), ctypes.byref(hp),
                                         ctypes.c_void_p(workspace), ctypes.c_size_t(workspace_bytes),
                                         ctypes.c_void_p(round1), ctypes.c_void_p(round2), ctypes.c_void_p(stream)))


def adafactor_shard_end(tensors, states, shards, n: int, step: int, hp: adaf_hparams, workspace: int,
                        workspace_bytes: int, round2: int, stream: int) -> None:
    _check(load().adafactor_shard_end(tensors, states, shards, int(n), int(step), ctypes.byref(hp),
                                      ctypes.c_void_p(workspace), ctypes.c_size_t(workspace_bytes),
                                      ctypes.c_void_p(round2), ctypes.c_void_p(stream)))


def adafactor_device_status(workspace: int, stream: int) -> int:
    out = ctypes.c_int32(0)
    _check(load().adafactor_device_status(ctypes.c_void_p(workspace), ctypes.c_void_p(stream), ctypes.byref(out)))
    return int(out.value)


def adafactor_noalloc_device_status(stream: int) -> int:
    """Status word of the last adafactor_step_noalloc() on the current device."""
    out = ctypes.c_int32(0)
    _check(load().adafactor_noalloc_device_status(ctypes.c_void_p(stream), ctypes.byref(out)))
    return int(out.value)


def adafactor_debug_stall_copies(on: bool) -> None:
    """Testing hook: make the bulk-copy producers issue nothing (see the header)."""
    load().adafactor_debug_stall_copies(1 if on else 0)


def adafactor_last_error() -> str:
    return load().adafactor_last_error().decode(errors="replace")


def adafactor_release_cache() -> None:
    load().adafactor_release_cache()


def adafactor_profile_enable(on: bool) -> None:
    _check(load().adafactor_profile_enable(1 if on else 0))


def adafactor_num_kernels() -> int:
    return int(load().adafactor_num_kernels())


def adafactor_kernel_name(k: int) -> str:
    return load().adafactor_kernel_name(int(k)).decode()


def adafactor_profile_read() -> dict:
    """{kernel name: (total ms, launches)} for the events recorded since the last read."""
    nk = adafactor_num_kernels()
    ms = (ctypes.c_double * nk)()
    launches = (ctypes.c_int64 * nk)()
    _check(load().adafactor_profile_read(ms, launches, nk))
    return {adafactor_kernel_name(k): (float(ms[k]), int(launches[k])) for k in range(nk)}


# ---- LAMB (include/lamb.h) --------------------------------------------------

def lamb_validate(hp: lamb_hparams) -> None:
    _check(load().lamb_validate(ctypes.byref(hp)))


def lamb_workspace_size(tensors, n: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().lamb_workspace_size(tensors, int(n), ctypes.byref(out)))
    return int(out.value)


def lamb_step(tensors, n: int, step: int, hp: lamb_hparams, workspace: int, workspace_bytes: int,
              stream: int) -> None:
    _check(load().lamb_step(tensors, int(n), int(step), ctypes.byref(hp), ctypes.c_void_p(workspace),
                            ctypes.c_size_t(workspace_bytes), ctypes.c_void_p(stream)))


def lamb_trust_ratios(workspace: int, n: int, stream: int) -> list:
    out = (ctypes.c_double * max(1, int(n)))()
    _check(load().lamb_trust_ratios(ctypes.c_void_p(workspace), int(n), out, ctypes.c_void_p(stream)))
    return [float(out[k]) for k in range(int(n))]


def lamb_profile_enable(on: bool) -> None:
    _check(load().lamb_profile_enable(1 if on else 0))


def lamb_num_kernels() -> int:
    return int(load().lamb_num_kernels())


def lamb_kernel_name(k: int) -> str:
    return load().lamb_kernel_name(int(k)).decode()


def lamb_profile_read() -> dict:
    """{kernel name: (total ms, launches)} for the LAMB events recorded since the last read."""
    nk = lamb_num_kernels()
    ms = (ctypes.c_double * nk)()
    launches = (ctypes.c_int64 * nk)()
    _check(load().lamb_profile_read(ms, launches, nk))
    return {lamb_kernel_name(k): (float(ms[k]), int(launches[k])) for k in range(nk)}


# ---- CAME (include/came.h) --------------------------------------------------

def came_default_hparams() -> came_hparams:
    hp = came_hparams()
    load().came_default_hparams(ctypes.byref(hp))
    return hp


def came_validate(hp: came_hparams) -> None:
    _check(load().came_validate(ctypes.byref(hp)))


def came_workspace_size(tensors, n: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().came_workspace_size(tensors, int(n), ctypes.byref(out)))
    return int(out.value)


def came_step(tensors, states, n: int, step: int, hp: came_hparams, workspace: int, workspace_bytes: int,
              stream: int) -> None:
    _check(load().came_step(tensors, states, int(n), int(step), ctypes.byref(hp), ctypes.c_void_p(workspace),
                            ctypes.c_size_t(workspace_bytes), ctypes.c_void_p(stream)))


def came_profile_enable(on: bool) -> None:
    _check(load().came_profile_enable(1 if on else 0))


def came_num_kernels() -> int:
    return int(load().came_num_kernels())


def came_kernel_name(k: int) -> str:
    return load().came_kernel_name(int(k)).decode()


def came_profile_read() -> dict:
    """{kernel name: (total ms, launches)} for the CAME events recorded since the last read."""
    nk = came_num_kernels()
    ms = (ctypes.c_double * nk)()
    launches = (ctypes.c_int64 * nk)()
    _check(load().came_profile_read(ms, launches, nk))
    return {came_kernel_name(k): (float(ms[k]), int(launches[k])) for k in range(nk)}


# ---- losses over a vocabulary (include/losses.h) ------------------------------

def loss_workspace_size(tokens: int, pairs: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(load().loss_workspace_size(int(tokens), int(pairs), ctypes.byref(out)))
    return int(out.value)


# The structs come as ctypes.Structure or packed as bytes (losses.py).  A
# second set of function objects takes both by address; pointers are ints, 0
# for NULL.
_loss_calls = {}


def _loss_call(name: str):
    f = _loss_calls.get(name)
    if f is None:
        f = load()[name]
        f.restype = ctypes.c_int
        f.argtypes = [ctypes.c_size_t if t is ctypes.c_size_t else ctypes.c_void_p for t in getattr(load(), name).argtypes]
        _loss_calls[name] = f
    return f


def _by_address(s):
    return s if s.__class__ is bytes or s is None else ctypes.byref(s)


def loss_token_logprobs(x, y, logp: int, stats: int, stream: int) -> None:
    st = _loss_call("loss_token_logprobs")(_by_address(x), _by_address(y), logp, stats, stream)
    if st:
        _check(st)


def loss_token_logprobs_backward(x, y, stats: int, grad_logp, grad, stream: int) -> None:
    st = _loss_call("loss_token_logprobs_backward")(_by_address(x), _by_address(y), stats, _by_address(grad_logp),
                                                    _by_address(grad), stream)
    if st:
        _check(st)


def loss_policy(x, y, args, grad, loss: int, logp: int, token_loss: int, workspace: int, workspace_bytes: int,
                stream: int) -> None:
    st = _loss_call("loss_policy")(_by_address(x), _by_address(y), _by_address(args), _by_address(grad), loss, logp,
                                   token_loss, workspace, workspace_bytes, stream)
    if st:
        _check(st)


def loss_preference(x, y, args, grad, loss: int, pair_loss: int, rewards: int, logp: int, workspace: int,
                    workspace_bytes: int, stream: int) -> None:
    st = _loss_call("loss_preference")(_by_address(x), _by_address(y), _by_address(args), _by_address(grad), loss,
                                       pair_loss, rewards, logp, workspace, workspace_bytes, stream)
    if st:
        _check(st)


def loss_distill(x, args, grad, loss: int, token_loss: int, workspace: int, workspace_bytes: int,
                 stream: int) -> None:
    st = _loss_call("loss_distill")(_by_address(x), _by_address(args), _by_address(grad), loss, token_loss, workspace,
                                    workspace_bytes, stream)
    if st:
        _check(st)


def loss_debug_stall_copies(on: bool) -> None:
    """Testing hook: the copies of this thread's next calls are expected but not made (see the header)."""
    load().loss_debug_stall_copies(1 if on else 0)


def loss_profile_enable(on: bool) -> None:
    _check(load().loss_profile_enable(1 if on else 0))


def loss_num_kernels() -> int:
    return int(load().loss_num_kernels())


def loss_kernel_name(k: int) -> str:
    return load().loss_kernel_name(int(k)).decode()


def loss_profile_read() -> dict:
    """{kernel name: (total ms, launches)} for the loss events recorded since the last read."""
    nk = loss_num_kernels()
    ms = (ctypes.c_double * nk)()
    launches = (ctypes.c_int64 * nk)()
    _check(load().loss_profile_read(ms, launches, nk))
    return {loss_kernel_name(k): (float(ms[k]), int(launches[k])) for k in range(nk)}


def muon_default_iteration() -> muon_iteration:
    it = muon_iteration()
    load().muon_default_iteration(ctypes.byref(it))
    return it


def muon_validate(hp: muon_hparams) -> None:
    _check(load().muon_validate(ctypes.byref(hp)))


def muon_validate_iteration(it: muon_iteration) -> None:
    _check(load().muon_validate_iteration(ctypes.byref(it)))


def muon_workspace_size(tensors, n: int) -> int:
    out = ctypes.c_size_t()
    _check(load().muon_workspace_size(tensors, n, ctypes.byref(out)))
    return int(out.value)


def muon_orthogonalize_workspace_size(batch: int, rows: int, cols: int) -> int:
    out = ctypes.c_size_t()
    _check(load().muon_orthogonalize_workspace_size(batch, rows, cols, ctypes.byref(out)))
    return int(out.value)


def muon_step(tensors, n: int, hp: muon_hparams, workspace: int, workspace_bytes: int, stream: int) -> None:
    _check(load().muon_step(tensors, n, ctypes.byref(hp), workspace, workspace_bytes, stream))


def muon_orthogonalize(x: muon_matrices, it: muon_iteration, out: int, out_dtype: int, workspace: int,
                       workspace_bytes: int, stream: int) -> None:
    _check(load().muon_orthogonalize(ctypes.byref(x), ctypes.byref(it), out, out_dtype, workspace, workspace_bytes,
                                     stream))


def muon_device_status(workspace: int, stream: int) -> int:
    out = ctypes.c_int32()
    _check(load().muon_device_status(workspace, stream, ctypes.byref(out)))
    return int(out.value)


def muon_debug_stall_copies(on: bool) -> None:
    """Testing hook: the copies of this thread's next calls are expected but not made (see the header)."""
    load().muon_debug_stall_copies(1 if on else 0)


def muon_profile_enable(on: bool) -> None:
    _check(load().muon_profile_enable(1 if on else 0))


def muon_num_kernels() -> int:
    return int(load().muon_num_kernels())


def muon_kernel_name(k: int) -> str:
    return load().muon_kernel_name(int(k)).decode()


def muon_profile_read() -> dict:
    """{kernel name: (total ms, launches)} for the Muon events recorded since the last read."""
    nk = muon_num_kernels()
    ms = (ctypes.c_double * nk)()
    launches = (ctypes.c_int64 * nk)()
    _check(load().muon_profile_read(ms, launches, nk))
    return {muon_kernel_name(k): (float(ms[k]), int(launches[k])) for k in range(nk)}


def linear_ce_workspace_size(hidden, weight, grad_hidden=None, grad_weight=None) -> int:
    out = ctypes.c_size_t()
    _check(_loss_call("linear_ce_workspace_size")(_by_address(hidden), _by_address(weight), _by_address(grad_hidden),
                                                  _by_address(grad_weight), ctypes.byref(out)))
    return int(out.value)


def linear_ce(hidden, weight, targets, args, grad_hidden, grad_weight, loss: int, logp: int, lse: int, workspace: int,
              workspace_bytes: int, stream: int) -> None:
    st = _loss_call("linear_ce")(_by_address(hidden), _by_address(weight), _by_address(targets), _by_address(args),
                                 _by_address(grad_hidden), _by_address(grad_weight), loss, logp, lse, workspace,
                                 workspace_bytes, stream)
    if st:
        _check(st)


def linear_ce_debug_stall_copies(on: bool) -> None:
    """Testing hook: the copies of this thread's next calls are expected but not made (see the header)."""
    load().linear_ce_debug_stall_copies(1 if on else 0)


def linear_ce_profile_enable(on: bool) -> None:
    _check(load().linear_ce_profile_enable(1 if on else 0))


def linear_ce_num_kernels() -> int:
    return int(load().linear_ce_num_kernels())


def linear_ce_kernel_name(k: int) -> str:
    return load().linear_ce_kernel_name(int(k)).decode()


def linear_ce_profile_read() -> dict:
    """{kernel name: (total ms, launches)} for the events of linear_ce recorded since the last read."""
    nk = linear_ce_num_kernels()
    ms = (ctypes.c_double * nk)()
    launches = (ctypes.c_int64 * nk)()
    _check(load().linear_ce_profile_read(ms, launches, nk))
    return {linear_ce_kernel_name(k): (float(ms[k]), int(launches[k])) for k in range(nk)}
