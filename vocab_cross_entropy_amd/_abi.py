"""ctypes declarations of include/ce.h (argument marshalling only).

The shared library is the one built in-tree by ``vocab_cross_entropy_amd/csrc/build.py``;
there is no fallback: if it is missing, importing this module fails.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libce.so")
# the same library with phase stamps compiled in; loaded only when
# VCE_PHASE_CLOCK=1 (bench.py --phases sets it)
PHASES_LIB_PATH = os.path.join(PKG, "libce_phases.so")

CE_OK, CE_EINVAL, CE_EDTYPE, CE_ELAYOUT, CE_EWORKSPACE, CE_EHIP, CE_EDEADLOCK = range(7)
CE_F32, CE_BF16 = 0, 1
CE_REDUCE_NONE, CE_REDUCE_MEAN, CE_REDUCE_SUM = 0, 1, 2
CE_SMOOTH_ALL, CE_SMOOTH_OTHERS = 0, 1
CE_GEMM_AUTO, CE_GEMM_NATIVE, CE_GEMM_LIBRARY = 0, 1, 2
CE_TEACHER_LOGITS, CE_TEACHER_LOGPROBS = 0, 1
CE_ABI_VERSION = 9


class CeLogits(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("d0", ctypes.c_int64),
        ("d1", ctypes.c_int64),
        ("s0", ctypes.c_int64),
        ("s1", ctypes.c_int64),
        ("v_local", ctypes.c_int64),
        ("vocab_start", ctypes.c_int64),
        ("vocab_total", ctypes.c_int64),
    ]


class CeTargets(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("s0", ctypes.c_int64), ("s1", ctypes.c_int64)]


class CeParams(ctypes.Structure):
    _fields_ = [
        ("label_smoothing", ctypes.c_float),
        ("reduce_loss", ctypes.c_int32),
        ("ignore_idx", ctypes.c_int64),
        ("split_chunks", ctypes.c_int32),
        ("smoothing", ctypes.c_int32),
    ]


class CeLinear(ctypes.Structure):
    _fields_ = [
        ("h", ctypes.c_void_p),
        ("w", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("gemm", ctypes.c_int32),
        ("N", ctypes.c_int64),
        ("D", ctypes.c_int64),
        ("V", ctypes.c_int64),
        ("h_ld", ctypes.c_int64),
        ("w_ld", ctypes.c_int64),
    ]


def _fields(spec: str):
    """"name:type ..." pairs: p pointer, q int64, i int32, f float."""
    types = {"p": ctypes.c_void_p, "q": ctypes.c_int64, "i": ctypes.c_int32, "f": ctypes.c_float}
    return [(name, types[code]) for name, code in (item.split(":") for item in spec.split())]


class CeProcess(ctypes.Structure):
    _fields_ = _fields("history:p history_s0:q history_s1:q history_max:q history_len:p prompt_len:p repetition:p "
                       "frequency:p presence:p temperature:p bias:p bias_s0:q bias_s1:q mask:p mask_s0:q mask_s1:q "
                       "signs:p signs_ld:q")


class CeEmbeddingDesc(ctypes.Structure):
    _fields_ = _fields("ids:p id_stride:q N:q D:q weight:p w_ld:q dtype:i reserved:i v_local:q vocab_start:q "
                       "vocab_total:q scale:f")


class CeNorm(ctypes.Structure):
    _fields_ = _fields("x:p residual:p weight:p dtype:i weight_dtype:i N:q D:q x_ld:q residual_ld:q eps:f")


class CeLogprobs(ctypes.Structure):
    _fields_ = _fields("ids:p ids_s0:q ids_s1:q M:i K:i ignore_idx:q")


class CeDistill(ctypes.Structure):
    _fields_ = _fields("ids:p ids_s0:q ids_s1:q values:p values_s0:q values_s1:q values_dtype:i kind:i K:i "
                       "temperature:f len:p")


# Every symbol include/ce.h declares, with its ctypes signature.
_P = ctypes.POINTER
_vp = ctypes.c_void_p
SIGNATURES = {
    "ce_workspace_bytes": (ctypes.c_size_t, [_P(CeLogits), _P(CeParams)]),
    "ce_combine_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, _P(CeParams)]),
    "ce_forward": (ctypes.c_int, [_P(CeLogits), _P(CeTargets), _P(CeParams), _vp, _vp, _vp, _vp, ctypes.c_size_t,
                                  _vp]),
    "ce_forward_ex": (ctypes.c_int, [_P(CeLogits), _P(CeTargets), _P(CeParams), _vp, _vp, _vp, _vp, _vp,
                                     ctypes.c_size_t, _vp]),
    "ce_backward_inplace": (ctypes.c_int, [_P(CeLogits), _P(CeTargets), _P(CeParams), _vp, _vp, _vp, _vp]),
    "ce_backward_inplace_ex": (ctypes.c_int, [_P(CeLogits), _P(CeTargets), _P(CeParams), _vp, _vp, _vp, _vp,
                                              _vp]),
    "ce_fwd_bwd_fused": (ctypes.c_int, [_P(CeLogits), _P(CeTargets), _P(CeParams), _vp, _vp, _vp, _vp,
                                        ctypes.c_size_t, _vp]),
    "ce_fwd_bwd_fused_noalloc": (ctypes.c_int, [_P(CeLogits), _P(CeTargets), _P(CeParams), _vp, _vp, _vp, _vp]),
    "ce_shards_workspace_bytes": (ctypes.c_size_t, [_P(CeLogits), ctypes.c_int32, _P(CeParams)]),
    "ce_shards_fwd_bwd_fused": (ctypes.c_int, [_P(CeLogits), ctypes.c_int32, _P(CeTargets), _P(CeParams), _vp, _vp,
                                               _vp, _vp, ctypes.c_size_t, _vp]),
    "ce_scale_grad_inplace": (ctypes.c_int, [_P(CeLogits), _vp, ctypes.c_int32, _vp]),
    "ce_stream_reference": (ctypes.c_int, [_vp, _vp, ctypes.c_int64, _vp]),
    "ce_shard_partial_stats": (ctypes.c_int, [_P(CeLogits), _P(CeTargets), _P(CeParams), _vp, _vp]),
    "ce_shard_combine": (ctypes.c_int, [_vp, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                        _P(CeTargets), _P(CeParams), _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "ce_shard_combine_ex": (ctypes.c_int, [_vp, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                           _P(CeTargets), _P(CeParams), _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                                           _vp]),
    "ce_workspace_init": (ctypes.c_int, [_vp, ctypes.c_size_t, _vp]),
    "ce_linear_gemm_plan": (ctypes.c_int32, [_P(CeLinear)]),
    "ce_linear_workspace_bytes": (ctypes.c_size_t, [_P(CeLinear), _P(CeParams), ctypes.c_int64,
                                                    _P(ctypes.c_int64)]),
    "ce_linear_tune": (ctypes.c_int, [_P(CeLinear), _P(CeParams), _vp, ctypes.c_int64, _vp, ctypes.c_int64,
                                      ctypes.c_int64, _vp, ctypes.c_size_t, _vp]),
    "ce_linear_cross_entropy": (ctypes.c_int, [_P(CeLinear), _vp, ctypes.c_int64, _P(CeParams), _vp, _vp, _vp, _vp,
                                               ctypes.c_int64, _vp, ctypes.c_int64, ctypes.c_int32, ctypes.c_int64,
                                               _vp, ctypes.c_size_t, _vp]),
    "ce_logits_process": (ctypes.c_int, [_P(CeLogits), _P(CeLogits), _P(CeProcess), _vp]),
    "ce_logits_process_backward": (ctypes.c_int, [_P(CeLogits), _P(CeLogits), _P(CeProcess), _vp]),
    "ce_embedding": (ctypes.c_int, [_P(CeEmbeddingDesc), _vp, ctypes.c_int64, _vp]),
    "ce_embedding_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64]),
    "ce_embedding_backward": (ctypes.c_int, [_P(CeEmbeddingDesc), _vp, ctypes.c_int64, ctypes.c_int64, _vp,
                                             ctypes.c_int64, ctypes.c_int32, _vp, ctypes.c_size_t, _vp]),
    "ce_rms_norm": (ctypes.c_int, [_P(CeNorm), _vp, ctypes.c_int64, _vp, ctypes.c_int64, _vp]),
    "ce_rms_norm_quant": (ctypes.c_int, [_P(CeNorm), _vp, ctypes.c_int64, ctypes.c_int32, _vp, _vp, ctypes.c_int64,
                                         _vp]),
    "ce_rms_norm_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "ce_rms_norm_backward": (ctypes.c_int, [_P(CeNorm), _vp, ctypes.c_int64, _vp, ctypes.c_int64, _vp,
                                            ctypes.c_int64, _vp, ctypes.c_int32, _vp, ctypes.c_size_t, _vp]),
    "ce_token_logprobs_workspace_bytes": (ctypes.c_size_t, [_P(CeLogits), ctypes.c_int32]),
    "ce_token_logprobs": (ctypes.c_int, [_P(CeLogits), _P(CeLogprobs), _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                         ctypes.c_size_t, _vp]),
    "ce_token_logprobs_backward": (ctypes.c_int, [_P(CeLogits), _P(CeLogits), _P(CeLogprobs), _vp, _vp, _vp, _vp, _vp,
                                                  _vp]),
    "ce_distill_workspace_bytes": (ctypes.c_size_t, [_P(CeLogits)]),
    "ce_distill_fwd_bwd": (ctypes.c_int, [_P(CeLogits), _P(CeLogits), _P(CeDistill), ctypes.c_int32, _vp, _vp, _vp,
                                          _vp, ctypes.c_size_t, _vp]),
    "ce_workspace_check": (ctypes.c_int, [_vp, _vp]),
    "ce_profile_start": (ctypes.c_int, [ctypes.c_int32]),
    "ce_profile_stop": (ctypes.c_int, [_vp, ctypes.c_int32, _P(ctypes.c_int32)]),
    "ce_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "ce_last_error": (ctypes.c_char_p, []),
    "ce_abi_version": (ctypes.c_int32, []),
}


def load(path: str | None = None) -> ctypes.CDLL:
    phases = path is None and os.environ.get("VCE_PHASE_CLOCK") == "1"
    if path is None:
        path = PHASES_LIB_PATH if phases else LIB_PATH
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is not built; run `python vocab_cross_entropy_amd/csrc/build.py"
            f"{' --phases' if phases else ''}` (hipcc, gfx950) first")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if phases:
        lib.ce_phase_clock.restype = ctypes.c_int
        lib.ce_phase_clock.argtypes = [ctypes.c_void_p, ctypes.c_size_t]
    if lib.ce_abi_version() != CE_ABI_VERSION:
        raise ImportError(f"{path} has ABI version {lib.ce_abi_version()}, expected {CE_ABI_VERSION}")
    return lib


class CeError(RuntimeError):
    """A non-OK ce_status; ``status`` holds the code."""

    def __init__(self, status: int, detail: str):
        super().__init__(f"{detail} [status {status}]")
        self.status = status


class CeArgumentError(CeError, ValueError):
    """Argument, dtype, layout or workspace error (nothing was enqueued)."""
