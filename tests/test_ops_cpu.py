"""Refusals of the operators around the loss, on the CPU: every bad argument is found on the host before any
HIP call (host stand-ins for device buffers, never read), and the binding refuses host tensors."""
import ctypes

import numpy as np
import pytest
import torch

import vocab_cross_entropy_amd as vce
from vocab_cross_entropy_amd import _abi

lib = _abi.load()
BUF = np.zeros(1 << 16, np.uint8)
P = (BUF.ctypes.data + 255) // 256 * 256
EINVAL, EDTYPE, ELAYOUT, EWS = _abi.CE_EINVAL, _abi.CE_EDTYPE, _abi.CE_ELAYOUT, _abi.CE_EWORKSPACE


def _set(s, kw):
    for k, v in kw.items():
        assert hasattr(s, k), k
        setattr(s, k, v)
    return s


def logits(**kw):
    return _set(_abi.CeLogits(P, _abi.CE_BF16, 0, 2, 3, 48, 16, 16, 0, 16), kw)


def _fields(s):
    return {k: getattr(s, k) for k, _ in s._fields_}


def process(x={}, out={}, p={}, backward=False, null=False):
    xd, zd = logits(**x), logits(**dict(x, **out))
    desc = _set(_abi.CeProcess(), dict(history=P, history_s0=30, history_s1=10, history_max=10, repetition=P, signs=P,
                                       signs_ld=2, mask=P, mask_s0=3, mask_s1=1) | p)
    fn = lib.ce_logits_process_backward if backward else lib.ce_logits_process
    return fn(ctypes.byref(xd), ctypes.byref(zd), None if null else ctypes.byref(desc), None)


PROCESS = [
    ("dtype", dict(x=dict(dtype=5)), EDTYPE),
    ("other_dtype", dict(out=dict(dtype=_abi.CE_F32, s0=96, s1=32)), EDTYPE),
    ("null_logits", dict(x=dict(data=None)), EINVAL),
    ("null_out", dict(out=dict(data=None)), EINVAL),
    ("null_process", dict(null=True), EINVAL),
    ("rows_overlap", dict(x=dict(s1=8)), ELAYOUT),
    ("other_shape", dict(out=dict(d1=2)), ELAYOUT),
    ("other_columns", dict(out=dict(v_local=15, vocab_total=15)), ELAYOUT),
    ("other_shard", dict(x=dict(vocab_total=99), out=dict(vocab_start=4)), ELAYOUT),
    ("in_place_other_strides", dict(out=dict(s0=64)), ELAYOUT),
    ("history_misaligned", dict(p=dict(history=P + 4)), ELAYOUT),
    ("history_negative_stride", dict(p=dict(history_s1=-1)), ELAYOUT),
    ("history_max_negative", dict(p=dict(history_max=-1)), EINVAL),
    ("history_max_large", dict(p=dict(history_max=1 << 31)), EINVAL),
    ("no_history_but_len", dict(p=dict(history=None, history_max=0, history_len=P)), EINVAL),
    ("no_history_but_prompt", dict(p=dict(history=None, history_max=0, prompt_len=P)), EINVAL),
    ("no_history_but_width", dict(p=dict(history=None)), EINVAL),
    ("penalty_without_history", dict(p=dict(history=None, history_max=0)), EINVAL),
    ("temperature_misaligned", dict(p=dict(temperature=P + 2)), ELAYOUT),
    ("mask_misaligned", dict(p=dict(mask=P + 1)), ELAYOUT),
    ("bias_misaligned", dict(p=dict(bias=P + 3)), ELAYOUT),
    ("bias_row_of_4gib", dict(x=dict(d0=1, d1=1, s0=1 << 30, s1=1 << 30, v_local=1 << 30, vocab_total=1 << 30),
                              p=dict(bias=P, signs_ld=1 << 28)), ELAYOUT),
    ("mask_negative_stride", dict(p=dict(mask_s0=-1)), ELAYOUT),
    ("bias_negative_stride", dict(p=dict(bias=P, bias_s1=-1)), ELAYOUT),
    ("signs_narrow", dict(p=dict(signs_ld=1)), ELAYOUT),
    ("backward_without_signs", dict(p=dict(signs=None), backward=True), EINVAL),
]


@pytest.mark.parametrize("change,status", [c[1:] for c in PROCESS], ids=[c[0] for c in PROCESS])
def test_process_refuses(change, status):
    assert process(**change) == status, lib.ce_last_error()
    assert lib.ce_last_error()
    if not change.get("backward") and change.get("p", {}).get("signs", 1):
        assert process(**dict(change, backward=True)) == status


def embedding(m={}, out=P, out_ld=8, backward=False, padding=-1, dw=P, dw_ld=8, accumulate=0, ws=P, ws_bytes=1 << 15,
              null=False):
    desc = _set(_abi.CeEmbeddingDesc(), dict(ids=P, id_stride=1, N=4, D=8, weight=P, w_ld=8, dtype=_abi.CE_BF16,
                                             v_local=16, vocab_total=16, scale=1.0) | m)
    d = None if null else ctypes.byref(desc)
    if backward:
        return lib.ce_embedding_backward(d, out, out_ld, padding, dw, dw_ld, accumulate, ws, ws_bytes, None)
    return lib.ce_embedding(d, out, out_ld, None)


EMBED = [
    ("null", dict(null=True), EINVAL),
    ("dtype", dict(m=dict(dtype=9)), EDTYPE),
    ("reserved", dict(m=dict(reserved=1)), EINVAL),
    ("tokens_negative", dict(m=dict(N=-1)), EINVAL),
    ("tokens_many", dict(m=dict(N=(1 << 26) + 1)), EINVAL),
    ("no_columns", dict(m=dict(D=0)), EINVAL),
    ("no_rows", dict(m=dict(v_local=0)), EINVAL),
    ("columns_many", dict(m=dict(D=1 << 31)), EINVAL),
    ("row_of_4gib", dict(m=dict(D=1 << 30, w_ld=1 << 30), out_ld=1 << 30), ELAYOUT),
    ("past_vocabulary", dict(m=dict(vocab_start=1)), ELAYOUT),
    ("null_ids", dict(m=dict(ids=None)), EINVAL),
    ("ids_misaligned", dict(m=dict(ids=P + 4)), ELAYOUT),
    ("ids_negative_stride", dict(m=dict(id_stride=-1)), ELAYOUT),
    ("null_out", dict(out=None), EINVAL),
    ("out_misaligned", dict(out=P + 1), ELAYOUT),
    ("out_narrow", dict(out_ld=7), ELAYOUT),
]
EMBED_FWD = [
    ("null_weight", dict(m=dict(weight=None)), EINVAL),
    ("weight_narrow", dict(m=dict(w_ld=7)), ELAYOUT),
]
EMBED_BWD = [
    ("null_dw", dict(dw=None), EINVAL),
    ("dw_misaligned", dict(dw=P + 2), ELAYOUT),
    ("dw_narrow", dict(dw_ld=7), ELAYOUT),
    ("accumulate", dict(accumulate=2), EINVAL),
    ("no_workspace", dict(ws=None), EWS),
    ("small_workspace", dict(ws_bytes=255), EWS),
    ("workspace_misaligned", dict(ws=P + 8), EWS),
]


@pytest.mark.parametrize("change,status", [c[1:] for c in EMBED + EMBED_FWD], ids=[c[0] for c in EMBED + EMBED_FWD])
def test_embedding_refuses(change, status):
    assert embedding(**change) == status, lib.ce_last_error()


@pytest.mark.parametrize("change,status", [c[1:] for c in EMBED + EMBED_BWD], ids=[c[0] for c in EMBED + EMBED_BWD])
def test_embedding_backward_refuses(change, status):
    assert embedding(backward=True, **change) == status, lib.ce_last_error()


def norm(m={}, form="y", y=P, y_ld=64, total=None, total_ld=0, group=0, scales=P, dsum=None, dsum_ld=0, dx=P, dx_ld=64,
         dweight=P, accumulate=0, ws=P, ws_bytes=1 << 15, null=False):
    desc = _set(_abi.CeNorm(), dict(x=P, weight=P, dtype=_abi.CE_BF16, weight_dtype=_abi.CE_F32, N=2, D=64, x_ld=64,
                                    eps=1e-6) | m)
    d = None if null else ctypes.byref(desc)
    if form == "y":
        return lib.ce_rms_norm(d, y, y_ld, total, total_ld, None)
    if form == "q":
        return lib.ce_rms_norm_quant(d, y, y_ld, group, scales, total, total_ld, None)
    return lib.ce_rms_norm_backward(d, y, y_ld, dsum, dsum_ld, dx, dx_ld, dweight, accumulate, ws, ws_bytes, None)


NORM = [
    ("null", dict(null=True), EINVAL),
    ("dtype", dict(m=dict(dtype=2)), EDTYPE),
    ("weight_dtype", dict(m=dict(weight_dtype=-1)), EDTYPE),
    ("rows_negative", dict(m=dict(N=-1)), EINVAL),
    ("rows_many", dict(m=dict(N=1 << 31)), EINVAL),
    ("no_columns", dict(m=dict(D=0)), EINVAL),
    ("columns_many", dict(m=dict(D=32769, x_ld=32769)), ELAYOUT),
    ("eps_negative", dict(m=dict(eps=-1e-6)), EINVAL),
    ("eps_nan", dict(m=dict(eps=float("nan"))), EINVAL),
    ("eps_infinite", dict(m=dict(eps=float("inf"))), EINVAL),
    ("null_x", dict(m=dict(x=None)), EINVAL),
    ("x_misaligned", dict(m=dict(x=P + 1)), ELAYOUT),
    ("x_narrow", dict(m=dict(x_ld=63)), ELAYOUT),
    ("null_weight", dict(m=dict(weight=None)), EINVAL),
    ("weight_misaligned", dict(m=dict(weight=P + 2)), ELAYOUT),
    ("null_y", dict(y=None), EINVAL),
    ("y_narrow", dict(y_ld=63), ELAYOUT),
]
NORM_FWD = [
    ("residual_narrow", dict(m=dict(residual=P, residual_ld=3)), ELAYOUT),
    ("residual_misaligned", dict(m=dict(residual=P + 1, residual_ld=64)), ELAYOUT),
    ("sum_narrow", dict(total=P, total_ld=3), ELAYOUT),
    ("sum_misaligned", dict(total=P + 1, total_ld=64), ELAYOUT),
]
NORM_QUANT = [
    ("group", dict(group=16), EINVAL),
    ("group_negative", dict(group=-1), EINVAL),
    ("null_scales", dict(scales=None), EINVAL),
    ("scales_misaligned", dict(scales=P + 2), ELAYOUT),
]
NORM_BWD = [
    ("residual", dict(m=dict(residual=P, residual_ld=64)), EINVAL),
    ("dsum_narrow", dict(dsum=P, dsum_ld=3), ELAYOUT),
    ("dx_narrow", dict(dx_ld=3), ELAYOUT),
    ("dx_misaligned", dict(dx=P + 1), ELAYOUT),
    ("dweight_misaligned", dict(dweight=P + 2), ELAYOUT),
    ("accumulate", dict(accumulate=-1), EINVAL),
    ("no_workspace", dict(ws=None), EWS),
    ("small_workspace", dict(ws_bytes=16), EWS),
    ("workspace_misaligned", dict(ws=P + 8), EWS),
]


@pytest.mark.parametrize("form,change,status", [("y", *c[1:]) for c in NORM + NORM_FWD]
                         + [("q", *c[1:]) for c in NORM + NORM_FWD + NORM_QUANT]
                         + [("grad", *c[1:]) for c in NORM + NORM_BWD],
                         ids=["y-" + c[0] for c in NORM + NORM_FWD] + ["q-" + c[0] for c in NORM + NORM_FWD + NORM_QUANT]
                         + ["grad-" + c[0] for c in NORM + NORM_BWD])
def test_norm_refuses(form, change, status):
    assert norm(form=form, **change) == status, lib.ce_last_error()


def test_workspace_sizes():
    assert vce.ce_embedding_workspace_bytes(0, 1, 1) >= 256 and vce.ce_rms_norm_workspace_bytes(0, 1) >= 256
    assert vce.ce_embedding_workspace_bytes(1 << 26, 1, (1 << 31) - 1) > 0
    # a workspace serves every smaller batch
    counts = sorted({max(0, (1 << k) + d) for k in range(18) for d in (-1, 0, 1, 7)} | {515, 1500, 3000, 65540})
    for D in (5, 600, 4096, 9000, 20000):
        for size in (lambda n: vce.ce_rms_norm_workspace_bytes(n, D), lambda n: vce.ce_embedding_workspace_bytes(n, D, 999)):
            sizes = [size(n) for n in counts]
            assert sizes == sorted(sizes)
    for call in (lambda: vce.ce_embedding_workspace_bytes(-1, 1, 1), lambda: vce.ce_embedding_workspace_bytes(1, 0, 1),
                 lambda: vce.ce_embedding_workspace_bytes((1 << 26) + 1, 1, 1),
                 lambda: vce.ce_rms_norm_workspace_bytes(1, 32769), lambda: vce.ce_rms_norm_workspace_bytes(-1, 8)):
        with pytest.raises(vce.CeArgumentError):
            call()


def test_binding_refuses_host_tensors():
    x, w, ids = torch.zeros((2, 3, 16)), torch.zeros((16, 8)), torch.zeros(4, dtype=torch.int64)
    h = torch.zeros((4, 8))
    for call in (lambda: vce.ce_logits_process(x), lambda: vce.ce_logits_process_backward(x),
                 lambda: vce.process_logits(x, temperature=torch.ones(6)), lambda: vce.ce_embedding(ids, w),
                 lambda: vce.processed_cross_entropy(x, torch.zeros((2, 3), dtype=torch.int64)),
                 lambda: vce.ce_embedding_backward(h, ids, 16), lambda: vce.embedding(ids, w),
                 lambda: vce.embedding(ids, w, grad_buffer=w), lambda: vce.ce_rms_norm(h, h[0]),
                 lambda: vce.ce_rms_norm_quant(h, h[0]), lambda: vce.ce_rms_norm_backward(h, h, h[0]),
                 lambda: vce.rms_norm(h, h[0]), lambda: vce.norm_linear_cross_entropy(h, h[0], w, ids)):
        with pytest.raises(vce.CeArgumentError):
            call()


def test_constants_of_the_processing_get_no_gradient():
    x = torch.zeros((1, 2, 16))
    for name in ("repetition", "frequency", "presence", "temperature", "bias"):
        kw = {name: torch.ones(2, requires_grad=True)}
        with pytest.raises(vce.CeArgumentError):
            vce.process_logits(x, **kw)
        with pytest.raises(vce.CeArgumentError):
            vce.processed_cross_entropy(x, None, **kw)


def test_rms_norm_refuses_another_shape():
    with pytest.raises(vce.CeArgumentError):
        vce.rms_norm(torch.zeros((4, 8)), torch.zeros(8), torch.zeros(8))


# x's rows stand at P, two of 128 bytes; Q and R are clear of them and of one another
Q, R = P + 4096, P + 8192
OVERLAP = [
    ("y_over_x_other_stride", "y", dict(y=P, y_ld=72)),
    ("y_half_a_row_on", "y", dict(y=P + 64)),
    ("y_a_row_on", "y", dict(y=P + 128)),
    ("y_a_row_back", "y", dict(m=dict(x=P + 128), y=P)),
    ("y_among_x", "y", dict(m=dict(x_ld=256), y=P + 64, y_ld=64)),
    ("y_over_residual_other_stride", "y", dict(m=dict(residual=Q, residual_ld=64), y=Q, y_ld=128)),
    ("y_into_residual", "y", dict(m=dict(residual=Q, residual_ld=100), y=Q + 126, y_ld=100)),
    ("sum_is_y", "y", dict(y=Q, total=Q, total_ld=64)),
    ("sum_and_y_in_place", "y", dict(y=P, total=P, total_ld=64)),
    ("sum_over_x_other_stride", "y", dict(y=Q, total=P, total_ld=66)),
    ("sum_into_residual", "y", dict(m=dict(residual=Q, residual_ld=64), y=R, total=Q + 2, total_ld=64)),
    ("q_over_x", "q", dict(y=P, y_ld=128)),
    ("q_over_residual", "q", dict(m=dict(residual=Q, residual_ld=64), y=Q + 100)),
    ("q_over_sum", "q", dict(y=Q + 130, y_ld=128, total=Q, total_ld=64)),
    ("q_sum_over_x_other_stride", "q", dict(y=Q, total=P, total_ld=70)),
    ("dx_over_dy_other_stride", "grad", dict(m=dict(x=Q), y=P, y_ld=64, dx=P, dx_ld=80)),
    ("dx_a_row_on_dy", "grad", dict(m=dict(x=Q), y=P, dx=P + 128)),
    ("dx_into_dsum", "grad", dict(m=dict(x=Q), y=Q, dsum=P, dsum_ld=64, dx=P + 8)),
    ("dx_over_x_other_stride", "grad", dict(m=dict(x=Q), y=P, dx=Q, dx_ld=65)),
]


@pytest.mark.parametrize("form,change", [c[1:] for c in OVERLAP], ids=[c[0] for c in OVERLAP])
def test_norm_refuses_overlaps(form, change):
    assert norm(form=form, ws=P + (1 << 15), ws_bytes=1 << 14, dweight=None, **change) == ELAYOUT, lib.ce_last_error()
    assert b"overlaps" in lib.ce_last_error()


# x's rows: (2, 3) of 32 bytes, 32 apart
PROCESS_OVERLAP = [
    ("half_a_row_on", dict(out=dict(data=P + 16))),
    ("a_row_on", dict(out=dict(data=P + 32))),
    ("a_row_back", dict(x=dict(data=P + 32), out=dict(data=P))),
    ("five_rows_on", dict(out=dict(data=P + 160))),
    ("other_stride_inside", dict(out=dict(data=P + 160, s0=96))),
    ("one_column_into_the_gap_of_rows", dict(x=dict(s0=120, s1=40), out=dict(data=P + 50))),
    ("turned", dict(out=dict(s0=16, s1=32))),
]


@pytest.mark.parametrize("change", [c[1] for c in PROCESS_OVERLAP], ids=[c[0] for c in PROCESS_OVERLAP])
@pytest.mark.parametrize("backward", [False, True])
def test_process_refuses_overlaps(change, backward):
    assert process(backward=backward, **change) == ELAYOUT, lib.ce_last_error()
    assert b"overlaps" in lib.ce_last_error()


def test_embedding_refuses_its_padding_at_the_call():
    ids, w = torch.zeros(4, dtype=torch.int64), torch.zeros((16, 8), requires_grad=True)
    with pytest.raises(vce.CeArgumentError, match="padding_idx"):
        vce.embedding(ids, w, padding_idx=-1)


def test_processing_refuses_by_its_own_error():
    """Logits of other dimensions, and numbers in place of per-row tensors, in both autograd forms."""
    x, rows = torch.zeros((2, 3, 16), requires_grad=True), torch.ones(6)
    t = torch.zeros((2, 3), dtype=torch.int64)
    for logits in (x[0], x[0, 0], x[None]):
        for call in (lambda **kw: vce.process_logits(logits, **kw), lambda **kw: vce.processed_cross_entropy(logits, t, **kw)):
            with pytest.raises(vce.CeArgumentError, match="3-d"):
                call(repetition=rows)
    for name in ("repetition", "frequency", "presence", "temperature", "bias"):
        for call in (lambda **kw: vce.process_logits(x, **kw), lambda **kw: vce.processed_cross_entropy(x, t, **kw)):
            with pytest.raises(vce.CeArgumentError):
                call(**{name: 0.7})
