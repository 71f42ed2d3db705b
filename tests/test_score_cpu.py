"""Refusals of token log-probabilities and distillation, on the CPU: every bad argument is found on the host before
any HIP call (host stand-ins for device buffers, never read), the binding refuses host tensors, and the 64-bit
definitions that the GPU tests compare with agree with torch's autograd."""
import ctypes
import math

import numpy as np
import pytest
import torch

import vocab_cross_entropy_amd as vce
from score_util import Row64, largest, ref_distill, ref_logprobs_grad
from vocab_cross_entropy_amd import _abi

lib = _abi.load()
BUF = np.zeros(1 << 16, np.uint8)
P = (BUF.ctypes.data + 255) // 256 * 256
EINVAL, EDTYPE, ELAYOUT, EWS = _abi.CE_EINVAL, _abi.CE_EDTYPE, _abi.CE_ELAYOUT, _abi.CE_EWORKSPACE
FAR = P + (1 << 15)  # past the 288 bytes of the logits below
BIG = dict(d0=1, d1=2, s0=1 << 21, s1=1 << 20, v_local=100000, vocab_total=100000)  # more than one chunk


def _set(s, kw):
    for k, v in kw.items():
        assert hasattr(s, k), k
        setattr(s, k, v)
    return s


def logits(**kw):
    return _set(_abi.CeLogits(P, _abi.CE_BF16, 0, 2, 3, 48, 16, 16, 0, 16), kw)


def logprobs(x={}, q={}, logp=P, entropy=P, lse=P, top_ids=P, top_logp=P, stats=P, ws=P, ws_bytes=1 << 15, null=""):
    desc = _set(_abi.CeLogprobs(P, 6, 2, 2, 3, -100), q)
    return lib.ce_token_logprobs(None if null == "x" else ctypes.byref(logits(**x)), None if null == "q" else ctypes.byref(desc),
                                 logp, entropy, lse, top_ids, top_logp, stats, ws, ws_bytes, None)


def logprobs_bwd(x={}, out={}, q={}, stats=P, dlogp=P, dentropy=P, top_ids=P, dtop=P, null=""):
    desc = _set(_abi.CeLogprobs(P, 6, 2, 2, 3, -100), q)
    return lib.ce_token_logprobs_backward(ctypes.byref(logits(**x)), None if null == "out" else ctypes.byref(logits(**dict(x, **out))),
                                          None if null == "q" else ctypes.byref(desc), stats, dlogp, dentropy, top_ids, dtop, None)


BOTH = [
    ("dtype", dict(x=dict(dtype=7)), EDTYPE),
    ("null_logits", dict(x=dict(data=None)), EINVAL),
    ("reserved", dict(x=dict(reserved=1)), EINVAL),
    ("logits_misaligned", dict(x=dict(data=P + 1)), ELAYOUT),
    ("rows_overlap", dict(x=dict(s1=8)), ELAYOUT),
    ("negative_stride", dict(x=dict(s0=-48)), ELAYOUT),
    ("a_shard", dict(x=dict(vocab_total=32)), ELAYOUT),
    ("a_later_shard", dict(x=dict(vocab_start=16, vocab_total=32)), ELAYOUT),
    ("rows_too_long", dict(x=dict(d0=1, d1=1, s0=0, s1=0, v_local=(1 << 20) + 1, vocab_total=(1 << 20) + 1)), ELAYOUT),
    ("rows_too_long_f32", dict(x=dict(dtype=_abi.CE_F32, d0=1, d1=1, v_local=(1 << 19) + 1, vocab_total=(1 << 19) + 1)), ELAYOUT),
    ("null_descriptor", dict(null="q"), EINVAL),
    ("tokens_negative", dict(q=dict(M=-1)), EINVAL),
    ("tokens_many", dict(q=dict(M=129)), EINVAL),
    ("alternatives_negative", dict(q=dict(K=-1)), EINVAL),
    ("alternatives_many", dict(x=dict(d0=1, d1=1, v_local=1000, vocab_total=1000), q=dict(K=129)), EINVAL),
    ("alternatives_above_columns", dict(q=dict(K=17)), EINVAL),
    ("null_ids", dict(q=dict(ids=None)), EINVAL),
    ("ids_misaligned", dict(q=dict(ids=P + 4)), ELAYOUT),
    ("ids_negative_stride", dict(q=dict(ids_s1=-2)), ELAYOUT),
    ("null_top_ids", dict(top_ids=None), EINVAL),
    ("top_ids_misaligned", dict(top_ids=P + 4), ELAYOUT),
    ("stats_misaligned", dict(stats=P + 8), ELAYOUT),
]
FORWARD = [
    ("null_x", dict(null="x"), EINVAL),
    ("null_logp", dict(logp=None), EINVAL),
    ("null_top_logp", dict(top_logp=None), EINVAL),
    ("logp_misaligned", dict(logp=P + 2), ELAYOUT),
    ("entropy_misaligned", dict(entropy=P + 2), ELAYOUT),
    ("lse_misaligned", dict(lse=P + 1), ELAYOUT),
    ("top_logp_misaligned", dict(top_logp=P + 2), ELAYOUT),
    ("no_workspace", dict(x=BIG, ws=None), EWS),
    ("small_workspace", dict(x=BIG, ws_bytes=300), EWS),
    ("workspace_misaligned", dict(x=BIG, ws=P + 64), EWS),
]
BACKWARD = [
    ("null_out", dict(null="out"), EINVAL),
    ("null_out_data", dict(out=dict(data=None)), EINVAL),
    ("other_dtype", dict(out=dict(data=FAR, dtype=_abi.CE_F32)), EDTYPE),
    ("other_shape", dict(out=dict(data=FAR, d1=2)), ELAYOUT),
    ("other_columns", dict(out=dict(data=FAR, v_local=15, vocab_total=15)), ELAYOUT),
    ("in_place_other_strides", dict(out=dict(s0=64)), ELAYOUT),
    ("half_a_row_off", dict(out=dict(data=P + 16)), ELAYOUT),
    ("null_stats", dict(stats=None), EINVAL),
    ("null_dlogp", dict(dlogp=None), EINVAL),
    ("null_dtop", dict(dtop=None), EINVAL),
    ("dlogp_misaligned", dict(dlogp=P + 2), ELAYOUT),
    ("dentropy_misaligned", dict(dentropy=P + 2), ELAYOUT),
    ("dtop_misaligned", dict(dtop=P + 3), ELAYOUT),
]


@pytest.mark.parametrize("change,status", [c[1:] for c in BOTH + FORWARD], ids=[c[0] for c in BOTH + FORWARD])
def test_logprobs_refuses(change, status):
    assert logprobs(**change) == status, lib.ce_last_error()
    assert lib.ce_last_error()


@pytest.mark.parametrize("change,status", [c[1:] for c in BOTH + BACKWARD], ids=[c[0] for c in BOTH + BACKWARD])
def test_logprobs_gradient_refuses(change, status):
    assert logprobs_bwd(**change) == status, lib.ce_last_error()


def distill(x={}, out={}, d={}, reduce=0, g=None, loss=P, n=None, ws=P, ws_bytes=1 << 15, null=""):
    desc = _set(_abi.CeDistill(P, 12, 4, P, 12, 4, _abi.CE_F32, 0, 4, 1.0, None), d)
    return lib.ce_distill_fwd_bwd(None if null == "x" else ctypes.byref(logits(**x)),
                                  None if null == "out" else ctypes.byref(logits(**dict(x, **out))),
                                  None if null == "d" else ctypes.byref(desc), reduce, g, loss, n, ws, ws_bytes, None)


DISTILL = [c for c in BOTH if set(c[1]) == {"x"} and "too_long" not in c[0] and "alternatives" not in c[0]] + [
    ("null_x", dict(null="x"), EINVAL),
    ("rows_too_long", dict(x=dict(d0=1, d1=1, v_local=(1 << 21) + 1, vocab_total=(1 << 21) + 1)), ELAYOUT),
    ("null_descriptor", dict(null="d"), EINVAL),
    ("other_dtype", dict(out=dict(data=FAR, dtype=_abi.CE_F32)), EDTYPE),
    ("other_shape", dict(out=dict(data=FAR, d0=1)), ELAYOUT),
    ("in_place_other_strides", dict(out=dict(s0=64)), ELAYOUT),
    ("overlap", dict(out=dict(data=P + 32)), ELAYOUT),
    ("no_entries", dict(d=dict(K=0)), EINVAL),
    ("many_entries", dict(d=dict(K=129)), EINVAL),
    ("values_dtype", dict(d=dict(values_dtype=4)), EDTYPE),
    ("kind", dict(d=dict(kind=2)), EINVAL),
    ("temperature_zero", dict(d=dict(temperature=0.0)), EINVAL),
    ("temperature_negative", dict(d=dict(temperature=-1.0)), EINVAL),
    ("temperature_nan", dict(d=dict(temperature=math.nan)), EINVAL),
    ("temperature_large", dict(d=dict(temperature=2.0 ** 33)), EINVAL),
    ("null_ids", dict(d=dict(ids=None)), EINVAL),
    ("null_values", dict(d=dict(values=None)), EINVAL),
    ("ids_misaligned", dict(d=dict(ids=P + 4)), ELAYOUT),
    ("ids_negative_stride", dict(d=dict(ids_s0=-1)), ELAYOUT),
    ("values_misaligned", dict(d=dict(values=P + 2)), ELAYOUT),
    ("values_negative_stride", dict(d=dict(values_s1=-4)), ELAYOUT),
    ("len_misaligned", dict(d=dict(len=P + 2)), ELAYOUT),
    ("reduction", dict(reduce=3), EINVAL),
    ("null_loss", dict(loss=None), EINVAL),
    ("loss_misaligned", dict(loss=P + 2), ELAYOUT),
    ("upstream_misaligned", dict(g=P + 1), ELAYOUT),
    ("count_misaligned", dict(n=P + 2), ELAYOUT),
    ("no_workspace", dict(ws=None), EWS),
    ("small_workspace", dict(ws_bytes=256), EWS),
    ("small_workspace_chunks", dict(x=BIG, ws_bytes=300), EWS),
    ("workspace_misaligned", dict(ws=P + 128), EWS),
]


@pytest.mark.parametrize("change,status", [c[1:] for c in DISTILL], ids=[c[0] for c in DISTILL])
def test_distill_refuses(change, status):
    assert distill(**change) == status, lib.ce_last_error()


def test_no_rows_are_checked_and_launch_nothing():
    assert logprobs(x=dict(d0=0, data=None), q=dict(ids=None), logp=None, top_ids=None, top_logp=None) == 0
    assert logprobs_bwd(x=dict(d0=0, data=None), q=dict(ids=None), stats=None, dlogp=None, top_ids=None, dtop=None) == 0
    assert distill(x=dict(d0=0, data=None), d=dict(ids=None, values=None), loss=None) == 0
    assert logprobs(q=dict(ids=None, M=0, K=0), logp=None, entropy=None, lse=None, top_ids=None, top_logp=None, stats=None) == 0


def test_workspace_sizes():
    x = logits()
    assert lib.ce_token_logprobs_workspace_bytes(ctypes.byref(x), 3) == 256
    assert lib.ce_distill_workspace_bytes(ctypes.byref(x)) == 512  # a header and a word a row
    big = logits(**BIG)
    none, most = (lib.ce_token_logprobs_workspace_bytes(ctypes.byref(big), k) for k in (0, 128))
    assert 256 < none < most and most % 256 == 0
    for bad in (logits(dtype=3), logits(vocab_total=17), logits(v_local=1 << 22, vocab_total=1 << 22, d0=1, d1=1)):
        assert lib.ce_token_logprobs_workspace_bytes(ctypes.byref(bad), 0) == 0
        assert lib.ce_distill_workspace_bytes(ctypes.byref(bad)) == 0
    assert lib.ce_token_logprobs_workspace_bytes(ctypes.byref(x), 17) == 0
    assert lib.ce_token_logprobs_workspace_bytes(None, 1) == 0 and lib.ce_distill_workspace_bytes(None) == 0


def test_binding_refuses_host_tensors():
    x, ids = torch.zeros(1, 2, 50), torch.zeros(1, 2, dtype=torch.int64)
    t = torch.zeros(1, 2, 3)
    for call in (lambda: vce.ce_token_logprobs(x, ids), lambda: vce.token_logprobs(x, ids, top_k=2),
                 lambda: vce.ce_token_logprobs_backward(x, torch.zeros(2, 4), ids, torch.zeros(1, 2)),
                 lambda: vce.ce_distill_fwd_bwd(x, ids.view(1, 2, 1).expand(1, 2, 3), t),
                 lambda: vce.distillation_loss(x, ids.view(1, 2, 1).expand(1, 2, 3), t), lambda: vce.ce_token_logprobs(None)):
        with pytest.raises(vce.CeArgumentError):
            call()
    with pytest.raises(vce.CeArgumentError):
        vce.token_logprobs(x)


def test_definitions_agree_with_autograd():
    """The 64-bit definitions of score_util against torch's gradients, and their budgets are small."""
    g = torch.Generator().manual_seed(3)
    N, V, M, K = 5, 61, 4, 7
    x = (torch.randn((N, V), generator=g, dtype=torch.float64) * 3).requires_grad_()
    ids = torch.randint(0, V, (N, M), generator=g)
    ids[:, 3] = ids[:, 0]
    w, wh = torch.randn((N, M), generator=g, dtype=torch.float64), torch.randn(N, generator=g, dtype=torch.float64)
    lp = torch.log_softmax(x, 1)
    h = -(lp.exp() * lp).sum(1)
    ((lp.gather(1, ids) * w).sum() + (h * wh).sum()).backward()
    r = Row64(x.detach().numpy())
    ref, tol = r.logp(ids.numpy())
    assert np.allclose(ref, lp.gather(1, ids).detach().numpy(), rtol=1e-12, atol=1e-13) and tol.max() < 1e-4
    assert np.allclose(r.H, h.detach().numpy(), rtol=1e-11, atol=1e-13) and r.tol_H.max() < 1e-4
    dx, tol = ref_logprobs_grad(x.detach().numpy(), ids.numpy(), w.numpy(), wh.numpy())
    assert np.allclose(dx, x.grad.numpy(), rtol=1e-10, atol=1e-12) and tol.max() < 1e-3
    assert np.array_equal(largest(np.array([[1.0, np.nan, 3.0, -0.0, 0.0, 3.0, -np.inf]]), 7), [[2, 5, 0, 3, 4, 6, 1]])

    cols = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)])
    cols[0, 1] = cols[0, 0]
    tv = torch.randn((N, K), generator=g, dtype=torch.float64)
    n = np.array([7, 3, 0, 1, 5])
    for tail in (False, True):
        t = torch.log_softmax(tv, 1) - 0.3 if tail else tv
        T, z = 1.7, x.detach().clone().requires_grad_()
        total = 0.0
        for i in range(N):
            if n[i] == 0:
                continue
            c, v = cols[i, :n[i]], t[i, :n[i]]
            lq = torch.log_softmax(z[i] / T, 0)
            lt = v if tail else torch.log_softmax(v / T, 0)
            row = (lt.exp() * (lt - lq[c])).sum()
            if tail:
                left = 1 - lt.exp().sum()
                other = torch.ones(V, dtype=torch.bool)
                other[c] = False
                row = row + left * (left.log() - lq[other].logsumexp(0))
            total = total + T * T * row * (i + 1)
        total.backward()
        l, _, dx, tol = ref_distill(x.detach().numpy(), cols.numpy(), t.numpy(), n, T, tail, np.arange(1, N + 1.0))
        assert abs((l * np.arange(1, N + 1)).sum() - total.item()) < 1e-10
        assert np.allclose(dx, z.grad.numpy(), rtol=1e-9, atol=1e-11) and tol.max() < 1e-3
