"""Distillation where the student is near its teacher: the loss and the named columns' gradient are small differences of
terms near 1, which 64 bits hold.  The definition here is in extended precision."""
import numpy as np
import pytest
import torch

import vocab_cross_entropy_amd as vce
from gpu_util import say
from ops_util import assert_within
from score_util import U, f64, half_step, ref_distill

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAMES = {BF16: "bf16", F32: "f32"}
U64, TINY = 2.0 ** -53, 2.0 ** -126
L = np.longdouble


def _ref(x, cols, t, T, logprobs, dtype):
    """(loss, budget, gradient of the named columns, budget, slack of the unnamed ones) of one row with distinct columns.

    The unnamed columns' sum is FP32: a thread adds up to 32 columns, twice, then 6 levels of a wave, 8 waves and 6
    levels of chunks, with weights; below 64 additions of U each, and an exponent rounded four times (4 U of a column's
    distance from their largest).  It moves the loss by |S q_o - r| of that, and by its square.  All else is 64-bit: z,
    p, their products and the logarithms are rounded fewer than 16 times, each U64 of the value."""
    x, t, T = x.astype(L), t.astype(L), L(np.float32(T))
    z = x / T
    m = z.max()
    named = np.zeros(len(x), bool)
    named[cols] = True
    e = np.exp(z - m)
    D = e.sum()
    logD = np.log(D)
    if logprobs:
        lt = t
    else:
        lt = t / T - (t / T).max()
        lt = lt - np.log(np.exp(lt).sum())
    p = np.exp(lt)
    q = e[cols] / D
    q_o = e[~named].sum() / D
    r = max(L(0), 1 - p.sum()) if logprobs and q_o > 0 else L(0)
    S = p.sum() + r if logprobs else L(1)
    lq = (z[cols] - m) - logD
    loss = (p * (lt - lq)).sum()
    rel = L(0)
    if q_o > 0:
        zo = z[~named]
        eo = np.exp(zo - zo.max())
        rel = U * (64 + 4 * (np.where(eo > 0, eo * (zo.max() - np.where(eo > 0, zo, zo.max())), 0).sum() / eo.sum()))
        if r > 0:
            loss = loss + r * (np.log(r) - np.log(q_o))
    size = np.abs(lt) + np.abs(z[cols] - m) + logD + 4
    tl = T * T * (abs(S * q_o - r) * rel + rel * rel * (q_o + r) + 16 * U64 * ((p * size).sum() + r * (abs(np.log(q_o)) + 4 if r > 0 else 0)))
    loss = loss * T * T
    dx = T * (q * S - p)
    tol = T * (q * S * (16 * U64 * size + q_o * rel) + p * 16 * U64 * size)
    # what the teacher leaves is 1 less a sum of 64 bits, on either side; the unnamed columns share it
    left = np.where(named, 0, T * e / D / q_o * 32 * U64 * (p * size).sum()) if r > 0 else np.zeros(len(x))
    return (float(loss), float(tl + 1.01 * U * (abs(loss) + tl) + TINY), dx.astype(np.float64),
            (tol + 1.01 * half_step(dtype) * (np.abs(dx) + tol) + TINY).astype(np.float64), left.astype(np.float64))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("V", [700, 5001, 70001])
@pytest.mark.parametrize("T", [1.25, 0.7, 3.0])
@pytest.mark.parametrize("kind", ["logits", "logprobs"])
def test_students_near_the_teacher(kind, T, V, dtype):
    K, g = 64, torch.Generator().manual_seed(V)
    tail = kind == "logprobs"
    rows = []  # (student, columns, teacher)
    for apart in (0.0, 1e-5, 1e-4, 1e-3, 1e-2):
        for elsewhere in (-float("inf"), -40.0, -8.0):
            cols = torch.randperm(V, generator=g)[:K]
            t = (torch.randn((K,), generator=g) * 3 + 5).to(dtype).float()
            x = torch.full((V,), elsewhere) + (torch.randn((V,), generator=g) if elsewhere > -1e9 else 0.0)
            near = (t + apart * torch.randn((K,), generator=g)).to(dtype).float()
            if dtype is BF16 and apart > 0:  # a step of BF16 in a few columns
                near = t.clone()
                near[:5] = (near[:5] * (1 + 2.0 ** -7)).to(dtype).float()
            x[cols] = near
            x = x.to(dtype)
            if tail:  # the student's own log-probabilities but for `apart`
                t = (torch.log_softmax(x.double() / T, 0)[cols] + apart * torch.randn((K,), generator=g) - 1e-9).float()
            rows.append((x, cols, t))
    N = len(rows)
    x = torch.stack([r[0] for r in rows]).view(N, 1, V)
    ids, t = torch.stack([r[1] for r in rows]).view(N, 1, K), torch.stack([r[2] for r in rows]).view(N, 1, K)
    say(f"distillation near the teacher {NAMES[dtype]} V{V} T{T} {kind}")
    out = torch.empty_like(x, device="cuda")
    loss, _ = vce.ce_distill_fwd_bwd(x.cuda(), ids.cuda(), t.cuda(), T, teacher=kind, out=out)
    got, have = f64(out).reshape(N, V), f64(loss)
    _, _, all_dx, all_tol = ref_distill(f64(x).reshape(N, V), ids.view(N, K).numpy(), f64(t).reshape(N, K), np.full(N, K),
                                        float(np.float32(T)), tail, np.ones(N), dtype)
    for n, (xr, cols, tr) in enumerate(rows):
        l, tl, dx, tol, left = _ref(f64(xr), cols.numpy(), f64(tr), T, tail, dtype)
        assert_within(got[n], all_dx[n], all_tol[n] + 1.01 * left, f"row {n}: dx")
        assert_within(have[n:n + 1], np.array([l]), np.array([tl]), f"row {n}: loss")
        assert_within(got[n][cols.numpy()], dx, tol, f"row {n}: named columns")
