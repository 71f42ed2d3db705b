"""64-bit definitions of the operators around the loss, on the CPU, and the error budgets their tests use.

U is half a step of FP32 relative to the value (2^-24); a budget counts the roundings a kernel makes, each at
most U of the value it rounds, and adds half a step of the output's type.
"""
import numpy as np
import torch

U = 2.0 ** -24
TINY = 2.0 ** -126  # below the normal range roundings are absolute


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def history_counts(history, history_len, prompt_len, N, V, vocab_start=0):
    """(seen [N, V], occurrences in the output [N, V]) from a [N, L] array of tokens."""
    seen, cnt = np.zeros((N, V), bool), np.zeros((N, V), np.int64)
    if history is None:
        return seen, cnt
    L = history.shape[1]
    for r in range(N):
        n = L if history_len is None else min(max(int(history_len[r]), 0), L)
        p = 0 if prompt_len is None else int(prompt_len[r])
        for i in range(n):
            j = int(history[r, i]) - vocab_start
            if 0 <= j < V:
                seen[r, j] = True
                cnt[r, j] += i >= p
    return seen, cnt


def allowed_columns(mask, V):
    """[N, V] truth values of [N, words] int32 masks."""
    words = np.asarray(mask).astype(np.int64) & 0xffffffff
    j = np.arange(V)
    return ((words[:, j // 32] >> (j % 32)) & 1) != 0


def ref_process(x, seen, cnt, repetition, frequency, presence, bias, temperature, allowed):
    """(z, budget of the FP32 steps) for [N, V] float64 logits.  Steps: the penalty's division or product, the
    frequency's fused multiply-add, the presence's subtraction and the bias' addition round a value of at most
    `size`; 1 / temperature and its product round z twice more."""
    N, V = x.shape

    def col(v, default):
        return np.full((N, 1), default) if v is None else np.asarray(v, np.float64).reshape(N, 1)

    th, f, p, T = col(repetition, 1.0), col(frequency, 0.0), col(presence, 0.0), col(temperature, 1.0)
    with np.errstate(invalid="ignore", over="ignore"):
        v = np.where(seen, np.where(x > 0, x / th, x * th), x)
        size = np.abs(v) + np.abs(f) * cnt + np.abs(p) * (cnt > 0)
        v = v - f * cnt - p * (cnt > 0)
        if bias is not None:
            v = v + bias
            size = size + np.abs(bias)
        z = v / T
        budget = 1.01 * U * (4 * size / T + 3 * np.abs(z)) + TINY
    if allowed is not None:
        z = np.where(allowed, z, -np.inf)
    return z, budget


def ref_process_grad(dz, up, seen, repetition, temperature, allowed):
    N, V = dz.shape
    th = np.ones((N, 1)) if repetition is None else np.asarray(repetition, np.float64).reshape(N, 1)
    T = np.ones((N, 1)) if temperature is None else np.asarray(temperature, np.float64).reshape(N, 1)
    dx = np.where(seen, np.where(up, dz / th, dz * th), dz) / T
    return dx if allowed is None else np.where(allowed, dx, 0.0)


def ref_norm(x, residual, w, eps):
    s = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    return s * rstd * w, s, rstd


# Relative error of 1 / rms in units of U: a thread adds at most 32 squares, a wave 6 levels and a workgroup up to
# 16 waves (54 additions; the sum's error counts half), the sum's own terms carry 2 U each, then the mean, the eps,
# the square root and the division.
NORM_RSTD = (54 + 2) / 2 + 4


def ref_norm_grad(dy, s, w, eps, dsum):
    """(dx, dw, budgets of both in FP32 steps)."""
    N, D = s.shape
    rstd = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    gw = dy * w
    dot, adot = (gw * s).sum(1, keepdims=True), np.abs(gw * s).sum(1, keepdims=True)
    k = rstd ** 3 * dot / D
    dx = rstd * gw - s * k
    bx = U * ((NORM_RSTD + 3) * rstd * np.abs(gw) + np.abs(s) * rstd ** 3 / D
              * ((54 + 2) * adot + (3 * NORM_RSTD + 6) * np.abs(dot)) + 2 * (np.abs(rstd * gw) + np.abs(s * k)))
    if dsum is not None:
        dx = dx + dsum
        bx = bx + U * np.abs(dx)
    terms = dy * s * rstd
    dw = terms.sum(0)
    bw = 1.01 * U * (N + NORM_RSTD + 20) * np.abs(terms).sum(0) + TINY
    return dx, dw, 1.01 * bx + TINY, bw


def ref_embed_grad(dout, ids, V, scale, padding_idx=None, vocab_start=0):
    """(dw, sum of the absolute terms, tokens per row)."""
    dw, size, m = np.zeros((V, dout.shape[1])), np.zeros((V, dout.shape[1])), np.zeros((V, 1))
    for n, i in enumerate(ids):
        j = int(i) - vocab_start
        if 0 <= j < V and i != padding_idx:
            dw[j] += dout[n]
            size[j] += np.abs(dout[n])
            m[j] += 1
    return dw * scale, size * abs(scale), m


def assert_within(got, ref, tol, what):
    """|got - ref| <= tol elementwise; infinities and NaN in the same places."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    tol = np.broadcast_to(tol, ref.shape)
    fine = np.isfinite(ref)
    same = (np.isnan(got) == np.isnan(ref)) & (fine | np.isnan(ref) | (got == ref))
    with np.errstate(invalid="ignore"):
        bad = ~same | (fine & ~(np.abs(got - ref) <= tol))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} elements off, first at {i}: got {got[i]!r}, "
                             f"reference {ref[i]!r}, allowed {tol[i]!r}")
