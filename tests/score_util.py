"""64-bit definitions of token log-probabilities and distillation, on the CPU, with the error budgets their tests use.

U is half a step of FP32 relative to the value (2^-24).  The kernels' FP32 steps, counted:
- an exponential's argument is one fused multiply-add: it rounds (x - ref) log2 e once, FP32's log2 e is off by
  less than U relative, and a chunk's maximum is weighted against the row's by two more such steps; the hardware's
  exp2 is within 2 U.  A term exp(-y) so carries U (4 y + 2), in sums the mean of that over the terms;
- sums add 8 columns in pairs, up to 8 vectors, 6 levels of a wave, up to 8 waves and 6 levels of chunks: below 36
  additions, each U of the sum; with the shift's correction and the terms' conversions 40 U are taken.
Outputs add half a step of their own type.
"""
import math

import numpy as np
import torch

U = 2.0 ** -24
TINY = 2.0 ** -126


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def _softmax_parts(z):
    """(m, exp(z - m), their sum without one column at the maximum, that with it) of float64 rows."""
    with np.errstate(invalid="ignore", over="ignore"):
        m = z.max(1, keepdims=True)
        e = np.exp(z - m)
        rest = e.copy()
        rest[np.arange(len(z)), z.argmax(1)] = 0.0
        rest = rest.sum(1)
    return m[:, 0], e, rest, 1.0 + rest


def _weighted(e, y):
    """sum of e y without the terms of e = 0."""
    with np.errstate(invalid="ignore"):
        return np.where(e > 0, e * y, 0.0).sum(1)


def largest(x, K):
    """The K columns of the largest values of each row: NaN last, equal ones by the lower column."""
    key = np.where(np.isnan(x), -np.inf, x)
    out = np.empty((len(x), K), np.int64)
    for r, row in enumerate(x):
        out[r] = np.lexsort((np.arange(row.size), -key[r], np.isnan(row)))[:K]
    return out


class Row64:
    """softmax statistics of float64 rows, with budgets: log D, entropy, lse."""

    def __init__(self, x):
        self.x = x
        self.m, e, rest, D = _softmax_parts(x)
        self.ok = np.isfinite(self.m) & ~np.isnan(x).any(1)
        with np.errstate(invalid="ignore", divide="ignore"):
            y = self.m[:, None] - x
            self.p = e / D[:, None]
            self.logd = np.log1p(rest)
            self.S = _weighted(e, y) / D
            self.H = self.logd + self.S
            self.lse = self.m + self.logd
            far = np.where(rest > 0, _weighted(e, y) / np.maximum(rest, 1e-300), 0.0)
            self.rel = U * (40 + 2 + 4 * far)         # of the rest's sum
            self.tol_logd = self.rel * rest / D + 2 * U * self.logd + TINY
            far2 = _weighted(e, y * y) / D
            self.tol_H = self.tol_logd + U * (46 * self.S + 4 * far2) + self.rel * self.S + 3 * U * self.H
        self.rest, self.D = rest, D
        for a in (self.logd, self.H):
            a[~self.ok] = np.nan
        with np.errstate(invalid="ignore"):
            self.lse = np.where(np.isneginf(self.m) & ~np.isnan(x).any(1), -np.inf, np.where(self.ok, self.lse, np.nan))

    def logp(self, ids, ignore_idx=-100):
        """(log-probabilities of [N, M] ids, budget)"""
        V = self.x.shape[1]
        inside = (ids >= 0) & (ids < V)
        xt = np.take_along_axis(self.x, np.where(inside, ids, 0), 1)
        with np.errstate(invalid="ignore"):
            d = xt - self.m[:, None]
            lp = d - self.logd[:, None]
            tol = np.where(np.isfinite(d), self.tol_logd[:, None] + 1.01 * U * (np.abs(d) + np.abs(lp)), 0.0) + TINY
        lp = np.where(inside & self.ok[:, None], lp, np.nan)
        # the outputs are FP32: what rounds past its largest number, (2 - 2^-23) 2^127, is an infinity there
        lp = np.where(lp <= -(2 - 2.0 ** -24) * 2.0 ** 127, -np.inf, lp)
        return np.where(ids == ignore_idx, 0.0, lp), tol


def ref_logprobs_grad(x, ids, g, dh, ignore_idx=-100, dtype=torch.float32):
    """(dx, budget) of float64 rows x for [N, L] ids (all lists together) with gradients g and [N] dh or None."""
    N, V = x.shape
    r = Row64(x)
    dx, tol = np.zeros((N, V)), np.zeros((N, V))
    for n in range(N):
        counts = ids[n] != ignore_idx
        if not r.ok[n] or (counts & ((ids[n] < 0) | (ids[n] >= V))).any():
            dx[n], tol[n] = np.nan, 0.0
            continue
        gn, idn = g[n][counts], ids[n][counts]
        G, absG = gn.sum(), np.abs(gn).sum()
        with np.errstate(divide="ignore", invalid="ignore"):
            lp = x[n] - r.m[n] - r.logd[n]
            h = 0.0 if dh is None else dh[n]
            y = np.where(np.isfinite(lp), np.abs(lp), 0.0)
            bend = np.where(r.p[n] > 0, h * (lp + r.H[n]), 0.0)
        own, abs_own = np.zeros(V), np.zeros(V)
        np.add.at(own, idn, gn)
        np.add.at(abs_own, idn, np.abs(gn))
        slope = G + bend
        dx[n] = own - r.p[n] * slope
        # p: its exponent's two steps, the stats' rounding of log D and (BF16) of c = lse log2 e, exp2
        rel_p = U * (4 * y + 2 * r.logd[n] + 4 + (2 * abs(r.lse[n]) if dtype == torch.bfloat16 else 0)) + r.tol_logd[n]
        size = absG + abs(h) * (y + abs(r.H[n]))
        terms = U * (len(idn) + 6) * absG + abs(h) * (U * 8 * (y + abs(r.H[n])) + r.tol_H[n] + 2 * r.tol_logd[n])
        # at a given token own (1 - p) - p (G - own + ...): 1 - p carries p's error, and roundings of what is added
        tol[n] = (r.p[n] * (size * (rel_p + 6 * U) + terms) + abs_own * np.minimum(r.p[n], 1 - r.p[n] + 4 * U)
                  * (rel_p + 4 * U) + U * (len(idn) + 6) * abs_own * (1 - r.p[n]) + 4 * U * np.abs(dx[n]) + TINY)
        tol[n] = 1.02 * tol[n] + half_step(dtype) * (np.abs(dx[n]) + tol[n])
    return dx, tol


def ref_distill(x, ids, t, n_entries, T, logprobs, scale, dtype=torch.float32):
    """(loss per row, budget, dx, budget) of float64 rows for [N, K] columns and teacher values, the first n_entries[n]
    of a row; scale [N] multiplies the gradient."""
    N, V = x.shape
    loss, tl, dx, tol = np.zeros(N), np.zeros(N), np.zeros((N, V)), np.zeros((N, V))
    for n in range(N):
        L = int(n_entries[n])
        if L == 0:
            continue
        c, tv = ids[n, :L], t[n, :L]
        z = x[n] / T
        with np.errstate(all="ignore"):
            bad = ((c < 0) | (c >= V)).any() or not np.isfinite(z.max()) or np.isnan(z).any() or np.isnan(tv).any()
            if logprobs:
                lt = tv
            else:
                top = (tv / T).max()
                lt = tv / T - top
                lt = lt - math.log(np.exp(lt).sum()) if np.isfinite(top) else np.full(L, np.nan)
            p = np.exp(lt)
        if bad or np.isnan(p).any():
            loss[n], dx[n] = np.nan, np.nan
            continue
        named = np.zeros(V, bool)
        named[c] = True
        m = z.max()
        e = np.exp(z - m)
        D = e.sum()
        logD = math.log(D)
        lse = m + logD
        q = e / D
        q_o = q[~named].sum()
        r = max(0.0, 1.0 - p.sum()) if logprobs and q_o > 0 else 0.0
        with np.errstate(divide="ignore", invalid="ignore"):
            lq = (z - m) - logD  # (where m is large, z - lse would leave log D out)
            far = np.where(q > 0, q * np.abs(lq), 0.0).sum()                 # mean distance under q
            zo = z[~named]
            if q_o > 0:
                lqo = math.log(q_o)
                # within the unnamed columns, relative to their own maximum
                eo = np.exp(zo - zo.max())
                far_o = np.where(eo > 0, eo * (zo.max() - zo), 0.0).sum() / eo.sum()
            else:
                lqo, far_o = 0.0, 0.0
            loss[n] = np.where(p > 0, p * (lt - lq[c]), 0.0).sum()
            y = np.where(np.isfinite(lq), np.abs(lq), 0.0)
        if r > 0:
            loss[n] += r * (math.log(r) - lqo)
        # log2(e) / T is rounded once: as logits scaled by 1 +- U.  rel is the unnamed columns' sum's
        rel = U * (42 + 4 * far_o)
        tl[n] = T * T * (rel * (p.sum() * q_o + r * (1 - q_o) + r) + 2 * U * ((p * (y[c] + far)).sum() + r * (far_o + far + abs(lqo))))
        # what is 64-bit on either side: z, its difference from the largest and the log-sums, in units that are 1 or
        # log2 e, are rounded fewer than 8 times by 2^-53 each; so are p and its logarithm.  (Equal z have no difference.)
        with np.errstate(invalid="ignore"):
            fin = np.where(np.isfinite(z), z, 0.0)
            own64 = 8 * 1.45 * 2.0 ** -53 * (np.where(fin == m, 0.0, np.abs(fin) + abs(m)) + logD + 4)
        lt64 = np.abs(np.where(p > 0, lt, 0.0))
        tl[n] += T * T * ((p * (own64[c] + 8 * 2.0 ** -53 * (lt64 + 4))).sum() + r * (own64.max() if r > 0 else 0.0))
        loss[n] *= T * T
        P = np.zeros(V)
        np.add.at(P, c, p)
        S = p.sum() + r
        s = scale[n] * T
        dx[n] = s * (q * S - P)
        if r > 0:
            dx[n][~named] -= s * q[~named] * r / q_o
        rel_q = U * (6 * y + 2 * far + 8 + (2 * abs(lse) if dtype == torch.bfloat16 else 0)) + rel * q_o
        size = np.where(named, S, S + (r / q_o if r > 0 else 0.0))
        p64 = np.zeros(V)
        np.add.at(p64, c, p * 8 * 2.0 ** -53 * (lt64 + 4))
        tol[n] = abs(s) * (q * S * own64 + p64)
        tol[n] += abs(s) * q * size * (rel_q + np.where(named, 0.0, 2 * rel + 2 * U * (far_o + far) + 4 * U)) + 2 * U * np.abs(dx[n]) + TINY
        tol[n] = 1.02 * tol[n] + half_step(dtype) * (np.abs(dx[n]) + tol[n])
    return loss, 1.02 * tl + 1.01 * U * np.abs(np.nan_to_num(loss, posinf=0.0)) + TINY, dx, tol
