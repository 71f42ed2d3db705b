"""Token log-probabilities where a workgroup streams a whole row in batches (many rows), where a chunk of a row is
several batches, and where a call takes several launches; special rows throughout, against 64-bit definitions."""
import math

import numpy as np
import pytest
import torch

import vocab_cross_entropy_amd as vce
from gpu_util import say
from ops_util import assert_within
from score_util import Row64, U, f64, largest, ref_distill, ref_logprobs_grad
from test_gpu_logprobs import _special_rows

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAMES = {BF16: "bf16", F32: "f32"}
SHAPES = ((64, 4), (64, 8), (256, 2), (256, 8))  # threads, vectors a thread and batch


def plan(N, V, dtype):
    """(threads, vectors, chunks of a row, batches of a chunk): the rule of logprob_plan, restated."""
    vec = 8 if dtype is BF16 else 4

    def batches(s, cols=V):
        return -(-cols // (SHAPES[s][0] * SHAPES[s][1] * vec))

    chunks = 1
    if batches(1) == 1:
        s = 0 if batches(0) == 1 else 1
    elif N >= 512 or (N >= 256 and batches(3) <= 4):
        s = 2 if batches(2) <= 2 else 3
    elif N * batches(3) >= 256:
        s, chunks = 3, min(-(-512 // N), batches(3), 64)
    else:
        chunks = min(-(-1024 // N), batches(2), 64)
        s = 2 if batches(2) <= chunks else 3
    cols = -(-(-(-V // chunks)) // vec) * vec
    return SHAPES[s][0], SHAPES[s][1], -(-V // cols), batches(s, cols)


def allowance(N, V, dtype):
    """Additions behind a row's sum, each U of it, beyond the 40 that Row64 counts: a thread's two running sums of a
    batch take half its columns each and are added; a batch adds to the sums before, which a new maximum multiplies;
    then 6 levels of a wave, the waves, and 6 levels of chunks with two weights each."""
    threads, vecs, chunks, nb = plan(N, V, dtype)
    adds = vecs * (4 if dtype is BF16 else 2) + 1 + 4 * nb + 6 + threads // 64 + (8 if chunks > 1 else 0) + 4
    return max(0, adds - 40)


class Row64Streamed(Row64):
    def __init__(self, x, more):
        super().__init__(x)
        with np.errstate(invalid="ignore"):
            extra = U * more
            self.rel = self.rel + extra
            self.tol_logd = self.tol_logd + extra * self.rest / self.D
            self.tol_H = self.tol_H + extra * (self.rest / self.D + 2 * self.S)


def _rows(V, dtype, vec, nb, seed):
    """The special rows, and rows whose batches rise or fall: batch b holds every nb-th line of 64 vectors from the
    b-th on, so a bound found from the batches so far lets all of the next ones through."""
    rows = _special_rows(V, dtype, seed)
    g = torch.Generator().manual_seed(seed + 1)
    batch = (torch.arange(V) // (64 * vec)) % nb
    noise = torch.randn((V,), generator=g)
    rows["rising batches"] = batch * 8.0 + noise
    rows["falling batches"] = batch * -8.0 + noise
    rows["rising in steps"] = batch * 2.0
    rows["the last batch alone"] = torch.where(batch == nb - 1, noise, torch.tensor(-math.inf))
    rows["a NaN in the last batch"] = torch.where((batch == nb - 1) & (noise > 2.0), torch.tensor(math.nan), noise)
    if V > 200000:  # (fewer of the longest, for the reference's time)
        rows = {k: v for i, (k, v) in enumerate(rows.items()) if i % 4 == 0 or "batch" in k}
    return rows


# (N, V): one chunk a row of 1 to 9 batches in both shapes of four waves; chunks of 3 and 11 batches
CASES = [(512, 5000, BF16), (512, 8192, BF16), (512, 8193, BF16), (512, 40001, BF16), (600, 60000, BF16),
         (512, 70001, BF16), (512, 98305, BF16), (512, 128000, BF16), (512, 140001, BF16), (256, 33000, BF16),
         (300, 65536, BF16), (255, 128000, BF16), (100, 1 << 20, BF16),
         (512, 2500, F32), (512, 4096, F32), (512, 4099, F32), (512, 20001, F32), (513, 32003, F32), (600, 33000, F32),
         (512, 70001, F32), (256, 20000, F32), (256, 32767, F32), (255, 64001, F32), (90, 1 << 19, F32)]


def test_the_cases_take_those_paths():
    plans = {(d, plan(N, V, d)) for N, V, d in CASES}
    for d in (BF16, F32):
        mine = {p for e, p in plans if e is d}
        assert {n for t, v, c, n in mine if (t, v, c) == (256, 8, 1)} >= {1, 3, 4, 5, 9}
        assert (256, 2, 1, 2) in mine
        assert {n for t, v, c, n in mine if c > 1} >= {3, 11}


@pytest.mark.parametrize("N,V,dtype", CASES, ids=[f"{n}x{v}-{NAMES[d]}" for n, v, d in CASES])
def test_rows_of_many_batches(N, V, dtype):
    vec = 8 if dtype is BF16 else 4
    threads, vecs, chunks, nb = plan(N, V, dtype)
    rows = _rows(V, dtype, vec, max(nb, 2), seed=V)
    names, R = list(rows), len(rows)
    x = torch.stack(list(rows.values())).to(dtype)
    # every row of the call is one of them: equal rows give equal bits
    source = torch.arange(N) % R
    xd = x.cuda()[source.cuda()].view(1, N, V)
    ids = torch.tensor([0, V // 3, V // 2, V - 1])
    idd = ids.cuda().view(1, 1, 4).expand(1, N, 4)
    xr = f64(x)
    ref = Row64Streamed(xr, allowance(N, V, dtype))
    lp, lp_tol = ref.logp(ids.expand(R, 4).numpy())
    top = largest(xr, 128)
    bits = torch.int32
    for K in (0, 1, 20, 128):
        say(f"streamed rows {NAMES[dtype]} {N}x{V} ({threads}x{vecs}, {chunks} chunks, {nb} batches) K{K}")
        got = vce.ce_token_logprobs(xd, idd, top_k=K, entropy=True, lse=True, stats=True)
        flat = [t.reshape(N, -1) for t in (got.logprobs, got.entropy, got.lse)]
        if K:
            flat += [got.top_ids.view(N, K), got.top_logprobs.view(N, K)]
        for t in flat:
            t = t if t.dtype is torch.int64 else t.view(bits)
            assert torch.equal(t, t[:R][(source % R).cuda()]), f"K={K}: equal rows, unequal results"
        top_lp, top_tol = ref.logp(top[:, :K], None)
        for i, name in enumerate(names):
            what, one = f"{name}, K={K}", slice(i, i + 1)
            assert_within(f64(flat[0][one]), lp[one], lp_tol[one], f"{what}: logprobs")
            assert_within(f64(flat[1][i]), ref.H[one], ref.tol_H[one], f"{what}: entropy")
            assert_within(f64(flat[2][i]), ref.lse[one], ref.tol_logd[one] + 1.01 * U * np.abs(np.nan_to_num(ref.lse[one]))
                          + 1e-40, f"{what}: lse")
            if K:
                have = flat[3][i].cpu().numpy()
                assert np.array_equal(have, top[i, :K]), f"{what}: alternatives {have[:8]}, not {top[i, :8]}"
                assert_within(f64(flat[4][one]), top_lp[one], top_tol[one], f"{what}: top_logprobs")


@pytest.mark.parametrize("N,V,dtype", [(512, 5000, BF16), (512, 2500, F32)], ids=["bf16", "f32"])
def test_gradient_from_streamed_statistics(N, V, dtype):
    assert plan(N, V, dtype)[:3] == (256, 2, 1) and allowance(N, V, dtype) == 0
    rows = _special_rows(V, dtype, seed=V + 1)
    R = len(rows)
    x = torch.stack(list(rows.values())).to(dtype)
    xd = x.cuda()[(torch.arange(N) % R).cuda()].view(1, N, V)
    g = torch.Generator().manual_seed(7)
    ids, dl, dh = torch.tensor([V // 2, V // 3]), torch.randn((N, 2), generator=g), torch.randn((N,), generator=g)
    idd = ids.cuda().view(1, 1, 2).expand(1, N, 2)
    say(f"gradient of streamed rows {NAMES[dtype]} {N}x{V}")
    stats = vce.ce_token_logprobs(xd, idd, entropy=True, stats=True).stats
    out = vce.ce_token_logprobs_backward(xd, stats, idd, dl.cuda().view(1, N, 2), dentropy=dh.cuda().view(1, N))
    part = slice(R, 2 * R)  # the second copy of each
    dx, tol = ref_logprobs_grad(f64(x), ids.expand(R, 2).numpy(), f64(dl[part]), f64(dh[part]), dtype=dtype)
    got = f64(out[0, part])
    for i, name in enumerate(rows):
        assert_within(got[i:i + 1], dx[i:i + 1], tol[i:i + 1], name)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
def test_more_rows_than_one_launch_holds(dtype):
    """2^22 workgroups in a launch: rows of the second one, in all three calls."""
    N, V, K, cut = (1 << 22) + 1001, 13, 3, 1 << 22
    g = torch.Generator("cuda").manual_seed(5)
    x = (torch.randn((1, N, V), generator=g, device="cuda") * 3).to(dtype)
    ids = torch.randint(0, V, (1, N, 2), generator=g, device="cuda")
    dl, dh = (torch.randn(s, generator=g, device="cuda") for s in ((1, N, 2), (1, N)))
    t = torch.randn((1, N, K), generator=g, device="cuda")
    n = torch.randint(0, K + 1, (N,), generator=g, device="cuda", dtype=torch.int32)
    n[-1] = K

    def run(a, b):
        xs, idn = x[:, a:b], ids[:, a:b]
        r = vce.ce_token_logprobs(xs, idn, top_k=K, entropy=True, stats=True)
        dx = vce.ce_token_logprobs_backward(xs, r.stats, idn, dl[:, a:b].contiguous(), dentropy=dh[:, a:b].contiguous())
        out = torch.empty_like(xs)
        loss, _ = vce.ce_distill_fwd_bwd(xs, r.top_ids, t[:, a:b], 1.5, "none", teacher_len=n[a:b], out=out)
        return r.logprobs[0], r.entropy[0], r.top_ids[0], r.top_logprobs[0], r.stats, dx[0], loss, out[0]

    say(f"[log-probabilities, distillation] {N} rows {dtype}")
    whole = run(0, N)
    for a, b in ((0, 4100), (cut - 300, cut), (cut, N)):
        for w, p in zip(whole, run(a, b)):
            assert torch.equal(w[a:b], p), (a, b)
    pick = torch.tensor([0, 1, cut - 1, cut, cut + 500, N - 1])
    xp = f64(x.cpu()[0, pick])
    ref = Row64(xp)
    lp, tol = ref.logp(ids.cpu()[0, pick].numpy())
    assert_within(f64(whole[0].cpu()[pick]), lp, tol, "logprobs")
    assert np.array_equal(whole[2].cpu()[pick].numpy(), largest(xp, K))
    dx, tol = ref_logprobs_grad(xp, ids.cpu()[0, pick].numpy(), f64(dl.cpu()[0, pick]), f64(dh.cpu()[0, pick]), dtype=dtype)
    assert_within(f64(whole[5].cpu()[pick]), dx, tol, "dx")
    l, tl, dx, tol = ref_distill(xp, whole[2].cpu()[pick].numpy(), f64(t.cpu()[0, pick]), n.cpu()[pick].numpy(), 1.5, False,
                                 np.ones(len(pick)), dtype)
    assert_within(f64(whole[6].cpu()[pick]), l, tl, "loss")
    assert_within(f64(whole[7].cpu()[pick]), dx, tol, "distillation's dx")
    # a reduction is brought together by the last launch
    total, _ = vce.ce_distill_fwd_bwd(x, whole[2].view(1, N, K), t, 1.5, "sum", teacher_len=n, out=torch.empty_like(x))
    want = float(whole[6].double().sum())
    assert abs(float(total) - want) <= 2 * U * abs(want)  # the same rows' FP32 losses, added in 64 bits, rounded once
