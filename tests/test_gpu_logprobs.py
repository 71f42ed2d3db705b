"""Token log-probabilities, entropy and alternatives, and their gradient, against 64-bit definitions."""
import ctypes
import math

import numpy as np
import pytest
import torch

import vocab_cross_entropy_amd as vce
from gpu_util import say
from ops_util import assert_within
from score_util import Row64, U, f64, half_step, largest, ref_logprobs_grad

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAMES = {BF16: "bf16", F32: "f32"}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _logits(d0, d1, V, dtype, seed, sigma=3.0):
    return (torch.randn((d0, d1, V), generator=_gen(seed)) * sigma).to(dtype)


def _ids(d0, d1, M, V, seed):
    ids = torch.randint(0, V, (d0, d1, M), generator=_gen(seed))
    if d0 * d1 > 2 and M:
        ids.view(-1, M)[2, 0] = -100
    return ids


def _sharpen(x, ids):
    """Rows in which the first given token is likely, nearly certain, or certain to FP32."""
    rows, V = x.view(-1, x.shape[2]), x.shape[2]
    for r in range(0, rows.shape[0], 2):
        t = int(ids.reshape(rows.shape[0], -1)[r, 0])
        if 0 <= t < V:
            rows[r, t] = float(rows[r].float().max()) + (2.0, 12.0, 30.0)[r // 2 % 3]


def _check(x, ids, K, got, what, dtype):
    N, V = x.shape[0] * x.shape[1], x.shape[2]
    xr = f64(x).reshape(N, V)
    ref = Row64(xr)
    if ids is not None:
        lp, tol = ref.logp(ids.reshape(N, -1).numpy())
        assert got.logprobs.shape == ids.shape and got.logprobs.dtype == F32
        assert_within(f64(got.logprobs).reshape(N, -1), lp, tol, f"{what}: logprobs")
    if got.entropy is not None:
        assert_within(f64(got.entropy).reshape(N), ref.H, ref.tol_H, f"{what}: entropy")
    if got.lse is not None:
        assert_within(f64(got.lse).reshape(N), ref.lse, ref.tol_logd + 1.01 * U * np.abs(np.nan_to_num(ref.lse)) + 1e-40,
                      f"{what}: lse")
    if K:
        top = largest(xr, K)
        have = got.top_ids.cpu().numpy().reshape(N, K)
        assert np.array_equal(have, top), f"{what}: alternatives, row {np.argwhere((have != top).any(1))[0]}"
        lp, tol = ref.logp(top, None)
        assert_within(f64(got.top_logprobs).reshape(N, K), lp, tol, f"{what}: top_logprobs")
    return ref


SHAPES = [(1, 1, 1), (1, 1, 2), (2, 3, 7), (3, 1, 8), (1, 5, 63), (1, 3, 300), (2, 2, 1023), (1, 3, 1025), (1, 2, 2048),
          (1, 3, 2049), (2, 1, 4097), (1, 2, 8191), (1, 2, 16384), (1, 2, 16385), (3, 2, 32003), (1, 2, 128000),
          (2, 65, 33001)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("d0,d1,V", SHAPES, ids=[f"{a}x{b}x{c}" for a, b, c in SHAPES])
def test_forward(d0, d1, V, dtype):
    x = _logits(d0, d1, V, dtype, seed=V)
    ids = _ids(d0, d1, 3, V, seed=V + 1)
    _sharpen(x, ids)
    xd, idd = x.cuda(), ids.cuda()
    for K in sorted({0, 1, min(V, 5), min(V, 20), min(V, 128)}):
        say(f"forward {NAMES[dtype]} {d0}x{d1}x{V} K{K}")
        got = vce.ce_token_logprobs(xd, idd, top_k=K, entropy=True, stats=True, lse=True)
        ref = _check(x, ids, K, got, f"K={K}", dtype)
        st = f64(got.stats)
        assert np.array_equal(st[:, 0], ref.m)
        assert_within(st[:, 1], ref.logd, ref.tol_logd, "stats: log D")
        assert_within(st[:, 2], ref.rest / ref.D, ref.rel * ref.rest / ref.D * 2 + 4 * U * ref.rest / ref.D + 1e-40,
                      "stats: 1 - p_max")
        assert torch.equal(got.stats[:, 3], got.entropy.view(-1))
        # each output by itself, bit for bit the same
        alone = vce.ce_token_logprobs(xd, idd, top_k=K)
        assert torch.equal(alone.logprobs, got.logprobs) and alone.entropy is None and alone.stats is None
        if K:
            assert torch.equal(alone.top_ids, got.top_ids) and torch.equal(alone.top_logprobs, got.top_logprobs)
    only = vce.ce_token_logprobs(xd, entropy=True)
    assert torch.equal(only.entropy, got.entropy) and only.logprobs is None and only.top_ids is None
    assert torch.equal(xd.cpu(), x), "the logits were written"


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("M", [1, 64, 65, 128])
def test_many_given_tokens(dtype, M):
    for d0, d1, V in ((2, 2, 500), (1, 2, 40000)):
        x, ids = _logits(d0, d1, V, dtype, seed=M), _ids(d0, d1, M, V, seed=M + 7)
        ids.view(-1, M)[-1, M // 2] = V          # outside: NaN
        ids.view(-1, M)[0, M - 1] = -7
        got = vce.ce_token_logprobs(x.cuda(), ids.cuda())
        _check(x, ids, 0, got, f"M={M} V={V}", dtype)
        # (d0, d1) ids stand for one token
        one = ids[..., 0].contiguous()
        got1 = vce.ce_token_logprobs(x.cuda(), one.cuda())
        assert got1.logprobs.shape == one.shape and torch.equal(got1.logprobs.isnan(), got.logprobs[..., 0].isnan())
        assert torch.equal(got1.logprobs.nan_to_num(), got.logprobs[..., 0].nan_to_num())


def _special_rows(V, dtype, seed):
    """Rows that alternatives and sums can go wrong at, by name."""
    g = _gen(seed)
    base = torch.randn((V,), generator=g) * 3
    rows = {"plain": base.clone(), "constant": torch.full((V,), 1.5), "zeros of both signs": torch.zeros(V)}
    rows["zeros of both signs"][::3] = -0.0
    rows["ascending"] = torch.arange(V, dtype=F32) / V * 40 - 20
    rows["descending"] = rows["ascending"].flip(0).clone()
    rows["coarse"] = (base * 0.5).round()
    masked = base.clone()
    masked[torch.rand(V, generator=g) < 0.75] = -math.inf
    masked[V // 2] = 0.25
    rows["a quarter left"] = masked
    few = torch.full((V,), -math.inf)
    few[[0, V // 3, V - 1]] = torch.tensor([1.0, 2.0, 1.0])
    rows["three left"] = few
    one = torch.full((V,), -math.inf)
    one[V // 2] = -3.0
    rows["one left"] = one
    rows["lowest value"] = torch.where(torch.isinf(masked), torch.tensor(torch.finfo(dtype).min), masked)
    rows["lowest values alone"] = torch.full((V,), torch.finfo(dtype).min)
    rows["masked by -1e9"] = torch.full((V,), -1e9)
    rows["masked by -1e4 but for one"] = torch.full((V,), -1e4)
    rows["masked by -1e4 but for one"][V // 2] = 7.0
    rows["around 1e5"] = base + 1e5
    huge = torch.full((V,), -2.9e38)
    huge[::3] = 2.9e38
    rows["out of range of the exponent"] = huge
    run = base.clone()  # the largest ones side by side, in one lane's vectors
    run[V // 4: V // 4 + min(V - V // 4, 130)] += 50
    rows["a run"] = run
    rows["large"] = base * 1e4
    rows["tiny"] = base * 1e-30
    rows["nothing left"] = torch.full((V,), -math.inf)
    nan = base.clone()
    nan[V // 5] = math.nan
    rows["a NaN"] = nan
    rows["all NaN"] = torch.full((V,), math.nan)
    half = base.clone()
    half[V // 2:] = math.nan
    rows["half NaN"] = half
    inf = base.clone()
    inf[V // 7] = math.inf
    rows["+inf"] = inf
    both = masked.clone()
    both[V // 3] = math.inf
    rows["+inf and -inf"] = both
    return rows


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("V", [9, 130, 700, 2000, 4099, 40001, 70000])
def test_special_rows(V, dtype):
    rows = _special_rows(V, dtype, seed=V)
    x = torch.stack(list(rows.values())).to(dtype).view(len(rows), 1, V)
    ids = torch.tensor([0, V // 3, V // 2, V - 1]).expand(len(rows), 1, 4)
    for K in {1, min(V, 20), min(V, 128)}:
        say(f"special rows {NAMES[dtype]} V{V} K{K}")
        got = vce.ce_token_logprobs(x.cuda(), ids.cuda(), top_k=K, entropy=True, lse=True)
        for i, name in enumerate(rows):
            part = vce.TokenLogprobs(*(None if t is None else t[i:i + 1] for t in got))
            _check(x[i:i + 1], ids[i:i + 1], K, part, f"{name}, K={K}", dtype)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
def test_layouts(dtype):
    V = 5003
    store = _logits(4, 6, V + 11, dtype, seed=5)
    views = {"transposed": store[:, :, :V].transpose(0, 1), "odd start": store[:, :, 3:V + 3],
             "every other row": store[::2, ::3, 1:V + 1]}
    ids_store = torch.randint(0, V, (7, 9, 5), generator=_gen(6))
    for name, x in views.items():
        d0, d1 = x.shape[:2]
        dev = store.cuda()
        xd = {"transposed": dev[:, :, :V].transpose(0, 1), "odd start": dev[:, :, 3:V + 3],
              "every other row": dev[::2, ::3, 1:V + 1]}[name]
        for ids in (ids_store[:d0, :d1, 1:4], ids_store[:1, :d1, :2].expand(d0, d1, 2),
                    ids_store[:d1, :d0, 0].t(), ids_store[:1, :1, :1].expand(d0, d1, 1)):
            idd = ids_store.cuda()
            idd = idd.as_strided(ids.shape, ids.stride(), ids.storage_offset())
            got = vce.ce_token_logprobs(xd, idd, top_k=7, entropy=True, stats=True)
            _check(x, ids, 7, got, name, dtype)
            dlogp = torch.randn(ids.shape, generator=_gen(8))
            flat_ids = ids.reshape(d0 * d1, -1).numpy()
            dx, tol = ref_logprobs_grad(f64(x).reshape(d0 * d1, V), flat_ids, f64(dlogp).reshape(d0 * d1, -1), None,
                                        dtype=dtype)
            out = torch.full_like(dev, 7.0)
            ov = {"transposed": out[:, :, :V].transpose(0, 1), "odd start": out[:, :, 3:V + 3],
                  "every other row": out[::2, ::3, 1:V + 1]}[name]
            vce.ce_token_logprobs_backward(xd, got.stats, idd, dlogp.cuda(), out=ov)
            assert_within(f64(ov).reshape(d0 * d1, V), dx, tol, f"{name}: dx")
            ov.fill_(7.0)
            assert bool((out == 7.0).all()), f"{name}: written outside its rows"


GRADS = [(1, 1, 1), (2, 3, 7), (1, 3, 300), (2, 2, 2049), (1, 2, 8193), (3, 2, 32003), (1, 2, 128000)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("d0,d1,V", GRADS, ids=[f"{a}x{b}x{c}" for a, b, c in GRADS])
@pytest.mark.parametrize("M,K,ent", [(1, 0, False), (1, 0, True), (5, 0, True), (0, 3, False), (2, 20, True),
                                     (128, 128, True), (0, 0, True)])
def test_gradient(d0, d1, V, dtype, M, K, ent):
    K = min(K, V)
    N, g = d0 * d1, _gen(V + M)
    x = _logits(d0, d1, V, dtype, seed=V + 3)
    ids = _ids(d0, d1, M, V, seed=V + M) if M else None
    if M:
        _sharpen(x, ids)
    if M > 3:  # the same token twice
        ids[..., 3] = ids[..., 1]
    xd = x.cuda()
    fwd = vce.ce_token_logprobs(xd, None if ids is None else ids.cuda(), top_k=K, entropy=True, stats=True)
    dlogp = torch.randn((d0, d1, M), generator=g) if M else None
    dtop = torch.randn((d0, d1, K), generator=g) if K else None
    dh = torch.randn((d0, d1), generator=g) if ent else None
    lists = [t.reshape(N, -1) for t in (ids, fwd.top_ids.cpu() if K else None) if t is not None]
    grads = [t.reshape(N, -1) for t in (dlogp, dtop) if t is not None]
    all_ids = torch.cat(lists, 1).numpy() if lists else np.zeros((N, 0), np.int64)
    all_g = f64(torch.cat(grads, 1)) if grads else np.zeros((N, 0))
    dx, tol = ref_logprobs_grad(f64(x).reshape(N, V), all_ids, all_g, None if dh is None else f64(dh).reshape(N), dtype=dtype)

    def cuda(t):
        return None if t is None else t.cuda()

    args = dict(dentropy=cuda(dh), top_ids=fwd.top_ids if K else None, dtop=cuda(dtop))
    out = vce.ce_token_logprobs_backward(xd, fwd.stats, cuda(ids), cuda(dlogp), **args)
    assert_within(f64(out).reshape(N, V), dx, tol, "dx")
    assert torch.equal(xd.cpu(), x)
    vce.ce_token_logprobs_backward(xd, fwd.stats, cuda(ids), cuda(dlogp), out=xd, **args)
    assert torch.equal(xd, out), "in place"


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
def test_gradient_of_masked_rows_and_bad_ids(dtype):
    V = 9001
    rows = _special_rows(V, dtype, seed=77)
    x = torch.stack(list(rows.values())).to(dtype).view(len(rows), 1, V)
    N = len(rows)
    ids = torch.tensor([V // 2, V // 3]).expand(N, 1, 2).contiguous()
    ids[0, 0, 1] = V       # outside the vocabulary: the row's gradient is NaN
    ids[1, 0, 0] = -100    # ignored
    g, dh = torch.randn((N, 1, 2), generator=_gen(1)), torch.randn((N, 1), generator=_gen(2))
    xd = x.cuda()
    stats = vce.ce_token_logprobs(xd, entropy=True, stats=True).stats
    out = vce.ce_token_logprobs_backward(xd, stats, ids.cuda(), g.cuda(), dentropy=dh.cuda())
    dx, tol = ref_logprobs_grad(f64(x).reshape(N, V), ids.reshape(N, 2).numpy(), f64(g).reshape(N, 2), f64(dh).reshape(N),
                                dtype=dtype)
    for i, name in enumerate(rows):
        assert_within(f64(out[i]).reshape(1, V), dx[i:i + 1], tol[i:i + 1], name)


def test_gradient_against_differences():
    """Central differences of the definition, in 64 bits, and the autograd form."""
    d0, d1, V, K = 2, 2, 37, 4
    x = _logits(d0, d1, V, F32, seed=3)
    ids = _ids(d0, d1, 3, V, seed=4)
    wl, wt, wh = (torch.randn(s, generator=_gen(5), dtype=torch.float64) for s in ((d0, d1, 3), (d0, d1, K), (d0, d1)))
    top = torch.from_numpy(largest(f64(x).reshape(-1, V), K)).view(d0, d1, K)

    def value(z):
        lp = torch.log_softmax(z, 2)
        h = -(lp.exp() * lp).sum(2)
        return ((torch.where(ids < 0, 0.0, lp.gather(2, ids.clamp(min=0))) * wl).sum() + (lp.gather(2, top) * wt).sum()
                + (h * wh).sum())

    xd = x.cuda().requires_grad_()
    r = vce.token_logprobs(xd, ids.cuda(), top_k=K, entropy=True)
    assert not r.top_ids.requires_grad and r.stats is None
    ((r.logprobs * wl.float().cuda()).sum() + (r.top_logprobs * wt.float().cuda()).sum()
     + (r.entropy * wh.float().cuda()).sum()).backward()
    got, z, step = f64(xd.grad), x.double(), 1e-5
    for at in [(0, 0, 0), (1, 1, 36), (0, 1, int(ids[0, 1, 0])), (1, 0, int(top[1, 0, 0])), (1, 1, 17)]:
        hi, lo = z.clone(), z.clone()
        hi[at] += step
        lo[at] -= step
        diff = float((value(hi) - value(lo)) / (2 * step))
        # the difference's own error: step^2 / 6 times third derivatives of at most the weights' sum, and 2^-53
        # roundings over the step
        assert abs(got[at] - diff) <= 1e-5 * (1 + abs(diff)), (at, got[at], diff)


def test_autograd_forms():
    d0, d1, V = 2, 3, 1001
    x = _logits(d0, d1, V, BF16, seed=9)
    ids = torch.randint(0, V, (d0, d1), generator=_gen(10))
    # only some of the outputs used; an upstream gradient that is expanded; logits that are a view
    for use in ("logprobs", "entropy", "top_logprobs", "none"):
        leaf = x.transpose(0, 1).contiguous().cuda().requires_grad_()
        r = vce.token_logprobs(leaf.transpose(0, 1), ids.cuda(), top_k=2, entropy=True)
        if use == "none":
            assert torch.autograd.grad(r.logprobs.sum() * 0, leaf)[0].abs().max() == 0
            continue
        getattr(r, use).sum().backward()
        N, h = d0 * d1, None
        sel = {"logprobs": ids.view(N, 1).numpy(), "top_logprobs": r.top_ids.cpu().view(N, 2).numpy(),
               "entropy": np.zeros((N, 0), np.int64)}[use]
        if use == "entropy":
            h = np.ones(N)
        dx, tol = ref_logprobs_grad(f64(x).reshape(N, V), sel, np.ones(sel.shape), h, dtype=BF16)
        assert_within(f64(leaf.grad.transpose(0, 1)).reshape(N, V), dx, tol, use)
    with torch.no_grad():
        assert vce.token_logprobs(x.cuda(), ids.cuda()).logprobs.requires_grad is False


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
def test_ignored_column_among_the_alternatives(dtype):
    """ignore_idx may be a column of the vocabulary: it is left out of the given tokens, not of the alternatives."""
    N, V, K, pad = 4, 5003, 6, 3
    x = _logits(1, N, V, dtype, seed=31)
    x[0, :, pad] = x.amax() + 1
    ids = torch.tensor([[pad, 7], [7, pad], [pad, pad], [8, 9]]).view(1, N, 2)
    g = torch.randn((N, 2 + K), generator=_gen(3))
    xd = x.cuda()
    r = vce.ce_token_logprobs(xd, ids.cuda(), top_k=K, stats=True, ignore_idx=pad)
    top = r.top_ids.cpu().view(N, K)
    assert bool((top[:, 0] == pad).all()) and bool((r.logprobs.cpu() == 0)[ids == pad].all())
    out = vce.ce_token_logprobs_backward(xd, r.stats, ids.cuda(), g[:, :2].contiguous().cuda(), top_ids=r.top_ids,
                                         dtop=g[:, 2:].contiguous().cuda(), ignore_idx=pad)
    # ignored tokens as ones of an index of no meaning, the alternatives as they are
    lists = torch.cat([torch.where(ids.view(N, 2) == pad, -100, ids.view(N, 2)), top], 1)
    dx, tol = ref_logprobs_grad(f64(x).reshape(N, V), lists.numpy(), f64(g), None, dtype=dtype)
    assert_within(f64(out).reshape(N, V), dx, tol, "dx")


def test_no_rows_and_nothing_asked():
    x = torch.empty((0, 3, 100), device="cuda")
    r = vce.ce_token_logprobs(x, torch.empty((0, 3), dtype=torch.int64, device="cuda"), top_k=4, entropy=True, stats=True)
    assert r.logprobs.shape == (0, 3) and r.top_ids.shape == (0, 3, 4) and r.stats.shape == (0, 4)
    assert vce.ce_token_logprobs_backward(x, r.stats, None, None, dentropy=r.entropy).shape == x.shape
    x = torch.randn((1, 2, 100), device="cuda")
    assert all(t is None for t in vce.ce_token_logprobs(x))
    with pytest.raises(vce.CeArgumentError):
        vce.token_logprobs(x)


def test_repeats_workspaces_and_streams():
    """Bit-equal repeats; one workspace for calls of several kinds and sizes; another stream; an unprepared one."""
    big, small = _logits(2, 3, 50021, BF16, seed=1).cuda(), _logits(1, 5, 20011, F32, seed=2).cuda()
    ids_b, ids_s = _ids(2, 3, 1, 50021, seed=3).cuda(), _ids(1, 5, 2, 20011, seed=4).cuda()
    t = torch.randint(0, 50021, (2, 3), generator=_gen(5)).cuda()
    want_b = vce.ce_token_logprobs(big, ids_b, top_k=9, entropy=True)
    want_s = vce.ce_token_logprobs(small, ids_s, top_k=3)
    nbytes = max(vce.ce_token_logprobs_workspace_bytes(big, 9), vce.ce_token_logprobs_workspace_bytes(small, 3),
                 vce.ce_workspace_bytes(big))
    ws = vce.ce_workspace_init(torch.empty(nbytes, dtype=torch.uint8, device="cuda"))
    side = torch.cuda.Stream()
    for i in range(6):
        with torch.cuda.stream(side if i % 2 else torch.cuda.current_stream()):
            got_b = vce.ce_token_logprobs(big, ids_b, top_k=9, entropy=True, ws=ws)
            vce.ce_fwd_bwd_fused(big.clone(), t, 0.1, "mean", ws=ws)
            got_s = vce.ce_token_logprobs(small, ids_s, top_k=3, ws=ws)
        torch.cuda.synchronize()
        for a, b in zip(list(got_b) + list(got_s), list(want_b) + list(want_s)):
            assert (a is None and b is None) or torch.equal(a, b)
    assert vce.ce_workspace_check(ws) is None
    raw = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    xd = vce._ops._logits(big, "x", 0, None)[0]
    q = vce._abi.CeLogprobs(ids_b.data_ptr(), ids_b.stride(0), ids_b.stride(1), 1, 9, -100)
    lp, ti, tl = (torch.zeros((6, n), dtype=d, device="cuda") for n, d in ((1, F32), (9, torch.int64), (9, F32)))
    assert vce.lib.ce_token_logprobs(xd, q, lp.data_ptr(), None, None, ti.data_ptr(), tl.data_ptr(), None, raw.data_ptr(),
                                     nbytes, None) == 0
    torch.cuda.synchronize()
    ignored = (ids_b.view(6, 1) == -100)
    assert bool((lp.isnan() | ignored).all()) and bool(tl.isnan().all()) and bool((ti == -1).all())
    assert vce.lib.ce_workspace_check(raw.data_ptr(), None) == vce._abi.CE_EWORKSPACE


def test_a_chunk_that_never_publishes():
    """The bounded wait, forced from the host: that row is NaN, the others are right, and the next call is whole."""
    x, ids = _logits(1, 4, 40001, BF16, seed=21), _ids(1, 4, 1, 40001, seed=22)
    xd, idd = x.cuda(), ids.cuda()
    ws = vce.ce_workspace_init(torch.empty(vce.ce_token_logprobs_workspace_bytes(xd, 5), dtype=torch.uint8, device="cuda"))
    words = ws.view(torch.int64)
    words[4] = (1 + 1) << 8 | 0  # row 1, chunk 0
    got = vce.ce_token_logprobs(xd, idd, top_k=5, ws=ws)
    with pytest.raises(vce.CeError):
        vce.ce_workspace_check(ws)
    assert bool(got.logprobs[0, 1].isnan().all()) and bool((got.top_ids[0, 1] == -1).all())
    keep = [0, 2, 3]
    part = vce.TokenLogprobs(got.logprobs[:, keep], None, got.top_ids[:, keep], got.top_logprobs[:, keep], None, None)
    _check(x[:, keep], ids[:, keep], 5, part, "others", BF16)
    words[4] = 0
    _check(x, ids, 5, vce.ce_token_logprobs(xd, idd, top_k=5, ws=ws), "next call", BF16)


def test_captured_calls():
    """Two graphs on one workspace, replayed in turn with eager calls between."""
    cases = [(_logits(1, 3, 40001, BF16, seed=31), 20), (_logits(2, 2, 17000, F32, seed=32), 6)]
    ids = [_ids(*x.shape[:2], 2, x.shape[2], seed=33) for x, _ in cases]
    dev = [(x.cuda(), i.cuda()) for (x, _), i in zip(cases, ids)]
    nbytes = max(vce.ce_token_logprobs_workspace_bytes(x, K) for (x, _), (_, K) in zip(dev, cases))
    ws = vce.ce_workspace_init(torch.empty(nbytes, dtype=torch.uint8, device="cuda"))

    def step(n):
        (x, i), K = dev[n], cases[n][1]
        r = vce.ce_token_logprobs(x, i, top_k=K, entropy=True, stats=True, ws=ws)
        return list(r[:5]) + [vce.ce_token_logprobs_backward(x, r.stats, i, r.logprobs, dentropy=r.entropy)]

    for n in (0, 1):
        step(n)
    torch.cuda.synchronize()
    graphs = []
    for n in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(n)
        graphs.append((g, out))
    for i in range(5):
        for n in (1, 0) if i % 2 else (0, 1):
            x, _ = dev[n]
            x.add_(0.25 * (i + 1) * torch.arange(x.shape[2], device="cuda").remainder(3).to(x.dtype))
            graphs[n][0].replay()
            for got, want in zip(graphs[n][1], step(n)):
                assert torch.equal(got, want), f"replay {i} of graph {n}"
    vce.ce_workspace_check(ws)


def test_far_rows():
    """Rows whose offsets pass 2^32 elements and bytes."""
    V, far = 33000, (1 << 32) + 5
    store = torch.empty(far + V, dtype=BF16, device="cuda")
    x = store.as_strided((2, 1, V), (far, V, 1))
    ref = _logits(2, 1, V, BF16, seed=41)
    x.copy_(ref)
    ids = _ids(2, 1, 2, V, seed=42)
    got = vce.ce_token_logprobs(x, ids.cuda(), top_k=5, entropy=True, stats=True)
    _check(ref, ids, 5, got, "far rows", BF16)
    g = torch.randn((2, 1, 2), generator=_gen(43))
    dx, tol = ref_logprobs_grad(f64(ref).reshape(2, V), ids.reshape(2, 2).numpy(), f64(g).reshape(2, 2), None, dtype=BF16)
    vce.ce_token_logprobs_backward(x, got.stats, ids.cuda(), g.cuda(), out=x)
    assert_within(f64(x).reshape(2, V), dx, tol, "dx in place")


def test_longest_rows():
    """The most chunks a row has."""
    for dtype, V in ((BF16, 1 << 20), (F32, 1 << 19)):
        x = (torch.randn((1, 1, V), generator=_gen(51)) * 4).to(dtype)
        ids = torch.tensor([[[0, V - 1, V // 2]]])
        for K in (0, 128):
            got = vce.ce_token_logprobs(x.cuda(), ids.cuda(), top_k=K, entropy=True)
            _check(x, ids, K, got, f"V={V} K={K}", dtype)
        with pytest.raises(vce.CeArgumentError):
            vce.ce_token_logprobs(torch.empty((1, 1, V + 1), dtype=dtype, device="cuda"), entropy=True)


def test_processed_then_read_and_distilled():
    """A serving step and a training step as they are used: processing in place, the sampled tokens' log-probabilities
    with alternatives; then a student's loss against those alternatives, end to end through autograd."""
    d0, d1, V, K = 2, 4, 12007, 8
    N = d0 * d1
    teacher = _logits(d0, d1, V, F32, seed=61)
    temp = torch.rand(N, generator=_gen(62)) + 0.5
    xt = teacher.cuda()
    vce.ce_logits_process(xt, temperature=temp.cuda())
    r = vce.ce_token_logprobs(xt, top_k=K)
    processed = xt.cpu()
    _check(processed, None, K, r, "processed", F32)
    student = _logits(d0, d1, V, BF16, seed=63)
    leaf = student.cuda().requires_grad_()
    loss = vce.distillation_loss(leaf * 1, r.top_ids, r.top_logprobs, 1.0, "mean", teacher="logprobs")
    loss.backward()
    from score_util import ref_distill
    l, tl, dx, tol = ref_distill(f64(student).reshape(N, V), r.top_ids.cpu().view(N, K).numpy(),
                                 f64(r.top_logprobs).reshape(N, K), np.full(N, K), 1.0, True, np.full(N, 1 / N), BF16)
    assert_within(np.array([loss.item()]), np.array([l.mean()]), tl.mean() + 2 * U * abs(l.mean()), "loss")
    assert_within(f64(leaf.grad).reshape(N, V), dx, tol, "student's gradient")
