"""Distillation from a teacher's top logits, loss and gradient, against the 64-bit definition."""
import math

import numpy as np
import pytest
import torch

import vocab_cross_entropy_amd as vce
from gpu_util import say
from ops_util import assert_within
from score_util import U, f64, ref_distill

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAMES = {BF16: "bf16", F32: "f32"}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _case(d0, d1, V, K, dtype, seed, tail, T=1.0, ragged=True, tdtype=F32, learnt=True):
    """(x, ids, values, len) on the CPU: distinct columns, lengths from none to past K."""
    g, N = _gen(seed), d0 * d1
    x = (torch.randn((N, V), generator=g) * 2).to(dtype)
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)])
    t = torch.randn((N, K), generator=g) * 2 + 5
    if learnt:  # the student puts most of its probability on the named columns, in one row nearly all of it
        x.scatter_(1, ids, (t + torch.randn((N, K), generator=g) + 4).to(dtype))
        x[0].scatter_(0, ids[0], (t[0] + 25).to(dtype))
    if tail:
        t = t / T
        t = t - t.logsumexp(1, keepdim=True) + torch.log(torch.rand((N, 1), generator=g) * 0.7 + 0.299)
    n = torch.randint(0, K + 1, (N,), generator=g, dtype=torch.int32) if ragged else None
    if ragged:
        n[0] = K + 3  # taken as K
        if N > 1:
            n[1] = 0
        if N > 2:
            n[2] = -2  # taken as 0
        past = torch.arange(K) >= n.view(N, 1)
        ids[past] = -100  # what stands behind the entries is not looked at
        t[past] = math.nan
    return x.view(d0, d1, V), ids.view(d0, d1, K), t.to(tdtype).view(d0, d1, K), n


def _ref(x, ids, t, n, T, tail, reduce, g, dtype):
    N, V, K = x.shape[0] * x.shape[1], x.shape[2], ids.shape[2]
    have = np.full(N, K) if n is None else np.clip(n.numpy(), 0, K)
    count = int((have > 0).sum())
    up = np.ones(N) if g is None else (f64(g) if reduce == "none" else np.full(N, float(g[0])))
    scale = up / count if reduce == "mean" and count else up
    l, tl, dx, tol = ref_distill(f64(x).reshape(N, V), ids.reshape(N, K).numpy(), f64(t).reshape(N, K), have, float(np.float32(T)),
                                 tail, scale, dtype)
    if reduce != "none":
        total = l.sum() / (count if reduce == "mean" else 1)
        # rows are rounded to FP32 and added in 64 bits
        tl = np.array([(tl.sum() + U * np.abs(l).sum()) / (count if reduce == "mean" else 1) + 2 * U * abs(total)])
        l = np.array([total])
    return l, tl, dx, tol, count


SHAPES = [(1, 1, 2), (2, 3, 7), (1, 5, 63), (2, 2, 500), (1, 3, 2049), (2, 2, 4100), (1, 3, 8195), (3, 2, 16391), (1, 3, 32003),
          (1, 2, 40009), (2, 2, 128000)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("tail", [False, True], ids=["logits", "logprobs"])
@pytest.mark.parametrize("d0,d1,V", SHAPES, ids=[f"{a}x{b}x{c}" for a, b, c in SHAPES])
def test_loss_and_gradient(d0, d1, V, tail, dtype):
    N = d0 * d1
    for K, T, reduce, tdtype in ((1, 1.0, "none", F32), (min(V, 5), 2.0, "mean", BF16), (min(V, 64), 0.75, "sum", F32),
                                 (min(V, 65), 4.0, "none", BF16), (min(V, 128), 1.25, "mean", F32)):
        say(f"distill {NAMES[dtype]} {d0}x{d1}x{V} K{K} T{T} {reduce} tail={tail}")
        x, ids, t, n = _case(d0, d1, V, K, dtype, V + K, tail, T, tdtype=tdtype)
        g = torch.randn(N if reduce == "none" else 1, generator=_gen(K))
        l, tl, dx, tol, count = _ref(x, ids, t, n, T, tail, reduce, g, dtype)
        what = f"K={K} T={T} {reduce}"
        args = (ids.cuda(), t.cuda(), T, reduce)
        kw = dict(teacher="logprobs" if tail else "logits", teacher_len=n.cuda(), grad_out=g.cuda())
        xd, out = x.cuda(), torch.full_like(x, 3.0, device="cuda")
        nv = torch.zeros(1, dtype=torch.int32, device="cuda")
        loss, nv2 = vce.ce_distill_fwd_bwd(xd, *args, out=out, n_valid=nv, **kw)
        assert nv2 is nv and int(nv) == count
        assert torch.equal(xd.cpu(), x)
        assert_within(f64(loss), l, tl, f"{what}: loss")
        assert_within(f64(out).reshape(N, V), dx, tol, f"{what}: dx")
        only, _ = vce.ce_distill_fwd_bwd(xd, *args, want_grad=False, **kw)
        assert torch.equal(only, loss) and torch.equal(xd.cpu(), x)
        again, _ = vce.ce_distill_fwd_bwd(xd, *args, **kw)
        assert torch.equal(xd, out) and torch.equal(again, loss), f"{what}: in place"
        for r in np.flatnonzero(np.clip(n.numpy(), 0, K) == 0):
            assert bool((out.view(N, V)[r].view(torch.int16 if dtype == BF16 else torch.int32) == 0).all()), "+0.0"


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
def test_without_lengths_and_upstream(dtype):
    x, ids, t, _ = _case(2, 3, 3001, 10, dtype, 5, False, ragged=False)
    for reduce in ("none", "mean", "sum"):
        l, tl, dx, tol, count = _ref(x, ids, t, None, 1.0, False, reduce, None, dtype)
        nv = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.empty_like(x, device="cuda")
        loss, _ = vce.ce_distill_fwd_bwd(x.cuda(), ids.cuda(), t.cuda(), 1.0, reduce, out=out, n_valid=nv)
        assert int(nv) == 6
        assert_within(f64(loss), l, tl, f"{reduce}: loss")
        assert_within(f64(out).reshape(6, -1), dx, tol, f"{reduce}: dx")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("V", [40, 5001, 70001])
def test_special_rows(V, dtype):
    """Masked students, teachers that are sure, columns named twice, all columns named, bad columns, NaN, infinities."""
    K, g = 32, _gen(V)
    base = torch.randn((V,), generator=g) * 2
    cols = torch.randperm(V, generator=g)[:K]
    tv = torch.randn((K,), generator=g)
    inf, nan = math.inf, math.nan

    def put(v, at, val):
        v = v.clone()
        v[at] = val
        return v

    only_named = torch.full((V,), -inf)
    only_named[cols] = tv * 2
    rows = {
        "plain": (base, cols, tv),
        "masked elsewhere": (torch.where(torch.rand(V, generator=g) < 0.75, torch.tensor(-inf), base).index_copy(0, cols, base[cols]), cols, tv),
        "named columns alone": (only_named, cols, tv),
        "a named column masked": (put(base, cols[3], -inf), cols, tv),
        "a named column masked, not wanted": (put(base, cols[3], -inf), cols, put(tv, 3, -inf)),
        "the teacher is sure": (base, cols, put(tv, 5, 60.0)),
        "both are sure": (put(base, cols[5], 60.0), cols, put(tv, 5, 60.0)),
        "the student is sure of another": (put(base, cols[6], 40.0), cols, put(tv, 5, 60.0)),
        "the same column twice": (base, put(put(cols, 1, cols[0]), 31, cols[0]), tv),
        "one column only": (base, cols[:1].expand(K), tv),
        "neighbours": (base, torch.arange(K) + V // 2 - 8 if V > 60 else torch.arange(K), tv),
        "lowest value": (put(base, cols[::8], torch.finfo(dtype).min), cols, tv),
        "lowest values alone": (torch.full((V,), torch.finfo(dtype).min), cols, tv),
        "masked by -1e9": (torch.full((V,), -1e9), cols, tv),
        "masked by -1e9 but for some": (torch.full((V,), -1e9).index_copy(0, cols[:5], tv[:5]), cols, tv),
        "around 1e5": (base + 1e5, cols, tv),
        "a teacher of -inf": (base, cols, torch.full((K,), -inf)),
        "a column outside": (base, put(cols, 7, V), tv),
        "a negative column": (base, put(cols, 7, -1), tv),
        "a NaN logit": (put(base, V // 2, nan), cols, tv),
        "a NaN logit named": (put(base, cols[2], nan), cols, tv),
        "a NaN teacher": (base, cols, put(tv, 2, nan)),
        "+inf": (put(base, V // 3, inf), cols, tv),
        "+inf named": (put(base, cols[2], inf), cols, tv),
        "nothing left": (torch.full((V,), -inf), cols, tv),
    }
    names, N = list(rows), len(rows)
    x = torch.stack([r[0] for r in rows.values()]).to(dtype).view(N, 1, V)
    ids = torch.stack([r[1] for r in rows.values()]).view(N, 1, K)
    for tail in (False, True):
        t = torch.stack([r[2] for r in rows.values()])
        if tail:
            shift = torch.logsumexp(torch.nan_to_num(t, nan=0.0, neginf=-100.0), 1, keepdim=True)
            t = torch.where(torch.isinf(t).all(1, keepdim=True), t, t - shift - 0.2)
        t = t.view(N, 1, K)
        l, tl, dx, tol, _ = _ref(x, ids, t, None, 1.5, tail, "none", None, dtype)
        out = torch.empty_like(x, device="cuda")
        say(f"special rows {NAMES[dtype]} V{V} tail={tail}")
        loss, _ = vce.ce_distill_fwd_bwd(x.cuda(), ids.cuda(), t.cuda(), 1.5, teacher="logprobs" if tail else "logits", out=out)
        for i, name in enumerate(names):
            assert_within(f64(loss[i:i + 1]), l[i:i + 1], tl[i:i + 1], f"{name}, tail={tail}: loss")
            assert_within(f64(out[i]).reshape(1, V), dx[i:i + 1], tol[i:i + 1], f"{name}, tail={tail}: dx")


@pytest.mark.parametrize("N", [2047, 2048, 2049, 5000])
def test_many_rows_are_counted(N):
    """The mean's rows, with and without their number asked for; the last row has no entry."""
    x, ids, t, n = _case(1, N, 37, 3, F32, N, True)
    n[-1] = 0
    l, tl, dx, tol, count = _ref(x, ids, t, n, 1.0, True, "mean", None, F32)
    say(f"distill {N} rows")
    for nv in (None, torch.zeros(1, dtype=torch.int32, device="cuda")):
        out = torch.empty_like(x, device="cuda")
        loss, _ = vce.ce_distill_fwd_bwd(x.cuda(), ids.cuda(), t.cuda(), 1.0, "mean", teacher="logprobs",
                                         teacher_len=n.cuda(), out=out, n_valid=nv)
        assert nv is None or int(nv) == count
        assert_within(f64(loss), l, tl, "loss")
        assert_within(f64(out).reshape(N, -1), dx, tol, "dx")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("V", [5001, 70001])
def test_students_sure_by_far(V, dtype):
    """Unnamed columns whose share of the student is far below FP32's smallest number, and named ones of such a share."""
    K, gaps, g = 8, (60.0, 100.0, 200.0, 600.0, -100.0, -600.0), _gen(V + 2)
    N = len(gaps)
    x = (torch.randn((N, V), generator=g) * 2).view(N, 1, V)
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in gaps]).view(N, 1, K)
    t = torch.log_softmax(torch.randn((N, 1, K), generator=g), 2) - 0.4
    for n, gap in enumerate(gaps):
        x[n, 0, ids[n, 0, :4 if n % 2 else K]] += gap
    x = x.to(dtype)
    for T in (1.0, 1.5):
        for tail in (True, False):
            l, tl, dx, tol, _ = _ref(x, ids, t, None, T, tail, "none", None, dtype)
            out = torch.empty_like(x, device="cuda")
            say(f"sure by far {NAMES[dtype]} V{V} T{T} tail={tail}")
            loss, _ = vce.ce_distill_fwd_bwd(x.cuda(), ids.cuda(), t.cuda(), T, teacher="logprobs" if tail else "logits",
                                             out=out)
            assert_within(f64(loss), l, tl, f"T={T} tail={tail}: loss")
            assert_within(f64(out).reshape(N, V), dx, tol, f"T={T} tail={tail}: dx")


def test_every_column_named():
    """No column is left for what the teacher leaves: it is left out."""
    V = 24
    x = torch.randn((3, 1, V), generator=_gen(1))
    ids = torch.stack([torch.randperm(V, generator=_gen(i)) for i in range(3)]).view(3, 1, V)
    t = torch.log_softmax(torch.randn((3, 1, V), generator=_gen(9)), 2) - 0.1
    l, tl, dx, tol, _ = _ref(x, ids, t, None, 1.0, True, "none", None, F32)
    out = torch.empty_like(x, device="cuda")
    loss, _ = vce.ce_distill_fwd_bwd(x.cuda(), ids.cuda(), t.cuda(), teacher="logprobs", out=out)
    assert_within(f64(loss), l, tl, "loss")
    assert_within(f64(out).reshape(3, V), dx, tol, "dx")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
def test_layouts(dtype):
    V, K = 5003, 6
    g = _gen(3)
    store = (torch.randn((4, 6, V + 9), generator=g) * 2).to(dtype)
    ids_store = torch.randint(0, V, (6, 6, 8), generator=g)
    t_store = torch.randn((6, 6, 8), generator=g)

    def view(s, name):
        return {"transposed": s[:, :, :V].transpose(0, 1), "odd start": s[:, :, 3:V + 3], "every other row": s[::2, ::3, 1:V + 1]}[name]

    for name in ("transposed", "odd start", "every other row"):
        x = view(store, name)
        d0, d1 = x.shape[:2]
        N = d0 * d1
        for ids, t in ((ids_store[:d0, :d1, 1:1 + K], t_store[:d1, :d0, 2:2 + K].transpose(0, 1)),
                       (ids_store[:1, :1, :K].expand(d0, d1, K), t_store[:1, :d1, :K].expand(d0, d1, K))):
            l, tl, dx, tol, _ = _ref(x, ids, t, None, 1.0, False, "none", None, dtype)
            xd, out = store.cuda(), torch.full_like(store, 7.0, device="cuda")
            idd = ids_store.cuda().as_strided(ids.shape, ids.stride(), ids.storage_offset())
            td = t_store.cuda().as_strided(t.shape, t.stride(), t.storage_offset())
            loss, _ = vce.ce_distill_fwd_bwd(view(xd, name), idd, td, out=view(out, name))
            assert_within(f64(loss), l, tl, f"{name}: loss")
            assert_within(f64(view(out, name)).reshape(N, V), dx, tol, f"{name}: dx")
            vce.ce_distill_fwd_bwd(view(xd, name), idd, td)
            assert torch.equal(view(xd, name), view(out, name))
            view(out, name).fill_(7.0)
            assert bool((out == 7.0).all()), f"{name}: written outside its rows"


def test_gradient_against_differences():
    d0, d1, V, K, T = 2, 2, 41, 5, 2.0
    for tail in (False, True):
        x, ids, t, n = _case(d0, d1, V, K, F32, 13, tail, T, learnt=False)
        n[:] = torch.tensor([5, 3, 0, 4])
        ids = torch.where(torch.arange(K) < n.view(d0, d1, 1), ids.clamp(min=0), -100)
        for i in range(4):
            ids.view(4, K)[i] = torch.randperm(V, generator=_gen(i))[:K]
        t = torch.nan_to_num(t, nan=0.0)
        leaf = x.cuda().requires_grad_()
        loss = vce.distillation_loss(leaf * 1, ids.cuda(), t.cuda(), T, "mean", teacher="logprobs" if tail else "logits",
                                     teacher_len=n.cuda())
        (3.0 * loss).backward()
        got, step = f64(leaf.grad), 1e-4

        def value(z):
            l = ref_distill(z.reshape(4, V), ids.view(4, K).numpy(), f64(t).reshape(4, K), n.numpy(), T, tail, np.ones(4))[0]
            return 3.0 * l.sum() / 3

        for at in [(0, 0, int(ids[0, 0, 0])), (0, 1, int(ids[0, 1, 1])), (0, 0, 7), (1, 1, 40), (1, 0, 3)]:
            hi, lo = f64(x).copy(), f64(x).copy()
            hi[at] += step
            lo[at] -= step
            diff = (value(hi) - value(lo)) / (2 * step)
            assert abs(got[at] - diff) <= 2e-6 * (1 + abs(diff)), (tail, at, got[at], diff)


@pytest.mark.parametrize("reduce", [False, "mean", "sum"])
def test_autograd_form(reduce):
    x, ids, t, n = _case(2, 3, 9001, 12, BF16, 17, False)
    N = 6
    up = torch.rand((2, 3) if not reduce else (), generator=_gen(2)) + 0.5
    l, tl, dx, tol, _ = _ref(x, ids, t, n, 2.0, False, reduce or "none", up.reshape(-1), BF16)
    leaf = x.cuda().requires_grad_()
    z = leaf * 1
    loss = vce.distillation_loss(z, ids.cuda(), t.cuda(), 2.0, reduce, teacher_len=n.cuda())
    assert loss.shape == up.shape
    loss.backward(up.cuda())
    assert_within(f64(loss).reshape(-1), l, tl, "loss")
    # a second BF16 rounding: by the upstream gradient
    assert_within(f64(leaf.grad).reshape(N, -1), dx, 2.1 * tol, "dx")
    plain = x.cuda()
    with torch.no_grad():
        assert torch.equal(vce.distillation_loss(plain, ids.cuda(), t.cuda(), 2.0, reduce, teacher_len=n.cuda()), loss)
    assert torch.equal(plain.cpu(), x), "without a gradient to give the logits stay"
    plain.requires_grad_()
    with torch.no_grad():
        assert torch.equal(vce.distillation_loss(plain, ids.cuda(), t.cuda(), 2.0, reduce, teacher_len=n.cuda()), loss)
    assert torch.equal(plain.detach().cpu(), x), "nor where none is recorded"
    with pytest.raises(vce.CeArgumentError):
        vce.distillation_loss(z, ids.cuda(), t.cuda().requires_grad_(), 2.0, reduce)


def test_no_rows():
    x = torch.empty((0, 3, 100), device="cuda")
    ids, t = torch.empty((0, 3, 4), dtype=torch.int64, device="cuda"), torch.empty((0, 3, 4), device="cuda")
    nv = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    assert vce.ce_distill_fwd_bwd(x, ids, t, 1.0, "sum", n_valid=nv)[0].item() == 0.0 and int(nv) == 0
    assert math.isnan(vce.ce_distill_fwd_bwd(x, ids, t, 1.0, "mean")[0].item())
    assert vce.ce_distill_fwd_bwd(x, ids, t)[0].shape == (0,)
    x, ids, t, n = _case(1, 4, 5000, 4, BF16, 3, False)
    n[:] = 0
    xd = x.cuda()
    loss, _ = vce.ce_distill_fwd_bwd(xd, ids.cuda(), t.cuda(), 1.0, "mean", teacher_len=n.cuda())
    assert math.isnan(loss.item()) and bool((xd == 0).all())


def test_repeats_workspaces_and_graphs():
    """Bit-equal repeats on one workspace shared with other calls and streams; replays of two graphs on it."""
    cases = [(_case(1, 5, 70001, 20, BF16, 41, True), "mean"), (_case(2, 3, 17000, 7, F32, 42, True), "sum")]
    dev = [([v.cuda() for v in c], red) for c, red in cases]
    nbytes = max([vce.ce_distill_workspace_bytes(c[0]) for c, _ in dev]
                 + [vce.ce_token_logprobs_workspace_bytes(dev[0][0][0], 5), vce.ce_workspace_bytes(dev[0][0][0])])
    ws = vce.ce_workspace_init(torch.empty(nbytes, dtype=torch.uint8, device="cuda"))

    def step(i, ws=ws):
        (x, ids, t, n), red = dev[i]
        out = torch.empty_like(x)
        loss, _ = vce.ce_distill_fwd_bwd(x, ids, t, 1.0, red, teacher="logprobs", teacher_len=n, out=out, ws=ws)
        return loss, out

    side = torch.cuda.Stream()
    want = [step(i, None) for i in (0, 1)]
    for i in range(4):
        with torch.cuda.stream(side if i % 2 else torch.cuda.current_stream()):
            got = [step(i, ws) for i in (0, 1)]
            vce.ce_token_logprobs(dev[0][0][0], top_k=5, ws=ws)
        torch.cuda.synchronize()
        for a, b in zip(sum(got, ()), sum(want, ())):
            assert torch.equal(a, b)
    graphs = []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(i)
        graphs.append((g, out))
    for i in range(5):
        for k in (1, 0) if i % 2 else (0, 1):
            x = dev[k][0][0]
            x.add_(0.25 * (i + 1) * torch.arange(x.shape[2], device="cuda").remainder(3).to(x.dtype))
            graphs[k][0].replay()
            for a, b in zip(graphs[k][1], step(k)):
                assert torch.equal(a, b), f"replay {i} of graph {k}"
    vce.ce_workspace_check(ws)


def test_unprepared_workspace_and_silent_chunk():
    x, ids, t, n = _case(1, 4, 70001, 6, BF16, 51, False, ragged=False)
    xd, idd, td = x.cuda(), ids.cuda(), t.cuda()
    nbytes = vce.ce_distill_workspace_bytes(xd)
    ws = vce.ce_workspace_init(torch.empty(nbytes, dtype=torch.uint8, device="cuda"))
    words = ws.view(torch.int64)
    words[4] = (2 + 1) << 8 | 1  # row 2's chunk 1 publishes nothing, forced from the host: a bounded wait, then NaN
    out = torch.empty_like(xd)
    loss, _ = vce.ce_distill_fwd_bwd(xd, idd, td, out=out, ws=ws)
    with pytest.raises(vce.CeError):
        vce.ce_workspace_check(ws)
    assert loss.isnan().tolist() == [False, False, True, False]
    l, tl, dx, tol, _ = _ref(x, ids, t, None, 1.0, False, "none", None, BF16)
    keep = [0, 1, 3]
    assert_within(f64(loss)[keep], l[keep], tl[keep], "others' loss")
    assert_within(f64(out).reshape(4, -1)[keep], dx[keep], tol[keep], "others' dx")
    assert bool(out[0, 2].isnan().all())
    words[4] = 0
    vce.ce_distill_fwd_bwd(xd, idd, td, out=out, ws=ws)
    assert_within(f64(out).reshape(4, -1), dx, tol, "next call")
    raw = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    d = vce._abi.CeDistill(idd.data_ptr(), idd.stride(0), idd.stride(1), td.data_ptr(), td.stride(0), td.stride(1), 0, 0, 6, 1.0, None)
    desc = [vce._ops._logits(v, "x", 0, None)[0] for v in (xd, out)]
    loss = torch.zeros(1, device="cuda")
    assert vce.lib.ce_distill_fwd_bwd(*desc, d, 2, None, loss.data_ptr(), None, raw.data_ptr(), nbytes, None) == 0
    torch.cuda.synchronize()
    assert bool(loss.isnan().all()) and bool(out.isnan().all())
    assert vce.lib.ce_workspace_check(raw.data_ptr(), None) == vce._abi.CE_EWORKSPACE


def test_far_and_long_rows():
    V, far = 33000, (1 << 32) + 5
    store = torch.empty(far + V, dtype=BF16, device="cuda")
    x = store.as_strided((2, 1, V), (far, V, 1))
    ref, ids, t, _ = _case(2, 1, V, 8, BF16, 61, True, ragged=False)
    x.copy_(ref)
    l, tl, dx, tol, _ = _ref(ref, ids, t, None, 1.0, True, "none", None, BF16)
    loss, _ = vce.ce_distill_fwd_bwd(x, ids.cuda(), t.cuda(), teacher="logprobs")
    assert_within(f64(loss), l, tl, "far: loss")
    assert_within(f64(x).reshape(2, V), dx, tol, "far: dx")
    del store, x
    for dtype, V in ((BF16, 1 << 21), (F32, 1 << 20)):  # the most chunks a row has
        x, ids, t, _ = _case(1, 1, V, 30, dtype, 62, True, ragged=False)
        l, tl, dx, tol, _ = _ref(x, ids, t, None, 1.0, True, "mean", None, dtype)
        xd = x.cuda()
        loss, _ = vce.ce_distill_fwd_bwd(xd, ids.cuda(), t.cuda(), 1.0, "mean", teacher="logprobs")
        assert_within(f64(loss), l, tl, f"V={V}: loss")
        assert_within(f64(xd).reshape(1, V), dx, tol, f"V={V}: dx")
        with pytest.raises(vce.CeArgumentError):
            vce.ce_distill_fwd_bwd(torch.empty((1, 1, V + 1), dtype=dtype, device="cuda"), ids.cuda(), t.cuda())
