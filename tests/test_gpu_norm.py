"""RMS norm, its 8-bit form and its gradient against the 64-bit definition, and a training step's end."""
import numpy as np
import pytest
import torch

import vocab_cross_entropy_amd as vce
from gpu_util import say
from ops_util import NORM_RSTD, TINY, U, assert_within, f64, half_step, ref_norm, ref_norm_grad

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]
SHAPES = [(1, 1), (1, 7), (5, 8), (3, 511), (2, 513), (7, 1024), (9, 2048), (4, 2049), (3, 4096), (2, 4099),
          (1, 8192), (2, 8200), (2, 16384), (1, 16391), (1, 32768), (700, 40), (2600, 24)]


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(shape, dtype, seed, sigma=1.0):
    return (torch.randn(shape, generator=_gen(seed)) * sigma).to(dtype)


def _y_tol(y, dtype):
    # the sum's rounding, 1 / rms, and two products
    return (1.01 * (NORM_RSTD + 4) * U + half_step(dtype) * 1.01) * np.abs(y) + TINY


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("N,D", SHAPES)
def test_forward(N, D, dtype):
    x, r = _rand((N, D), dtype, D), _rand((N, D), dtype, D + 1, 3.0)
    for wdtype in DTYPES:
        w = _rand((D,), wdtype, 3)
        for residual in (None, r):
            say(f"[norm] {N} {D} {dtype} {wdtype} {residual is not None}")
            rd = None if residual is None else residual.cuda()
            y, s = vce.ce_rms_norm(x.cuda(), w.cuda(), rd, 1e-5)
            ref, total, _ = ref_norm(f64(x), None if residual is None else f64(r), f64(w), np.float64(np.float32(1e-5)))
            assert_within(f64(y), ref, _y_tol(ref, dtype), "y")
            if residual is None:
                assert s is None
            else:
                assert_within(f64(s), total, (half_step(dtype) * 1.01 + U) * np.abs(total) + TINY, "sum")


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("N,D", SHAPES)
def test_quantised(N, D, dtype, group):
    x, r, w = _rand((N, D), dtype, D), _rand((N, D), dtype, D + 1, 3.0), _rand((D,), dtype, 3)
    say(f"[norm e4m3] {N} {D} {dtype} {group}")
    q, scales, s = vce.ce_rms_norm_quant(x.cuda(), w.cuda(), r.cuda(), 1e-5, group=group)
    ref, total, _ = ref_norm(f64(x), f64(r), f64(w), np.float64(np.float32(1e-5)))
    assert_within(f64(s), total, (half_step(dtype) * 1.01 + U) * np.abs(total) + TINY, "sum")
    G = group or D
    groups = -(-D // G)
    assert scales.shape == (N, groups) and q.dtype == torch.float8_e4m3fn
    top = np.stack([np.abs(ref[:, k * G:(k + 1) * G]).max(1) for k in range(groups)], 1)
    rel = 1.01 * (NORM_RSTD + 4) * U
    sc = np.maximum(top / 448.0, 2.0 ** -126)
    assert_within(f64(scales), sc, (rel + 2 * U) * sc, "scales")
    # half a step of e4m3: 2^-4 of the value, 2^-10 below its normal range; the value y / scale carries 3 roundings more
    per = np.repeat(f64(scales), G, axis=1)[:, :D]
    qv = f64(q.float())
    assert np.isfinite(qv).all() and np.abs(qv).max() == 448
    assert_within(qv * per, ref, (2.0 ** -4 + 1.1 * (rel + 5 * U)) * np.abs(ref) + 2.0 ** -10 * per * 1.01, "values")
    # the nearest value of the type, and not a neighbour: from the quotient, away from the borders
    quot = ref / per
    near = torch.from_numpy(quot).float().to(torch.float8_e4m3fn).float().double().numpy()
    lo = torch.from_numpy(quot * (1 - 4 * rel)).float().to(torch.float8_e4m3fn).float().double().numpy()
    hi = torch.from_numpy(quot * (1 + 4 * rel)).float().to(torch.float8_e4m3fn).float().double().numpy()
    assert np.array_equal(qv[lo == hi], near[lo == hi])


def test_strides_and_in_place():
    N, D = 6, 777
    for dtype in DTYPES:
        say(f"[norm] strides {dtype}")
        x, r, w = _rand((N, D), dtype, 1), _rand((N, D), dtype, 2), _rand((D,), dtype, 3)
        ref, total, _ = ref_norm(f64(x), f64(r), f64(w), np.float64(np.float32(1e-6)))

        def wide(t, off):
            b = torch.full((N, D + 5), 3.0, dtype=dtype, device="cuda")
            b[:, off:off + D] = t.cuda()
            return b, b[:, off:off + D]

        (bx, vx), (br, vr) = wide(x, 1), wide(r, 3)
        vce.ce_rms_norm(vx, w.cuda(), vr, out=vx, sum_out=vr)
        assert_within(f64(vx), ref, _y_tol(ref, dtype), "y in place")
        assert_within(f64(vr), total, (half_step(dtype) * 1.01 + U) * np.abs(total) + TINY, "sum in place")
        for b, off in ((bx, 1), (br, 3)):
            edge = torch.cat([b[:, :off], b[:, off + D:]], 1)
            assert (edge == 3).all()
        # the sum over x, the output elsewhere; an 8-bit output with a row stride
        bx, vx = wide(x, 1)
        q = torch.zeros((N, D + 3), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        _, sc, _ = vce.ce_rms_norm_quant(vx, w.cuda(), r.cuda(), group=64, out=q[:, 1:1 + D], sum_out=vx)
        assert_within(f64(vx), total, (half_step(dtype) * 1.01 + U) * np.abs(total) + TINY, "sum over x")
        raw = q.view(torch.uint8)
        assert not raw[:, 0].any() and not raw[:, -2:].any()
        dense, sc2, _ = vce.ce_rms_norm_quant(x.cuda(), w.cuda(), r.cuda(), group=64)
        assert torch.equal(raw[:, 1:1 + D], dense.view(torch.uint8)) and torch.equal(sc, sc2)


def test_rows_of_zeros_infinities_and_nan():
    D = 300
    x = torch.randn((5, D), generator=_gen(1))
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[3] = 1e30  # its squares pass FP32
    w = torch.ones(D)
    say("[norm] zeros, infinities, NaN")
    y, _ = vce.ce_rms_norm(x.cuda(), w.cuda())
    y = f64(y)
    assert not y[0].any() and np.isnan(y[1]).all() and np.isnan(y[2, 7]) and not np.delete(y[2], 7).any()
    assert not y[3].any() and np.isfinite(y[4]).all()
    for group in (0, 128):
        q, sc, _ = vce.ce_rms_norm_quant(x.cuda(), w.cuda(), group=group)
        q, sc = f64(q.float()), f64(sc)
        assert not q[0].any() and (sc[0] == 2.0 ** -126).all() and np.isnan(q[1]).all()
        assert (sc[1] == 2.0 ** -126).all() and np.isfinite(q[4]).all()
    y, _ = vce.ce_rms_norm(torch.zeros((1, D), device="cuda"), w.cuda(), eps=0.0)
    assert torch.isnan(y).all()  # 0 times infinity, as the definition says


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("N,D", SHAPES)
def test_backward(N, D, dtype):
    s, dy, ds = _rand((N, D), dtype, D, 2.0), _rand((N, D), dtype, D + 1), _rand((N, D), dtype, D + 2)
    for wdtype in DTYPES:
        w = _rand((D,), wdtype, 3)
        for dsum in (None, ds):
            say(f"[norm grad] {N} {D} {dtype} {wdtype} {dsum is not None}")
            dd = None if dsum is None else dsum.cuda()
            dx, dw = vce.ce_rms_norm_backward(dy.cuda(), s.cuda(), w.cuda(), 1e-5, dsum=dd)
            rx, rw, bx, bw = ref_norm_grad(f64(dy), f64(s), f64(w), np.float64(np.float32(1e-5)),
                                           None if dsum is None else f64(ds))
            assert_within(f64(dx), rx, bx + half_step(dtype) * 1.01 * np.abs(rx), "dx")
            assert_within(f64(dw), rw, bw, "dweight")
    again = vce.ce_rms_norm_backward(dy.cuda(), s.cuda(), w.cuda(), 1e-5, dsum=dd)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    # each output by itself, adding, and in place over the incoming gradients
    only = vce.ce_rms_norm_backward(dy.cuda(), s.cuda(), w.cuda(), 1e-5, dsum=dd, want_dweight=False)
    assert only[1] is None and torch.equal(only[0], dx)
    base = torch.full((D,), 2.5, device="cuda")
    none, acc = vce.ce_rms_norm_backward(dy.cuda(), s.cuda(), w.cuda(), 1e-5, want_dx=False, dweight=base,
                                         accumulate=True)
    assert none is None
    assert_within(f64(acc), rw + 2.5, bw + U * np.abs(rw + 2.5) * 1.01, "added")
    for which in (0, 1):
        g, d = dy.cuda(), ds.cuda()
        vce.ce_rms_norm_backward(g, s.cuda(), w.cuda(), 1e-5, dsum=d, dx=(g, d)[which])
        assert torch.equal((g, d)[which], dx)


def test_refusals():
    x, w = torch.ones((4, 8), device="cuda"), torch.ones(8, device="cuda")
    for call in (lambda: vce.ce_rms_norm(x.half(), w), lambda: vce.ce_rms_norm(x, w.half()),
                 lambda: vce.ce_rms_norm(x, w[:7]), lambda: vce.ce_rms_norm(x, w.cpu()), lambda: vce.ce_rms_norm(x, None),
                 lambda: vce.ce_rms_norm(x[0], w), lambda: vce.ce_rms_norm(x.t(), w[:4]),
                 lambda: vce.ce_rms_norm(x[:, :1].expand(4, 8), w), lambda: vce.ce_rms_norm(x[:1].expand(4, 8), w),
                 lambda: vce.ce_rms_norm(x, w, x[:3]), lambda: vce.ce_rms_norm(x, w, x.bfloat16()),
                 lambda: vce.ce_rms_norm(x, w, out=x.bfloat16()), lambda: vce.ce_rms_norm(x, w, eps=-1.0),
                 lambda: vce.ce_rms_norm_quant(x, w, group=48), lambda: vce.ce_rms_norm_quant(x, w, out=x),
                 lambda: vce.ce_rms_norm_quant(x, w, scales=w[:3]),
                 lambda: vce.ce_rms_norm_backward(None, x, w), lambda: vce.ce_rms_norm_backward(x[:3], x, w),
                 lambda: vce.ce_rms_norm_backward(x, x, w, dsum=x.bfloat16()),
                 lambda: vce.ce_rms_norm_backward(x, x, w, dweight=w[:5]),
                 lambda: vce.ce_rms_norm_backward(x, x, w, accumulate=True),
                 lambda: vce.ce_rms_norm_backward(x, x, w, ws=torch.empty(1, dtype=torch.uint8, device="cuda")),
                 lambda: vce.ce_rms_norm(torch.ones((1, 32769), device="cuda"), torch.ones(32769, device="cuda")),
                 lambda: vce.rms_norm(x, w, x[:3])):
        with pytest.raises(vce.CeArgumentError):
            call()


def test_no_rows():
    w = torch.ones(12, device="cuda")
    e = torch.empty((0, 12), device="cuda")
    y, s = vce.ce_rms_norm(e, w, e)
    assert y.shape == (0, 12) and s.shape == (0, 12)
    q, sc, _ = vce.ce_rms_norm_quant(e, w, group=32)
    assert q.shape == (0, 12) and sc.shape == (0, 1)
    dx, dw = vce.ce_rms_norm_backward(e, e, w, dsum=e)
    assert dx.shape == (0, 12) and not dw.any()
    kept = torch.full((12,), 4.0, device="cuda")
    vce.ce_rms_norm_backward(e, e, w, dweight=kept, accumulate=True)
    assert (kept == 4).all()


def test_autograd_forms():
    """rms_norm against torch in 64 bits: both outputs used, either alone, an expanded gradient, 3-d inputs."""
    shape = (2, 3, 130)
    x, r, w = _rand(shape, torch.float32, 1), _rand(shape, torch.float32, 2), _rand((130,), torch.float32, 3)
    c, e = _rand(shape, torch.float32, 4), _rand(shape, torch.float32, 5)
    for use in ("both", "y", "sum", "ones", "plain"):
        say(f"[norm] autograd {use}")
        ref = [t.double().requires_grad_() for t in (x, r, w)]
        dev = [t.cuda().requires_grad_() for t in (x, r, w)]

        def loss(y, s, c, e):
            return {"both": lambda: (y * c).sum() + (s * e).sum(), "y": lambda: (y * c).sum(),
                    "sum": lambda: (s * e).sum(), "ones": lambda: y.sum(), "plain": lambda: (y * c).sum()}[use]()

        s64 = ref[0] + ref[1] if use != "plain" else ref[0]
        y64 = s64 * torch.rsqrt(s64.square().mean(-1, keepdim=True) + np.float64(np.float32(1e-6))) * ref[2]
        loss(y64, s64, c.double(), e.double()).backward()
        got = vce.rms_norm(dev[0], dev[2], dev[1] if use != "plain" else None)
        y, s = got if use != "plain" else (got, None)
        loss(y, s, c.cuda(), e.cuda()).backward()
        for name, a, b in zip("x residual weight".split(), dev, ref):
            if b.grad is None:
                assert a.grad is None or not a.grad.any(), (use, name)
            else:
                g = f64(b.grad)
                # the FP32 sum s rounds by U, which moves each term by as much: the largest term bounds the budget
                assert_within(f64(a.grad), g, 200 * U * (np.abs(g) + np.abs(g).max()), f"{use} {name}")


def test_expanded_inputs():
    """A residual (and an input) broadcast over the rows: the same values, and their gradients summed."""
    x, r, w = _rand((5, 40), torch.float32, 1), _rand((40,), torch.float32, 2), _rand((40,), torch.float32, 3)
    c = _rand((5, 40), torch.float32, 4).cuda()
    for swap in (False, True):
        grads = []
        for dense in (False, True):
            xd, rd = x.cuda().requires_grad_(), r.cuda().requires_grad_()
            re = rd.expand(5, 40).contiguous() if dense else rd.expand(5, 40)
            y, s = vce.rms_norm(re, w.cuda(), xd) if swap else vce.rms_norm(xd, w.cuda(), re)
            ((y + s) * c).sum().backward()
            grads.append((y.detach(), xd.grad, rd.grad))
        for a, b in zip(*grads):
            assert torch.equal(a, b)
    one = vce.rms_norm(r.cuda().expand(3, 40), w.cuda())
    assert torch.equal(one[0], one[2])


def test_gradient_against_differences():
    N, D = 4, 96
    s, w, c = _rand((N, D), torch.float32, 1), _rand((D,), torch.float32, 2), _rand((N, D), torch.float32, 3)
    v, u = _rand((N, D), torch.float64, 4), _rand((D,), torch.float64, 5)
    dx, dw = vce.ce_rms_norm_backward(c.cuda(), s.cuda(), w.cuda(), 1e-5)
    h = 1e-6
    f = lambda a, b: (ref_norm(a, None, b, np.float64(np.float32(1e-5)))[0] * f64(c)).sum()  # noqa: E731
    S, W = f64(s), f64(w)
    num_x = (f(S + h * f64(v), W) - f(S - h * f64(v), W)) / (2 * h)
    num_w = (f(S, W + h * f64(u)) - f(S, W - h * f64(u))) / (2 * h)
    # the differences' own error: h^2 of third derivatives, and 1e-16 / h of the value
    for got, num, size in (((f64(dx) * f64(v)).sum(), num_x, np.abs(f64(dx) * f64(v)).sum()),
                           ((f64(dw) * f64(u)).sum(), num_w, np.abs(f64(dw) * f64(u)).sum())):
        assert abs(got - num) <= 1e-5 * size, (got, num, size)


def test_graph_replays_and_streams():
    N, D = 37, 4096
    x, r, w = _rand((N, D), torch.bfloat16, 1).cuda(), _rand((N, D), torch.bfloat16, 2).cuda(), torch.ones(D).cuda()
    ws = torch.empty(vce.ce_rms_norm_workspace_bytes(N, D), dtype=torch.uint8, device="cuda")
    y, s, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    q, sc = torch.empty((N, D), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((N, 32), device="cuda")
    dw = torch.empty(D, device="cuda")
    outs = [y, s, dx, q.view(torch.uint8), sc, dw]

    def run():
        vce.ce_rms_norm(x, w, r, out=y, sum_out=s)
        vce.ce_rms_norm_quant(x, w, r, group=128, out=q, scales=sc)
        vce.ce_rms_norm_backward(y, s, w, dsum=r, dx=dx, dweight=dw, ws=ws)

    say("[norm] graph")
    run()
    torch.cuda.synchronize()
    ref = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    torch.cuda.synchronize()
    for rep in range(4):
        for o in outs:
            o.zero_()
        ws.fill_(rep * 85)
        graph.replay()
        torch.cuda.synchronize()
        for o, k in zip(outs, ref):
            assert torch.equal(o, k), rep
        if rep == 1:
            with torch.cuda.stream(side):
                run()
            torch.cuda.synchronize()


def test_training_step_of_a_tied_model():
    """Embedding, a residual, the final norm, the head and the loss, with one table for both ends: the loss and
    every gradient against torch in 64 bits; and the same step with one FP32 buffer for the table's gradient."""
    N, V, D = 60, 211, 72
    table, nw = _rand((V, D), torch.float32, 1, 0.3), 1 + _rand((D,), torch.float32, 2, 0.1)
    ids = (torch.rand(N, generator=_gen(3)) ** 3 * V).long()
    t = torch.randint(0, V, (N,), generator=_gen(4))
    t[5] = -100
    r = _rand((N, D), torch.float32, 5)
    leaves = [a.double().requires_grad_() for a in (table, nw, r)]
    s = torch.nn.functional.embedding(ids, leaves[0]) * 2.0 + leaves[2]
    y = s * torch.rsqrt(s.square().mean(1, keepdim=True) + np.float64(np.float32(1e-6))) * leaves[1]
    ref = torch.nn.functional.cross_entropy(y @ leaves[0].t(), t, ignore_index=-100)
    ref.backward()
    dev = [a.cuda().requires_grad_() for a in (table, nw, r)]
    say("[training step] tied")
    loss = vce.norm_linear_cross_entropy(vce.embedding(ids.cuda(), dev[0], 2.0), dev[1], dev[0], t.cuda(),
                                         residual=dev[2])
    loss.backward()
    assert abs(loss.item() - ref.item()) <= 1e-4 * max(1, abs(ref.item()))
    # sums of V, N and D terms in FP32 along the step: their roundings, of the largest entry
    tol = (V + N + D + 200) * U
    for name, a, b in zip(("table", "norm weight", "residual"), dev, leaves):
        g = f64(b.grad)
        assert_within(f64(a.grad), g, tol * (np.abs(g) + np.abs(g).max()), name)
    # one buffer: the head adds its dw, the embedding's backward adds to it
    buf = torch.zeros((V, D), device="cuda")
    w, h = table.cuda().requires_grad_(), None
    h = vce.embedding(ids.cuda(), w, 2.0, grad_buffer=buf)
    yd = vce.rms_norm(h, nw.cuda(), r.cuda())[0]
    _, dh, _, _ = vce.ce_linear_cross_entropy(yd.detach(), table.cuda(), t.cuda(), reduce_loss="mean", dw=buf,
                                              accumulate_dw=True)
    yd.backward(dh)
    g = f64(leaves[0].grad)
    assert w.grad is None
    assert_within(f64(buf), g, tol * (np.abs(g) + np.abs(g).max()), "one buffer")


# rows whose 1 / rms is far from 1: its cube passes FP32's range where the inputs and the gradient do not
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("N,D", [(5, 24), (3, 777), (3, 4096), (2, 8200), (2, 16392)])
@pytest.mark.parametrize("rms,eps", [(1e-14, 0.0), (1e-14, 1e-30), (1e13, 1e-6), (1e14, 1e-6), (1e17, 1e-6)])
def test_backward_of_tiny_and_huge_rows(rms, eps, N, D, dtype):
    """dy correlated with s, so that the mean's term is as large as the other; a row of zeros where eps allows one."""
    s = _rand((N, D), torch.float32, D, rms)
    dy = (_rand((N, D), torch.float32, D + 1) + s / rms).to(dtype)
    if rms < 1 and eps:
        s[1] = 0
    s, w = s.to(dtype), _rand((D,), torch.float32, 3)
    say(f"[norm grad] rms {rms} eps {eps} {N} {D} {dtype}")
    dx, dw = vce.ce_rms_norm_backward(dy.cuda(), s.cuda(), w.cuda(), eps)
    rx, rw, bx, bw = ref_norm_grad(f64(dy), f64(s), f64(w), np.float64(np.float32(eps)), None)
    assert_within(f64(dx), rx, bx + half_step(dtype) * 1.01 * np.abs(rx), "dx")
    assert_within(f64(dw), rw, bw, "dweight")


def _border_weights(cols, lead, seed):
    """``cols`` values whose quotients by the scale of their largest, ``lead``, lie within two FP32 steps of a border
    between e4m3 values; the first is ``lead``."""
    grid = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double()  # 0 .. 448
    scale = np.float32(lead) / np.float32(448)
    g = _gen(seed)
    at = ((grid[1:] + grid[:-1]) / 2)[torch.randint(0, 126, (cols,), generator=g)]
    w = (at * float(scale)).float()
    w = (w.view(torch.int32) + torch.randint(-2, 3, (cols,), generator=g, dtype=torch.int32)).view(torch.float32)
    w = w * (torch.randint(0, 2, (cols,), generator=g) * 2 - 1)
    w[0] = lead
    return w


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [640, 4096, 8192, 16512])
@pytest.mark.parametrize("group", [0, 32, 128])
def test_quantised_at_the_borders(group, D, dtype):
    """Rows of +-1 at eps 0 have 1 / rms = 1 exactly, so y is the weight: q is the value nearest to the FP32 quotient
    y / scale, bit for bit, also where that lies next to a border between two of the type's values."""
    N, G = 3, group or D
    leads = torch.rand(D // G, generator=_gen(D)).add_(0.5).mul_(100.0).tolist()
    w = torch.cat([_border_weights(G, lead, D + k) for k, lead in enumerate(leads)])
    x = (torch.randint(0, 2, (N, D), generator=_gen(group + 1)) * 2 - 1).to(dtype)
    y = x.float() * w
    scale = y.view(N, -1, G).abs().amax(2) / 448
    want = (y.view(N, -1, G) / scale.unsqueeze(2)).view(N, D).to(torch.float8_e4m3fn)
    say(f"[norm e4m3] borders {group} {D} {dtype}")
    q, scales, _ = vce.ce_rms_norm_quant(x.cuda(), w.cuda(), eps=0.0, group=group)
    assert torch.equal(scales.cpu(), scale)
    assert torch.equal(q.cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("D", [640, 16512])
@pytest.mark.parametrize("group", [0, 128])
def test_quantised_extremes(group, D):
    """The quotient at the ends of the range: an infinite y (its scale is infinite, the others' quotients 0 with their
    signs), y near FP32's largest, zeros of both signs, and y below the smallest scale."""
    G = group or D
    w = torch.ones(D)
    x = torch.ones((4, D))
    x[:, 3::7] = -1
    for name, lead, fill in (("infinite", float("inf"), 2.0), ("largest", 3.3e38, 1.1e38), ("zero", 0.0, 0.0),
                             ("tiny", 2.0 ** -126, 2.0 ** -130)):
        w[:G] = fill
        w[5] = lead
        y = x * w
        scale = (y.view(4, -1, G).abs().amax(2) / 448).clamp(min=2.0 ** -126)
        want = (y.view(4, -1, G) / scale.unsqueeze(2)).view(4, D).to(torch.float8_e4m3fn)
        say(f"[norm e4m3] {name} {group} {D}")
        q, scales, _ = vce.ce_rms_norm_quant(x.cuda(), w.cuda(), eps=0.0, group=group)
        assert torch.equal(scales.cpu(), scale), name
        got, nan = q.cpu().view(torch.uint8), torch.isnan(want.float())
        assert torch.equal(torch.isnan(q.cpu().float()), nan) and bool(nan.any()) == (name == "infinite")
        assert torch.equal(got[~nan], want.view(torch.uint8)[~nan]), name


@pytest.mark.parametrize("N,D", [(5, 96), (4, 2000), (2, 16392)])
def test_buffers_shared_without_overlap(N, D):
    """Inputs and outputs side by side or in turn in one buffer, and the gradient over the sum's own rows: the same
    bits as in buffers of their own.  Rows that meet are refused and left as they are."""
    for dtype in DTYPES:
        x, r, w = _rand((N, D), dtype, 1).cuda(), _rand((N, D), dtype, 2).cuda(), _rand((D,), dtype, 3).cuda()
        y, s = vce.ce_rms_norm(x, w, r)
        dx, dw = vce.ce_rms_norm_backward(r, s, w, dsum=x)
        say(f"[norm] shared buffers {N} {D} {dtype}")
        for side in (True, False):
            b = torch.empty((N, 4, D) if side else (4 * N, D), dtype=dtype, device="cuda")
            xs, rs, ys, ss = (b[:, k] for k in range(4)) if side else (b[k::4] for k in range(4))
            xs.copy_(x), rs.copy_(r)
            vce.ce_rms_norm(xs, w, rs, out=ys, sum_out=ss)
            assert torch.equal(ys, y) and torch.equal(ss, s) and torch.equal(xs, x) and torch.equal(rs, r)
            got, gw = vce.ce_rms_norm_backward(rs, ss, w, dsum=xs, dx=ss)
            assert got is ss and torch.equal(ss, dx) and torch.equal(gw, dw) and torch.equal(xs, x)
        b = torch.zeros(2 * N * D + D, dtype=dtype, device="cuda")
        a = b[:N * D].view(N, D)
        a.copy_(x)
        wide = b[:2 * N * D].view(N, 2 * D)[:, :D]
        before = b.clone()
        for call in (lambda: vce.ce_rms_norm(a, w, out=wide), lambda: vce.ce_rms_norm(a, w, out=b[D:D + N * D].view(N, D)),
                     lambda: vce.ce_rms_norm(a, w, r, out=y, sum_out=y), lambda: vce.ce_rms_norm(a, w, r, sum_out=wide),
                     lambda: vce.ce_rms_norm(r, w, a, out=b[1:1 + N * D].view(N, D)),
                     lambda: vce.ce_rms_norm_quant(a, w, out=b.view(torch.float8_e4m3fn)[:N * D].view(N, D)),
                     lambda: vce.ce_rms_norm_backward(a, x, w, dx=wide), lambda: vce.ce_rms_norm_backward(x, a, w, dx=wide),
                     lambda: vce.ce_rms_norm_backward(x, x, w, dsum=a, dx=b[D:D + N * D].view(N, D))):
            with pytest.raises(vce.CeArgumentError, match="overlaps"):
                call()
        assert torch.equal(b, before)


# several rows for each workgroup and a ragged last round: prefetched rows, alternating exchange buffers, dw over rows
ROUNDS = [(4099, 24), (4200, 1000), (1030, 2048), (515, 4096), (515, 2731), (300, 8200), (259, 16384), (258, 16392)]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("N,D", ROUNDS)
def test_backward_of_several_rounds(N, D, dtype):
    test_backward(N, D, dtype)
    # and over the sum's own rows
    s, dy, w = _rand((N, D), dtype, D).cuda(), _rand((N, D), dtype, D + 1).cuda(), _rand((D,), dtype, 3).cuda()
    dx, dw = vce.ce_rms_norm_backward(dy, s, w)
    over, dw2 = vce.ce_rms_norm_backward(dy, s, w, dx=s)
    assert over is s and torch.equal(over, dx) and torch.equal(dw2, dw)


def _rows_of_a_batch(x, r, w, parts, group):
    """The forward calls over a whole batch and over parts of its rows: a row's outputs do not depend on the others."""
    y, s = vce.ce_rms_norm(x, w, r)
    q, sc, s2 = vce.ce_rms_norm_quant(x, w, r, group=group)
    assert torch.equal(s, s2)
    for a, b in parts:
        yp, sp = vce.ce_rms_norm(x[a:b], w, r[a:b])
        qp, scp, _ = vce.ce_rms_norm_quant(x[a:b], w, r[a:b], group=group)
        assert torch.equal(y[a:b], yp) and torch.equal(s[a:b], sp), (a, b)
        assert torch.equal(q[a:b].view(torch.uint8), qp.view(torch.uint8)) and torch.equal(sc[a:b], scp), (a, b)
    return y, s, q


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("N,D,group", [(4100, 4096, 128), (1030, 16384, 0), (40000, 448, 32), (8200, 2048, 64)])
def test_outputs_larger_than_the_caches(N, D, group, dtype):
    """More than 32 MiB in an output, which the kernels write past the caches."""
    g = torch.Generator("cuda").manual_seed(N)
    x, r = (torch.randn((N, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    w = _rand((D,), torch.float32, 3).cuda()
    say(f"[norm] large {N} {D} {dtype} {group}")
    step = (8 << 20) // D
    y, s, _ = _rows_of_a_batch(x, r, w, [(a, min(a + step, N)) for a in range(0, N, step)], group)
    pick = torch.tensor([0, 1, N // 2, N - 2, N - 1])
    ref, total, _ = ref_norm(f64(x[pick]), f64(r[pick]), f64(w), np.float64(np.float32(1e-6)))
    assert_within(f64(y[pick]), ref, _y_tol(ref, dtype), "y")
    assert_within(f64(s[pick]), total, (half_step(dtype) * 1.01 + U) * np.abs(total) + TINY, "sum")


@pytest.mark.parametrize("N,D,group", [((1 << 23) + 4003, 8, 0), ((1 << 23) + 4003, 40, 32), ((1 << 21) + 503, 1032, 0)])
def test_more_rows_than_one_launch_holds(N, D, group):
    """Workgroups that take a second row (2^21 of them in a launch, four narrow rows each)."""
    g = torch.Generator("cuda").manual_seed(D)
    x, r = (torch.randn((N, D), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = _rand((D,), torch.float32, 3).cuda()
    say(f"[norm] {N} rows of {D}")
    last = (1 << 21) * (4 if D <= 1024 else 1)
    _rows_of_a_batch(x, r, w, [(0, 4100), (last - 300, last), (last, N)], group)
