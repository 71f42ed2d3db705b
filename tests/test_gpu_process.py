"""Logit processing and its gradient against the 64-bit definition."""
import ctypes

import numpy as np
import pytest
import torch

import vocab_cross_entropy_amd as vce
from gpu_util import say
from vocab_cross_entropy_amd import _abi
from ops_util import (U, allowed_columns, assert_within, f64, half_step, history_counts, ref_process,
                      ref_process_grad)

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _inputs(d0, d1, V, dtype, L, seed, prompt=True, prefix=False):
    """CPU inputs; a few hot tokens, some ids outside the vocabulary, lengths from 0 past the buffer's width."""
    g = _gen(seed)
    N = d0 * d1
    s = dict(x=(torch.randn((d0, d1, V), generator=g) * 3).to(dtype))
    if L is not None:
        rows = (d0, 1, L) if prefix else (d0, d1, L)
        h = (torch.rand(rows, generator=g) ** 3 * V).long().clamp(max=V - 1)
        bad = torch.rand(rows, generator=g)
        h[bad < 0.03] = -1
        h[(bad >= 0.03) & (bad < 0.05)] = V
        h[(bad >= 0.05) & (bad < 0.06)] = -2 ** 63
        h[(bad >= 0.06) & (bad < 0.07)] = 2 ** 62 + 5
        s["history"] = h.expand(d0, d1, L)
        n = torch.randint(0, L + 1, (N,), generator=g, dtype=torch.int32)
        n[0] = L + 7  # taken as L
        if N > 1:
            n[1] = 0
        if N > 2:
            n[2] = -4  # taken as 0
        s["history_len"] = torch.arange(N, dtype=torch.int32) % (L + 1) if prefix else n
        s["prompt_len"] = torch.randint(0, L + 3, (N,), generator=g, dtype=torch.int32) if prompt else None
        s["repetition"] = torch.rand(N, generator=g) + 0.7
        s["frequency"] = torch.rand(N, generator=g) - 0.3
        s["presence"] = torch.rand(N, generator=g) - 0.3
    s["temperature"] = torch.rand(N, generator=g) + 0.4
    return s


def _mask(d0, d1, V, seed, empty_row=True):
    m = torch.randint(-2 ** 31, 2 ** 31, (d0, d1, (V + 31) // 32), generator=_gen(seed), dtype=torch.int64)
    m = m.to(torch.int32)
    if empty_row:
        m[-1, -1] = 0
    return m


def _dev(s):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) and k != "history" else v) for k, v in s.items()} | (
        {"history": s["history"][:, :1].cuda().expand(s["history"].shape)
         if s["history"].stride(1) == 0 else s["history"].cuda()} if s.get("history") is not None else {})


def _reference(s, vocab_start=0):
    d0, d1, V = s["x"].shape
    N = d0 * d1
    h = s.get("history")
    seen, cnt = history_counts(None if h is None else h.reshape(N, -1).numpy(), s.get("history_len"),
                               s.get("prompt_len"), N, V, vocab_start)
    allowed = None if s.get("mask") is None else allowed_columns(s["mask"].reshape(N, -1).numpy(), V)
    b = s.get("bias")
    get = lambda k: None if s.get(k) is None else f64(s[k])  # noqa: E731
    z, budget = ref_process(f64(s["x"]).reshape(N, V), seen, cnt, get("repetition"), get("frequency"),
                            get("presence"), None if b is None else f64(b).reshape(N, V), get("temperature"), allowed)
    return z, budget, seen, allowed


def _call(s, **kw):
    steps = {k: v for k, v in s.items() if k != "x"}
    return vce.ce_logits_process(s["x"], **steps, **kw)


def _check(z, ref, budget, dtype, what):
    assert_within(f64(z).reshape(ref.shape), ref, budget + half_step(dtype) * np.abs(ref) * 1.01, what)


SHAPES = [(1, 1, 1, 1), (1, 1, 7, 5), (2, 3, 8, 9), (3, 1, 33, 64), (1, 5, 1000, 300), (2, 2, 8191, 700),
          (1, 3, 8193, 257), (2, 1, 20011, 3000)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("form", ["all", "no_prompt", "mask_only", "temperature_only", "bias_shared"])
def test_process_matches_definition(shape, dtype, form):
    d0, d1, V, L = shape
    say(f"[process] {shape} {dtype} {form}")
    s = _inputs(d0, d1, V, dtype, L if form in ("all", "no_prompt") else None, seed=V + L, prompt=form == "all")
    if form in ("all", "mask_only"):
        s["mask"] = _mask(d0, d1, V, seed=V)
    if form == "all":
        s["bias"] = torch.randn((d0, d1, V), generator=_gen(V))
    if form == "bias_shared":
        s["bias"] = torch.randn(V, generator=_gen(V)).expand(d0, d1, V)
    z, budget, _, allowed = _reference(s)
    d = _dev(s)
    if form == "bias_shared":
        d["bias"] = s["bias"][0, 0].cuda().expand(d0, d1, V)
    signs = vce.logits_signs(d["x"]).fill_(255)
    out = _call(d, out=torch.empty_like(d["x"]), signs=signs)
    torch.cuda.synchronize()
    _check(out, z, budget, dtype, f"{form} {shape}")
    if allowed is not None:
        assert np.isneginf(f64(out).reshape(z.shape)[-1]).all()
    up = np.unpackbits(signs.cpu().numpy(), axis=1, bitorder="little")
    assert np.array_equal(up[:, :V] != 0, f64(s["x"]).reshape(z.shape) > 0) and not up[:, V:].any()
    # in place, and the same bits on a repeat
    inplace = _call(d)
    assert inplace is d["x"]
    kind = torch.int16 if dtype == torch.bfloat16 else torch.int32
    assert torch.equal(inplace.view(kind), out.view(kind))


def test_history_of_more_than_32767_tokens():
    """Counts beyond 15 bits, at one column, and a long prompt."""
    V, L = 5003, 70001
    s = _inputs(1, 2, V, torch.float32, L, seed=5)
    s["history"] = s["history"].clone()
    s["history"][0, 0, ::2] = 17
    s["history_len"] = torch.tensor([L, L - 1], dtype=torch.int32)
    s["prompt_len"] = torch.tensor([3, 40000], dtype=torch.int32)
    z, budget, _, _ = _reference(s)
    say("[process] 70001 tokens")
    _check(_call(_dev(s), out=torch.empty((1, 2, V), device="cuda")), z, budget, torch.float32, "long history")


@pytest.mark.parametrize("L", [32767, 32768])
def test_one_token_fills_the_history(L):
    """Every token the same: the largest count of either width, beside flagged neighbours."""
    V = 64
    s = _inputs(1, 1, V, torch.float32, L, seed=L)
    s["history"] = torch.full((1, 1, L), 20)
    s["history"][0, 0, 0], s["history"][0, 0, 1] = 19, 21
    s["history_len"], s["prompt_len"] = torch.tensor([L], dtype=torch.int32), torch.tensor([2], dtype=torch.int32)
    z, budget, _, _ = _reference(s)
    say(f"[process] one token, {L}")
    _check(_call(_dev(s), out=torch.empty((1, 1, V), device="cuda")), z, budget, torch.float32, "one token")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_strides_offsets_and_prefix_histories(dtype):
    """The transposed view, rows at odd addresses inside a wider buffer, histories shared by a sequence's rows."""
    d0, d1, V, L = 3, 5, 1237, 11
    s = _inputs(d0, d1, V, dtype, L, seed=9, prefix=True)
    s["mask"] = _mask(d0, d1, V, seed=10)
    z, budget, _, _ = _reference(s)
    wide = torch.full((d1, d0, V + 5), 7.0, dtype=dtype, device="cuda")
    view = wide[:, :, 3:3 + V].transpose(0, 1)
    view.copy_(s["x"].cuda())
    wide_out = torch.full((d0, d1 + 1, V + 9), 7.0, dtype=dtype, device="cuda")
    out = wide_out[:, :d1, 1:1 + V]
    d = _dev(s)
    wide_mask = torch.zeros((d0, d1, s["mask"].shape[2] + 3), dtype=torch.int32, device="cuda")
    wide_mask[..., :-3] = d["mask"]
    d["mask"], d["x"] = wide_mask[..., :-3], view
    say(f"[process] strides {dtype}")
    _call(d, out=out)
    _check(out, z, budget, dtype, "strided")
    _call(d)
    _check(view, z, budget, dtype, "strided, in place")
    for buf, inner in ((wide, wide[:, :, 3:3 + V]), (wide_out, out)):
        outside = torch.ones(buf.shape, dtype=torch.bool, device="cuda")
        if buf is wide:
            outside[:, :, 3:3 + V] = False
        else:
            outside[:, :d1, 1:1 + V] = False
        assert (buf[outside] == 7.0).all(), "written outside the rows"


def test_vocabulary_shards_agree_with_the_whole():
    d0, d1, V, L = 2, 2, 3001, 200
    s = _inputs(d0, d1, V, torch.float32, L, seed=13)
    s["mask"] = _mask(d0, d1, V, seed=14)
    d = _dev(s)
    whole = _call(d, out=torch.empty_like(d["x"]))
    cut = 1024  # a multiple of 32, so that a shard's mask is a slice of words
    say("[process] shards")
    for lo, hi in ((0, cut), (cut, V)):
        part = dict(d, x=d["x"][..., lo:hi].contiguous(), mask=d["mask"][..., lo // 32:])
        z = _call(part, out=torch.empty_like(part["x"]), vocab_start=lo, vocab_total=V)
        assert torch.equal(z, whole[..., lo:hi])


def test_infinities_and_nan():
    """-inf stays -inf, NaN stays NaN where allowed and goes where masked; the type's lowest value is a value."""
    V = 64
    x = torch.zeros((1, 2, V))
    x[..., 0], x[..., 1], x[..., 2], x[..., 3] = -np.inf, np.nan, torch.finfo(torch.float32).min, np.inf
    mask = torch.full((1, 2, 2), -1, dtype=torch.int32)
    mask[0, 1] = ~0xf  # the first four columns of each word
    h = torch.tensor([0, 1, 2, 3, 2]).expand(1, 2, 5)
    for dtype in (torch.float32, torch.bfloat16):
        say(f"[process] infinities {dtype}")
        z = vce.ce_logits_process(x.to("cuda", dtype), history=h.cuda(), repetition=torch.full((2,), 0.5).cuda(),
                                  mask=mask.cuda(), temperature=torch.full((2,), 2.0).cuda())
        z = f64(z)[0]
        low = float(x.to(dtype)[0, 0, 2])
        assert z[0, 0] == -np.inf and np.isnan(z[0, 1]) and z[0, 2] == low * 0.25 and z[0, 3] == np.inf
        masked = np.arange(V) % 32 < 4
        assert (z[1, masked] == -np.inf).all() and (z[1, ~masked] == 0).all() and (z[0, 4:] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward_matches_definition(shape, dtype):
    d0, d1, V, L = shape
    N = d0 * d1
    say(f"[process backward] {shape} {dtype}")
    s = _inputs(d0, d1, V, dtype, L, seed=V * 3 + L)
    s["mask"] = _mask(d0, d1, V, seed=V)
    _, _, seen, allowed = _reference(s)
    d = _dev(s)
    signs = vce.logits_signs(d["x"])
    _call(d, out=torch.empty_like(d["x"]), signs=signs)
    dz = torch.randn((d0, d1, V), generator=_gen(V)).to(dtype)
    ref = ref_process_grad(f64(dz).reshape(N, V), f64(s["x"]).reshape(N, V) > 0, seen, f64(s["repetition"]),
                           f64(s["temperature"]), allowed)
    dz[~torch.from_numpy(allowed).view(d0, d1, V)] = float("nan")  # what reaches a masked column does not matter
    dzd = dz.cuda()
    keep = {k: d[k] for k in ("history", "history_len", "prompt_len", "repetition", "mask", "temperature")}
    dx = vce.ce_logits_process_backward(dzd, out=torch.empty_like(dzd), signs=signs, **keep)
    assert_within(f64(dx).reshape(N, V), ref, (3.03 * U + half_step(dtype)) * np.abs(ref) + 1e-37, "dx")
    vce.ce_logits_process_backward(dzd, signs=signs, **keep)
    kind = torch.int16 if dtype == torch.bfloat16 else torch.int32
    assert torch.equal(dzd.view(kind), dx.view(kind))
    assert not dx.view(kind)[~torch.from_numpy(allowed).view(d0, d1, V).cuda()].any(), "masked columns must be +0.0"


def test_gradient_against_differences():
    """Central differences of the 64-bit definition along a random direction, away from x = 0."""
    d0, d1, V, L = 1, 3, 501, 120
    s = _inputs(d0, d1, V, torch.float32, L, seed=21)
    s["x"] = torch.where(s["x"].abs() < 0.05, torch.full_like(s["x"], 0.05), s["x"])
    x = s["x"].cuda().requires_grad_()
    d = _dev(s)
    c = torch.randn((d0, d1, V), generator=_gen(3))
    say("[process] differences")
    z = vce.process_logits(x, **{k: v for k, v in d.items() if k != "x"})
    (z * c.cuda()).sum().backward()
    step = 1e-3
    v = torch.randn((d0, d1, V), generator=_gen(4))
    vals = []
    for sign in (1, -1):
        shifted = dict(s, x=s["x"].double() + sign * step * v.double())
        vals.append((_reference(shifted)[0] * f64(c).reshape(3, V)).sum())
    num = (vals[0] - vals[1]) / (2 * step)  # the map is linear between sign changes: differences are exact
    got = (f64(x.grad) * f64(v)).sum()
    size = np.abs(f64(x.grad) * f64(v)).sum()
    assert abs(got - num) <= 4 * U * size + 1e-9 * size, (got, num)


def test_process_logits_leaves_its_input_and_takes_any_gradient():
    s = _dev(_inputs(2, 3, 300, torch.bfloat16, 40, seed=2))
    x = s["x"].requires_grad_()
    before = x.detach().clone()
    steps = {k: v for k, v in s.items() if k != "x"}
    say("[process] autograd")
    z = vce.process_logits(x, **steps)
    z.sum().backward()  # an expanded gradient: stride 0
    assert torch.equal(x.detach(), before)
    first, x.grad = x.grad, None
    z = vce.process_logits(x, **steps)
    z.backward(torch.ones_like(z))
    assert torch.equal(first, x.grad)
    z = vce.process_logits(x.transpose(0, 1), temperature=steps["temperature"])
    assert z.shape == (3, 2, 300)
    wide = vce.process_logits(x[:1].expand(2, 3, 300), temperature=steps["temperature"])
    assert torch.equal(wide[1], vce.process_logits(x[:1], temperature=steps["temperature"][3:])[0])


def test_processed_cross_entropy_refuses_before_it_writes():
    s = _dev(_inputs(2, 3, 70, torch.float32, 10, seed=1))
    x, before = s.pop("x"), None
    before = x.clone()
    good = torch.zeros((2, 3), dtype=torch.int64, device="cuda")
    for target, kw in ((good[:1], {}), (good.int(), {}), (good.cpu(), {}), (None, {}), (good, dict(label_smoothing=2.0)),
                       (good, dict(smoothing="some")), (good, dict(reduce_loss="avg"))):
        with pytest.raises(vce.CeArgumentError):
            vce.processed_cross_entropy(x, target, **kw, **s)
    assert torch.equal(x, before)


def test_tokens_past_the_length_are_not_read():
    """Rows of a history laid end to end: the last row's tokens end with the buffer, its width is another row's."""
    V = 100
    flat = torch.randint(0, V, (13,), generator=_gen(1)).cuda()  # (torch refuses the view: the C descriptor allows it)
    x = torch.randn((1, 2, V), generator=_gen(2)).cuda()
    want = x.clone()
    n = torch.tensor([10, 3], dtype=torch.int32).cuda()
    pen = torch.full((2,), 0.5, device="cuda")
    xd = vce.logits_desc(x)
    p = _abi.CeProcess(flat.data_ptr(), 0, 10, 10, n.data_ptr(), None, None, pen.data_ptr(), None, None, None, 0, 0,
                       None, 0, 0, None, 0)
    say("[process] rows end to end")
    assert vce.lib.ce_logits_process(ctypes.byref(xd), ctypes.byref(xd), ctypes.byref(p),
                                     torch.cuda.current_stream().cuda_stream) == 0
    for r, tokens in ((0, flat[:10]), (1, flat[10:])):
        want[0, r] -= 0.5 * torch.bincount(tokens, minlength=V)
    assert torch.allclose(x, want, rtol=0, atol=1e-6)


@pytest.mark.parametrize("reduce", ["none", "mean", "sum"])
def test_processed_cross_entropy(reduce):
    """processed_cross_entropy against torch in 64 bits, through the same definition."""
    d0, d1, V, L = 2, 4, 2003, 150
    s = _inputs(d0, d1, V, torch.float32, L, seed=31)
    s["mask"] = _mask(d0, d1, V, seed=32, empty_row=False)
    t = torch.randint(0, V, (d0, d1), generator=_gen(33))
    allowed = torch.from_numpy(allowed_columns(s["mask"].reshape(8, -1).numpy(), V)).view(d0, d1, V)
    for i in range(d0):  # targets that the mask allows, as sampled tokens are
        for j in range(d1):
            t[i, j] = torch.nonzero(allowed[i, j])[int(t[i, j]) % int(allowed[i, j].sum())]
    t[1, 2] = -100
    _, _, seen, _ = _reference(s)
    N = d0 * d1
    seen = torch.from_numpy(seen).view(d0, d1, V)
    cnt = torch.from_numpy(history_counts(s["history"].reshape(N, -1).numpy(), s["history_len"], s["prompt_len"], N,
                                          V)[1]).view(d0, d1, V)
    xr = s["x"].double().requires_grad_()
    row = lambda k: s[k].double().view(d0, d1, 1)  # noqa: E731
    zr = torch.where(seen, torch.where(xr > 0, xr / row("repetition"), xr * row("repetition")), xr)
    zr = (zr - row("frequency") * cnt - row("presence") * (cnt > 0)) / row("temperature")
    zr = torch.where(allowed, zr, -torch.inf)
    ref = torch.nn.functional.cross_entropy(zr.view(-1, V), t.view(-1), reduction=reduce, ignore_index=-100)
    up = torch.rand(ref.shape, generator=_gen(34), dtype=torch.float64) + 0.5
    ref.backward(up)
    d = _dev(s)
    x = d["x"].requires_grad_()
    say(f"[processed cross-entropy] {reduce}")
    loss = vce.processed_cross_entropy(x, t.cuda(), reduce_loss=reduce, **{k: v for k, v in d.items() if k != "x"})
    loss.backward(up.to("cuda", torch.float32).view(loss.shape))
    assert_within(f64(loss).reshape(-1), f64(ref).reshape(-1), 1e-4 * np.maximum(1, np.abs(f64(ref).reshape(-1))), "loss")
    g = f64(xr.grad)
    assert_within(f64(x.grad), g, 2e-5 * np.abs(g) + 1e-7, "gradient")
    assert not x.grad[1, 2].view(torch.int32).any(), "an ignored row's gradient must be +0.0"


def test_graph_replays_and_streams():
    """Captured forward and backward, replayed among eager calls, and eager calls on another stream."""
    s = _dev(_inputs(3, 2, 9001, torch.bfloat16, 500, seed=41))
    s["mask"] = _mask(3, 2, 9001, seed=42).cuda()
    out, dx = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    signs = vce.logits_signs(s["x"])
    keep = {k: s[k] for k in ("history", "history_len", "prompt_len", "repetition", "mask", "temperature")}

    def run():
        _call(s, out=out, signs=signs)
        vce.ce_logits_process_backward(s["x"], out=dx, signs=signs, **keep)

    say("[process] graph")
    run()
    torch.cuda.synchronize()
    ref = out.clone(), dx.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    torch.cuda.synchronize()
    for rep in range(4):
        out.zero_(), dx.zero_(), signs.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), ref[0].view(torch.int16)), rep
        assert torch.equal(dx.view(torch.int16), ref[1].view(torch.int16)), rep
        if rep == 1:
            with torch.cuda.stream(side):
                run()
            torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(60, 10, 500, 7), (2, 600, 20001, 40), (41, 200, 70, 4), (3, 1000, 24000, 9)], ids=str)
def test_many_rows(shape, dtype):
    """Enough rows for the larger chunks; both directions, checked on the first, the last and some other rows."""
    d0, d1, V, L = shape
    N = d0 * d1
    say(f"[process] many rows {shape} {dtype}")
    s = _inputs(d0, d1, V, dtype, L, seed=N)
    s["mask"] = _mask(d0, d1, V, seed=N)
    d = _dev(s)
    signs = vce.logits_signs(d["x"])
    z = f64(_call(d, out=torch.empty_like(d["x"]), signs=signs).view(N, V)[:])
    keep = {k: d[k] for k in ("history", "history_len", "prompt_len", "repetition", "mask", "temperature")}
    dx = f64(vce.ce_logits_process_backward(d["x"], out=torch.empty_like(d["x"]), signs=signs, **keep).view(N, V))
    pick = np.unique(np.concatenate([[0, 1, 2, N - 2, N - 1], np.random.RandomState(1).randint(0, N, 40)]))
    sub = {k: v.reshape(N, 1, -1)[pick] if k in ("x", "history", "mask") else v[pick] for k, v in s.items()}
    ref, budget, seen, allowed = _reference(sub)
    _check(torch.from_numpy(z[pick]), ref, budget, dtype, "z")
    x = f64(sub["x"]).reshape(len(pick), V)
    ref = ref_process_grad(x, x > 0, seen, f64(sub["repetition"]), f64(sub["temperature"]), allowed)
    assert_within(dx[pick], ref, (3.03 * U + half_step(dtype)) * np.abs(ref) + 1e-37, "dx")


def test_refusals():
    s = _dev(_inputs(2, 3, 70, torch.float32, 10, seed=1))
    s["mask"] = _mask(2, 3, 70, seed=1).cuda()
    x = s["x"]
    for change in (dict(x=x[0]), dict(x=x.half()), dict(x=x.transpose(1, 2)), dict(x=x[:1].expand(2, 3, 70)),
                   dict(history=s["history"].int()), dict(history=s["history"][0]), dict(history=s["history"][:1]),
                   dict(history=s["history"].transpose(1, 2)), dict(history_len=s["history_len"].long()),
                   dict(history_len=s["history_len"][:5]), dict(prompt_len=s["prompt_len"].cpu()),
                   dict(history=None), dict(repetition=s["repetition"].double()), dict(temperature=s["temperature"][:5]),
                   dict(mask=s["mask"][..., :2]), dict(mask=s["mask"].long()), dict(mask=s["mask"][:1]),
                   dict(bias=x[..., :69]), dict(bias=x.bfloat16()), dict(bias=x[0]), dict(out=x[..., :69]),
                   dict(out=x.bfloat16()), dict(signs=torch.empty((6, 8), dtype=torch.uint8, device="cuda")),
                   dict(signs=torch.empty((5, 9), dtype=torch.uint8, device="cuda")), dict(vocab_start=1)):
        kw = dict(s, **change)
        with pytest.raises(vce.CeArgumentError):
            vce.ce_logits_process(kw.pop("x"), **kw)
    keep = {k: s[k] for k in ("history", "history_len", "prompt_len", "repetition", "mask", "temperature")}
    with pytest.raises(vce.CeArgumentError):
        vce.ce_logits_process_backward(x, **keep)  # no signs
    assert torch.equal(x, _dev(_inputs(2, 3, 70, torch.float32, 10, seed=1))["x"]), "a refused call must touch nothing"


def test_no_rows_and_empty_history():
    x = torch.empty((0, 3, 17), device="cuda")
    assert vce.ce_logits_process(x, temperature=torch.empty(0, device="cuda")).numel() == 0
    s = _inputs(1, 2, 40, torch.float32, 0, seed=1)
    s["prompt_len"] = None
    d = _dev(s)
    say("[process] empty history")
    z = _call(d, out=torch.empty_like(d["x"]))
    assert_within(f64(z), f64(s["x"]) / f64(s["temperature"]).reshape(1, 2, 1), 4 * U * np.abs(f64(z)), "no history")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_output_beside_the_input(dtype):
    """Input and output rows side by side or in turn in one buffer; rows that meet are refused."""
    d0, d1, V, L = 3, 4, 301, 20
    s = _dev(_inputs(d0, d1, V, dtype, L, seed=61))
    x = s.pop("x")
    want = vce.ce_logits_process(x, out=torch.empty_like(x), **s)
    say(f"[process] shared buffer {dtype}")
    for cut in (lambda b, k: b.view(d0, d1, 2, V)[:, :, k], lambda b, k: b.view(d0, 2, d1, V)[:, k],
                lambda b, k: b.view(2, d1, d0, V)[k].transpose(0, 1), lambda b, k: b.view(d1, 2, d0, V)[:, k].transpose(0, 1)):
        b = torch.empty(2 * d0 * d1 * V, dtype=dtype, device="cuda")
        xs, out = cut(b, 0), cut(b, 1)
        xs.copy_(x)
        vce.ce_logits_process(xs, out=out, **s)
        assert torch.equal(out, want) and torch.equal(xs, x)
    b = torch.zeros(2 * d0 * d1 * V, dtype=dtype, device="cuda")
    xs = b[:d0 * d1 * V].view(d0, d1, V)
    xs.copy_(x)
    before = b.clone()
    for out in (b[V:V + d0 * d1 * V].view(d0, d1, V), b[8:8 + d0 * d1 * V].view(d0, d1, V),
                xs.view(d1, d0, V).transpose(0, 1), b.view(d0, 2 * d1, V)[:, :d1]):
        with pytest.raises(vce.CeArgumentError, match="overlaps"):
            vce.ce_logits_process(xs, out=out, **s)
    assert torch.equal(b, before)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(2, 300, 5000, 32768), (2, 130, 20000, 32768), (3, 7, 1500, 32768)], ids=str)
def test_many_rows_with_long_histories(shape, dtype):
    """32-bit counts in every chunk shape, both directions."""
    test_many_rows(shape, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("L", [5, 32768])
def test_more_rows_than_one_launch_holds(L, dtype):
    """2^22 workgroups in a launch: some take a second row, whose counts use the same LDS."""
    N, V = (1 << 22) + 1001, 13
    g = torch.Generator("cuda").manual_seed(L)
    x = torch.randn((1, N, V), generator=g, device="cuda", dtype=dtype)
    uniform = lambda: torch.rand(N, generator=g, device="cuda") + 0.5  # noqa: E731
    h = torch.randint(-1, V + 1, (1, 1, L), generator=g, device="cuda")
    rows = dict(history_len=torch.randint(0, 6, (N,), generator=g, device="cuda", dtype=torch.int32),
                prompt_len=torch.randint(0, 4, (N,), generator=g, device="cuda", dtype=torch.int32),
                repetition=uniform(), frequency=uniform(), presence=uniform(), temperature=uniform())
    mask = torch.randint(0, 1 << 13, (1, N, 1), generator=g, device="cuda", dtype=torch.int32)
    back = ("history_len", "prompt_len", "repetition", "temperature")

    def run(a, b):
        xs, sub = x[:, a:b], {k: v[a:b] for k, v in rows.items()}
        signs = vce.logits_signs(xs).fill_(255)
        steps = dict(history=h.expand(1, b - a, L), mask=mask[:, a:b])
        z = vce.ce_logits_process(xs, out=torch.empty_like(xs), signs=signs, **steps, **sub)
        dx = vce.ce_logits_process_backward(xs, out=torch.empty_like(xs), signs=signs, **steps,
                                            **{k: sub[k] for k in back})
        return z, dx, signs

    say(f"[process] {N} rows, {L} {dtype}")
    z, dx, signs = run(0, N)
    for a, b in ((0, 4100), ((1 << 22) - 300, 1 << 22), (1 << 22, N)):
        for whole, part in zip((z[:, a:b], dx[:, a:b], signs[a:b]), run(a, b)):
            assert torch.equal(whole, part), (a, b)
    pick = torch.tensor([0, 1, (1 << 22) - 1, 1 << 22, N - 1])
    sub = {k: v.cpu()[pick] for k, v in rows.items()} | dict(
        x=x.cpu()[0, pick].view(5, 1, V), history=h.cpu().expand(5, 1, L), mask=mask.cpu()[0, pick].view(5, 1, 1))
    ref, budget, _, _ = _reference(sub)
    _check(z[0].cpu()[pick], ref, budget, dtype, "z")


@pytest.mark.parametrize("dtype,V", [(torch.float32, (1 << 30) - 1), (torch.bfloat16, (1 << 31) - 1)], ids=["f32", "bf16"])
def test_a_row_of_nearly_4_gib(dtype, V):
    """The widest rows: byte offsets up to 2^32, in both directions, with tokens at both ends."""
    x = torch.empty((1, 1, V), dtype=dtype, device="cuda").fill_(3.0)
    h = torch.tensor([0, 7, V // 2, V - 9, V - 2, V - 1, V - 1], device="cuda").view(1, 1, -1)
    two, half = torch.full((1,), 2.0, device="cuda"), torch.full((1,), 0.5, device="cuda")
    signs = vce.logits_signs(x)
    say(f"[process] a row of {V} {dtype}")
    vce.ce_logits_process(x, history=h, repetition=two, presence=half, temperature=half, signs=signs)
    want = {0: 2.0, 7: 2.0, V // 2: 2.0, V - 9: 2.0, V - 2: 2.0, V - 1: 2.0}  # (3 / 2 - 1 / 2) / (1 / 2)
    assert all(float(x[0, 0, j]) == z for j, z in want.items())
    flat, step = x.view(-1), 1 << 28
    others = [int((flat[a:a + step] != 6.0).sum()) for a in range(0, V, step)]
    assert sum(others) == len(want), others
    x.fill_(3.0)
    vce.ce_logits_process_backward(x, history=h, repetition=two, temperature=half, signs=signs)
    assert all(float(x[0, 0, j]) == 3.0 for j in want)  # 3 / 2 / (1 / 2)
    others = [int((flat[a:a + step] != 6.0).sum()) for a in range(0, V, step)]
    assert sum(others) == len(want), others
