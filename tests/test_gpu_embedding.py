"""Embedding and its gradient against the 64-bit definition."""
import numpy as np
import pytest
import torch

import vocab_cross_entropy_amd as vce
from gpu_util import say
from ops_util import TINY, U, assert_within, f64, half_step, ref_embed_grad

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _ids(N, V, seed, kind):
    g = _gen(seed)
    if kind == "same":
        return torch.full((N,), V // 2)
    if kind == "uniform":
        return torch.randint(0, V, (N,), generator=g)
    if kind == "pairs":  # runs of two
        return torch.arange(N) // 2 % V
    if kind == "runs":  # ids that occur 1, 2, ... 50 times, in any order
        count = torch.arange(1, 51).repeat(V // 50 + 1)[:V]
        ids = torch.repeat_interleave(torch.arange(V), count)[:N]
        return ids[torch.randperm(N, generator=g)]
    return (torch.rand(N, generator=g, dtype=torch.float64) ** 4 * V).long().clamp(max=V - 1)  # long tail


DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("N,V,D", [(1, 1, 1), (1, 50, 4096), (5, 7, 3), (300, 100, 17), (33, 1000, 2051), (64, 9, 640)])
def test_lookup(N, V, D, dtype):
    w = torch.randn((V, D), generator=_gen(N)).to(dtype)
    ids = _ids(N, V, N, "tail")
    for scale in (1.0, -3.7):
        say(f"[embed] {N} {V} {D} {dtype} {scale}")
        out = vce.ce_embedding(ids.cuda(), w.cuda(), scale)
        ref = f64(w)[ids.numpy()] * np.float64(np.float32(scale))
        assert_within(f64(out), ref, (half_step(dtype) * 1.01 + U) * np.abs(ref) + TINY, "lookup")


def test_lookup_strides_shards_and_bad_ids():
    V, D = 100, 41
    w = torch.randn((V, D), generator=_gen(1))
    wide = torch.zeros((V, D + 6), dtype=torch.float32, device="cuda")
    wide[:, 3:3 + D] = w.cuda()
    ids = torch.tensor([0, 99, -1, 100, 42, -2 ** 63, 2 ** 63 - 1, 5])
    strided = torch.stack([ids, ids * 0 + 7], 1).cuda()[:, 0]
    buf = torch.full((8, D + 2), 9.0, device="cuda")
    say("[embed] strides")
    vce.ce_embedding(strided, wide[:, 3:3 + D], 2.0, out=buf[:, 1:1 + D])
    got = f64(buf)
    for n, i in enumerate(ids.tolist()):
        if 0 <= i < V:
            assert np.array_equal(got[n, 1:1 + D], f64(w)[i] * 2)
        else:
            assert np.isnan(got[n, 1:1 + D]).all(), "an id outside the vocabulary must give NaN"
    assert (got[:, 0] == 9).all() and (got[:, -1] == 9).all()
    # shards: other shards' ids are zeros, so the parts add up
    good = ids[[0, 1, 4, 7]].cuda()
    parts = [vce.ce_embedding(good, w[lo:hi].cuda(), 2.0, vocab_start=lo, vocab_total=V) for lo, hi in
             ((0, 43), (43, 100))]
    assert torch.equal(parts[0] + parts[1], vce.ce_embedding(good, w.cuda(), 2.0))
    far = vce.ce_embedding(torch.tensor([100, -1]).cuda(), w[:43].cuda(), vocab_start=0, vocab_total=V)
    assert torch.isnan(far).all()


GRAD = [(1, 1, 1, "tail"), (1, 60, 40, "tail"), (2, 3, 8, "same"), (15, 4, 9, "tail"), (16, 4, 64, "pairs"),
        (17, 40, 5, "same"), (33, 5, 130, "tail"), (400, 30, 2051, "tail"), (700, 3000, 33, "uniform"),
        (2049, 500, 24, "same"), (5000, 700, 12, "tail"), (8192, 50, 7, "pairs"), (8193, 50, 7, "tail"),
        (600, 3, 520, "same"), (3001, 2, 300, "pairs"), (4000, 400, 270, "runs"), (4000, 400, 8, "runs"),
        (9000, 600, 1030, "runs"), (5000, 1 << 20, 1, "uniform"), (12345, 70000, 5, "uniform"), (20000, 300, 3, "same"), (66000, 1100, 2, "tail")]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("N,V,D,kind", GRAD, ids=lambda v: str(v))
def test_gradient(N, V, D, kind, dtype):
    """Overwriting and adding, with and without a padding id: the sum of m terms rounds at most m times on
    partial sums of at most their absolute sum, the scale and the addition once more."""
    ids = _ids(N, V, N + V, kind)
    dout = torch.randn((N, D), generator=_gen(D)).to(dtype)
    scale = 1.7
    s64 = np.float64(np.float32(scale))
    pad = int(ids[0]) if V > 1 and kind != "same" else None
    for padding in {None, pad}:
        say(f"[embed grad] {N} {V} {D} {kind} {dtype} padding {padding}")
        ref, size, m = ref_embed_grad(f64(dout), ids.numpy(), V, s64, padding)
        tol = 1.01 * U * (m + 2) * size + TINY
        dw = torch.full((V, D), float("nan"), device="cuda")
        vce.ce_embedding_backward(dout.cuda(), ids.cuda(), V, scale, padding_idx=padding, dw=dw)
        assert_within(f64(dw), ref, tol, "overwritten")
        assert not dw.view(torch.int32)[torch.from_numpy(m[:, 0] == 0).cuda()].any(), "unnamed rows must be +0.0"
        again = vce.ce_embedding_backward(dout.cuda(), ids.cuda(), V, scale, padding_idx=padding)
        assert torch.equal(again.view(torch.int32), dw.view(torch.int32)), "repeats must be equal bit for bit"
        base = torch.randn((V, D), generator=_gen(7))
        acc = base.cuda()
        vce.ce_embedding_backward(dout.cuda(), ids.cuda(), V, scale, padding_idx=padding, dw=acc, accumulate=True)
        assert_within(f64(acc), ref + f64(base), tol + U * np.abs(ref + f64(base)) * 1.01, "added")
        untouched = torch.from_numpy(m[:, 0] == 0)
        assert torch.equal(acc.cpu()[untouched], base[untouched])


# rows of several units and of partial quads, with runs shorter and longer than a unit's tokens, in both forms of the sum
MORE = [(1500, 700, 515, "tail"), (2000, 64, 1030, "pairs"), (1100, 3, 1027, "uniform"), (2500, 2500, 257, "uniform"),
        (1025, 40, 128, "tail"), (3000, 150, 129, "runs"), (7200, 40, 1027, "tail"), (29000, 1200, 257, "runs"),
        (7400, 2, 1001, "pairs"), (66000, 900, 131, "tail"), (70000, 3, 6, "uniform"), (65537, 65537, 4, "runs")]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("N,V,D,kind", MORE, ids=lambda v: str(v))
def test_gradient_units(N, V, D, kind, dtype):
    test_gradient(N, V, D, kind, dtype)


@pytest.mark.parametrize("N", [1, 200, 900, 1500, 9000, 66000])
@pytest.mark.parametrize("V,D", [(1, 1), (9000, 1), (3001, 3), (700, 7), (333, 64), (211, 515), (41, 1037)])
def test_rows_that_no_token_names(N, V, D):
    """Zeros in every row no token names, whichever way they are written, and nothing before or behind dW."""
    ids = torch.randint(0, V, (N,), generator=_gen(N)) // 3 * 3
    dout = torch.ones((N, D), device="cuda", dtype=torch.bfloat16)
    count = torch.bincount(ids, minlength=V).float()[:, None].expand(V, D)
    say(f"[embed grad] fill {N} {V} {D}")
    for ld in (D, D + 1):  # rows end to end, and with a gap
        for first in (4, 5):  # on a 16-byte boundary, and off it
            buf = torch.full((first + V * ld + 4,), -3.0, device="cuda")
            dw = torch.as_strided(buf, (V, D), (ld, 1), first)
            vce.ce_embedding_backward(dout, ids.cuda(), V, 1.0, dw=dw)
            assert torch.equal(dw.cpu(), count)
            dw.fill_(-3.0)
            assert (buf == -3.0).all()


def test_gradient_strides_shards_and_bad_ids():
    N, V, D = 500, 64, 30
    ids = torch.randint(-20, V + 20, (N,), generator=_gen(5))
    ids[3], ids[4] = -2 ** 63, 2 ** 63 - 1
    dout = torch.randn((N, D), generator=_gen(6))
    wide = torch.zeros((N, D + 3), device="cuda")
    wide[:, 1:1 + D] = dout.cuda()
    for lo, hi in ((0, V), (0, 20), (20, V)):
        say(f"[embed grad] shard {lo} {hi}")
        buf = torch.full((hi - lo, D + 4), 5.0, device="cuda")
        vce.ce_embedding_backward(wide[:, 1:1 + D], torch.stack([ids, ids], 1).cuda()[:, 1], hi - lo, 0.5,
                                  dw=buf[:, 2:2 + D], vocab_start=lo, vocab_total=V)
        ref, size, m = ref_embed_grad(f64(dout), ids.numpy(), hi - lo, 0.5, vocab_start=lo)
        assert_within(f64(buf)[:, 2:2 + D], ref, 1.01 * U * (m + 2) * size + TINY, "shard")
        assert (f64(buf)[:, :2] == 5).all() and (f64(buf)[:, -2:] == 5).all()


def test_every_token_is_padding():
    ids = torch.full((70,), 3).cuda()
    dout = torch.ones((70, 20), device="cuda")
    dw = vce.ce_embedding_backward(dout, ids, 5, padding_idx=3, dw=torch.full((5, 20), float("nan"), device="cuda"))
    assert not dw.any()
    kept = torch.full((5, 20), 2.0, device="cuda")
    vce.ce_embedding_backward(dout, ids, 5, padding_idx=3, dw=kept, accumulate=True)
    assert (kept == 2).all()


def test_one_workspace_for_smaller_batches():
    """A workspace sized for the largest batch serves every smaller one, whichever sort that takes."""
    V, D = 300, 10
    ws = torch.empty(vce.ce_embedding_workspace_bytes(70000, D, V), dtype=torch.uint8, device="cuda")
    for N in (70000, 66000, 65536, 8193, 8192, 100, 1):
        ids, dout = _ids(N, V, N, "tail"), torch.randn((N, D), generator=_gen(N))
        say(f"[embed grad] workspace {N}")
        dw = vce.ce_embedding_backward(dout.cuda(), ids.cuda(), V, dw=torch.empty((V, D), device="cuda"), ws=ws)
        ref, size, m = ref_embed_grad(f64(dout), ids.numpy(), V, 1.0)
        assert_within(f64(dw), ref, 1.01 * U * (m + 2) * size + TINY, str(N))


def test_refusals():
    w, ids, dout = torch.ones((6, 5), device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda"), \
        torch.ones((4, 5), device="cuda")
    for call in (lambda: vce.ce_embedding(ids.int(), w), lambda: vce.ce_embedding(ids.cpu(), w),
                 lambda: vce.ce_embedding(ids.view(2, 2), w), lambda: vce.ce_embedding(ids, w.half()),
                 lambda: vce.ce_embedding(ids, w.t()), lambda: vce.ce_embedding(ids, w, out=dout[:3]),
                 lambda: vce.ce_embedding(ids, w, out=dout.bfloat16()), lambda: vce.ce_embedding(ids, w, vocab_start=1),
                 lambda: vce.ce_embedding_backward(dout, ids[:3], 6),
                 lambda: vce.ce_embedding_backward(dout, ids, 6, dw=w.bfloat16()),
                 lambda: vce.ce_embedding_backward(dout, ids, 6, dw=w[:5]),
                 lambda: vce.ce_embedding_backward(dout, ids, 6, accumulate=True),
                 lambda: vce.ce_embedding_backward(dout, ids, 6, padding_idx=-1),
                 lambda: vce.ce_embedding_backward(dout, ids, 6, ws=torch.empty(8, dtype=torch.uint8, device="cuda")),
                 lambda: vce.ce_embedding_backward(dout[:, :1].expand(4, 5), ids, 6),
                 lambda: vce.embedding(ids, w, grad_buffer=w[:5])):
        with pytest.raises(vce.CeArgumentError):
            call()


def test_no_tokens():
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    w = torch.ones((6, 5), device="cuda")
    assert vce.ce_embedding(ids, w).shape == (0, 5)
    dw = vce.ce_embedding_backward(torch.empty((0, 5), device="cuda"), ids, 6, dw=w.clone())
    assert not dw.any()
    dw = vce.ce_embedding_backward(torch.empty((0, 5), device="cuda"), ids, 6, dw=w.clone(), accumulate=True)
    assert torch.equal(dw, w)


def test_infinities_stay_in_their_rows():
    ids = torch.tensor([1, 2, 1, 3])
    dout = torch.ones((4, 9))
    dout[0, 4], dout[3, 5] = float("inf"), float("nan")
    dw = f64(vce.ce_embedding_backward(dout.cuda(), ids.cuda(), 5))
    assert dw[1, 4] == np.inf and np.isnan(dw[3, 5]) and np.isfinite(dw).sum() == 5 * 9 - 2


def test_autograd_and_grad_buffer():
    V, D = 50, 24
    ids = torch.randint(0, V, (3, 7), generator=_gen(1))
    c = torch.randn((3, 7, D), generator=_gen(2))
    for dtype in DTYPES:
        say(f"[embed] autograd {dtype}")
        w = torch.randn((V, D), generator=_gen(3)).to(dtype)
        wd = w.cuda().requires_grad_()
        out = vce.embedding(ids.cuda().t(), wd, 2.0, padding_idx=4).transpose(0, 1)
        (out.float() * c.cuda()).sum().backward()
        ref, size, m = ref_embed_grad(f64(c.to(dtype)).reshape(-1, D), ids.reshape(-1).numpy(), V, 2.0, 4)
        assert_within(f64(wd.grad), ref, 1.01 * U * (m + 2) * size + half_step(dtype) * np.abs(ref) + TINY, "grad")
        buf = torch.ones((V, D), device="cuda")
        w2 = w.cuda().requires_grad_()
        (vce.embedding(ids.cuda(), w2, 2.0, padding_idx=4, grad_buffer=buf).float() * c.cuda()).sum().backward()
        assert w2.grad is None
        assert_within(f64(buf), ref + 1, 1.01 * U * ((m + 2) * size + np.abs(ref + 1)), "buffer")
    # differences of the 64-bit lookup: the map is linear in the table
    v = torch.randn((V, D), generator=_gen(9), dtype=torch.float64)
    live = (ids.reshape(-1) != 4).double().view(-1, 1)
    num = (v[ids.reshape(-1)] * 2.0 * c.double().view(-1, D) * live).sum()
    w32 = torch.zeros((V, D), device="cuda").requires_grad_()
    (vce.embedding(ids.cuda(), w32, 2.0, padding_idx=4) * c.cuda()).sum().backward()
    got = (w32.grad.double().cpu() * v).sum()
    assert abs(float(got - num)) <= 30 * U * float((w32.grad.double().cpu() * v).abs().sum())


@pytest.mark.parametrize("N", [900, 9000])
def test_graph_replays_and_streams(N):
    V, D = 700, 40
    ids, dout = _ids(N, V, 3, "tail").cuda(), torch.randn((N, D), generator=_gen(4)).cuda()
    ws = torch.empty(vce.ce_embedding_workspace_bytes(N, D, V), dtype=torch.uint8, device="cuda")
    w = torch.randn((V, D), generator=_gen(5)).cuda()
    out, dw = torch.empty((N, D), device="cuda"), torch.empty((V, D), device="cuda")

    def run():
        vce.ce_embedding(ids, w, 3.0, out=out)
        vce.ce_embedding_backward(dout, ids, V, 2.0, dw=dw, ws=ws)

    say(f"[embed] graph {N}")
    run()
    torch.cuda.synchronize()
    ref = out.clone(), dw.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    torch.cuda.synchronize()
    for rep in range(4):
        out.zero_(), dw.fill_(float("nan")), ws.fill_(rep * 85)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[0]) and torch.equal(dw, ref[1]), rep
        if rep == 1:
            with torch.cuda.stream(side):
                run()
            torch.cuda.synchronize()
    # two calls at once, each with its own workspace
    streams = [torch.cuda.Stream() for _ in range(2)]
    res = []
    for k in range(6):
        streams[k % 2].wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(streams[k % 2]):
            res.append(vce.ce_embedding_backward(dout, ids, V, 2.0))
    torch.cuda.synchronize()
    assert all(torch.equal(r, ref[1]) for r in res)


# wide rows with a length of whole 16-byte words in batches that the sum by tiles takes; more than 64 tokens to a tile
LARGE = [(2100, 700, 4096, "tail"), (15000, 600, 520, "runs"), (300000, 5000, 136, "tail"), (300000, 12000, 136, "runs")]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("N,V,D,kind", LARGE, ids=lambda v: str(v))
def test_gradient_of_large_batches(N, V, D, kind, dtype):
    ids = _ids(N, V, N + V, kind)
    assert ids.shape == (N,)
    dout = torch.randn((N, D), generator=_gen(D)).to(dtype)
    ref = torch.zeros((V, D), dtype=torch.float64).index_add_(0, ids, dout.double()).mul_(0.75).numpy()
    size = torch.zeros((V, D), dtype=torch.float64).index_add_(0, ids, dout.double().abs_()).mul_(0.75).numpy()
    m = torch.bincount(ids, minlength=V).numpy()[:, None]
    tol = 1.01 * U * (m + 2) * size + TINY
    say(f"[embed grad] large {N} {V} {D} {kind} {dtype}")
    dd, idd = dout.cuda(), ids.cuda()
    dw = vce.ce_embedding_backward(dd, idd, V, 0.75, dw=torch.full((V, D), float("nan"), device="cuda"))
    assert_within(f64(dw), ref, tol, "overwritten")
    base = torch.randn((V, D), generator=_gen(7))
    acc = vce.ce_embedding_backward(dd, idd, V, 0.75, dw=base.cuda(), accumulate=True)
    assert_within(f64(acc), ref + f64(base), tol + U * np.abs(ref + f64(base)) * 1.01, "added")
    again = vce.ce_embedding_backward(dd, idd, V, 0.75, dw=base.cuda(), accumulate=True)
    assert torch.equal(again.view(torch.int32), acc.view(torch.int32))


def test_more_tokens_than_one_launch_holds():
    """2^23 workgroups in a launch, a wide row each: some take a second one."""
    N, V, D = (1 << 23) + 300, 50, 1032
    w = torch.randn((V, D), generator=_gen(1)).bfloat16().cuda()
    ids = torch.randint(0, V, (N,), generator=_gen(2)).cuda()
    say(f"[embed] {N} tokens")
    out = vce.ce_embedding(ids, w)
    for a, b in ((0, 300), ((1 << 23) - 300, 1 << 23), (1 << 23, N)):
        assert torch.equal(out[a:b], w[ids[a:b]])


@pytest.mark.parametrize("N", [3, 1500])
def test_more_unnamed_rows_than_one_launch_holds(N):
    """Zeros in 2^26 rows and more, eight to a workgroup, with a gap between rows that is left alone."""
    V, D = (1 << 26) + 4003, 3
    ids = torch.randint(0, V, (N,), generator=_gen(N))
    ids[0], ids[1] = V - 1, 1 << 26
    dout = torch.ones((N, D), device="cuda")
    say(f"[embed grad] fill of {V} rows")
    buf = torch.full((V, D + 1), -3.0, device="cuda")
    vce.ce_embedding_backward(dout, ids.cuda(), V, dw=buf[:, :D])
    want = torch.bincount(ids, minlength=V).float().cuda()
    assert all(torch.equal(buf[:, k], want) for k in range(D)) and bool((buf[:, D] == -3).all())


@pytest.mark.parametrize("D", [3, 40, 130])
def test_the_most_tokens(D):
    """2^26 tokens, a twentieth of them one id: whole numbers, so that the sums are exact in any order."""
    N, V = 1 << 26, 70001
    g = torch.Generator("cuda").manual_seed(D)
    ids = torch.randint(0, V, (N,), generator=g, device="cuda")
    ids[torch.randint(0, N, (N // 20,), generator=g, device="cuda")] = 12345
    ids[::1009] = 777  # the padding
    value = ((torch.arange(V, device="cuda")[:, None] * 7 + torch.arange(D, device="cuda")) % 5).float()
    dout = value.bfloat16()[ids]
    say(f"[embed grad] {N} tokens x {D}")
    dw = vce.ce_embedding_backward(dout, ids, V, 2.0, padding_idx=777)
    count = torch.bincount(ids, minlength=V)
    count[777] = 0
    assert torch.equal(dw, value * count.float()[:, None] * 2)
