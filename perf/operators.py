"""The operators around the vocabulary, as they are measured: logit processing, embedding, RMS norm.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges, ``prepare(case, seed)`` makes a
case's inputs on the GPU, ``run(state)`` makes one pass through an operator and ``exact(case, seed)`` gives
the same outputs from the definition in 64 bits.  With ``own`` false ``run`` is the plain form in elementary
torch operations (32 bits, one rounding at the end); with ``own`` true it calls the library.

Per row r of logits x, with c the occurrences of column j among the row's output tokens:
    process   z = ((pen(x) - frequency c - presence [c > 0]) + bias) / temperature, -inf where masked,
              pen(x) = x / repetition (x > 0) or x repetition for columns seen in prompt or output, else x
    embed     out_n = scale W[id_n];   dW[v] = scale sum over id_n = v of dout_n
    norm      s = x + residual;  y = s rsqrt(mean s^2 + eps) weight
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
FP8_MAX = 448.0
FP32_TINY = 2.0 ** -126


def listed():
    return [
        # one sequence being generated: latency of a single row under a grammar, sampling parameters set
        dict(name="process one row", op="process", d0=1, d1=1, V=128000, dtype="bf16", L=300, prefix=False, mask=True,
             bias=False, seed_shift=0),
        # a decoding batch with FP32 logits, long ragged histories, a shared bias and a grammar for every row
        dict(name="process batch", op="process", d0=64, d1=1, V=128000, dtype="f32", L=4096, prefix=False, mask=True,
             bias=True, seed_shift=1),
        # log-probabilities of a sampled policy: every position of every sequence has its own prefix as history
        dict(name="process train", op="process", d0=4, d1=2048, V=128000, dtype="bf16", L=2048, prefix=True,
             mask=False, bias=False, seed_shift=2),
        # the gradient of that step at a smaller, odd vocabulary: rows that start at every alignment
        dict(name="process backward odd", op="process_bwd", d0=2, d1=512, V=32003, dtype="bf16", L=512, prefix=True,
             mask=False, bias=False, seed_shift=3),
        # a decoding step's tokens
        dict(name="embed few", op="embed", N=5, V=128000, D=4096, dtype="bf16"),
        # a prompt's, or a training batch's tokens
        dict(name="embed batch", op="embed", N=8192, V=128000, D=4096, dtype="bf16"),
        # the gradient added to the tied head's FP32 gradient
        dict(name="embed grad tied", op="embed_bwd", N=8192, V=128000, D=4096, dtype="bf16", add=True),
        # the gradient of an untied table, FP32, odd width, more tokens
        dict(name="embed grad odd", op="embed_bwd", N=20011, V=32000, D=1037, dtype="f32", add=False),
        # a decoding step's final norm
        dict(name="norm few", op="norm", N=3, D=4096, dtype="bf16", residual=True, group=-1),
        # a prompt's norm in front of an 8-bit product: values in e4m3 with a scale for each 128
        dict(name="norm fp8", op="norm", N=8192, D=4096, dtype="bf16", residual=True, group=128),
        # the training step's gradient
        dict(name="norm backward", op="norm_bwd", N=8192, D=4096, dtype="bf16", residual=True),
        # FP32, odd width, few rows
        dict(name="norm backward odd", op="norm_bwd", N=515, D=2731, dtype="f32", residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["process", "process_bwd", "embed", "embed_bwd", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("process"):
        V = rng.choice([128000, 32000, 8192, _log(rng, 500, 131072), _log(rng, 500, 131072)])
        d0, d1 = _log(rng, 1, 64), rng.choice([1, _log(rng, 1, 1024)])
        d1 = max(1, min(d1, (2048 * 128000) // (d0 * V)))
        prefix = d1 > 1
        return dict(op=op, d0=d0, d1=d1, V=V, dtype=dtype, L=d1 if prefix else _log(rng, 1, 4096), prefix=prefix,
                    mask=rng.random() < 0.5, bias=op == "process" and rng.random() < 0.4,
                    seed_shift=rng.randrange(1 << 20))
    if op.startswith("embed"):
        case = dict(op=op, N=_log(rng, 1, 32768), V=_log(rng, 1000, 131072), D=rng.choice([4096, _log(rng, 16, 8192)]),
                    dtype=dtype)
        if op == "embed_bwd":
            case["add"] = rng.random() < 0.5
            case["V"] = min(case["V"], 128000 * 4096 // case["D"])
        return case
    case = dict(op=op, N=_log(rng, 1, 16384), D=rng.choice([4096, 8192, _log(rng, 16, 16384)]), dtype=dtype,
                residual=rng.random() < 0.7)
    if op == "norm":
        case["group"] = rng.choice([-1, -1, 0, 128])  # -1: the type's own output; 0: e4m3 with a scale for each row
    return case


def _gen(seed, case):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + int(case.get("seed_shift", 0)))


def _tokens(shape, V, g):
    """Token ids with a long tail: id 0 makes up about 5% of a 128000-word vocabulary's text."""
    u = torch.rand(shape, generator=g, device="cuda", dtype=torch.float64)
    return (u.pow_(4) * V).long().clamp_(max=V - 1)


def prepare(case, seed):
    g, op = _gen(seed, case), case["op"]
    dt = DTYPES[case["dtype"]]

    def normal(*shape, sigma=1.0, dtype=dt):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(sigma)

    def uniform(n, lo, hi):
        return torch.rand(n, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(case=case)
    if op.startswith("process"):
        d0, d1, V, L = case["d0"], case["d1"], case["V"], case["L"]
        N = d0 * d1
        x = normal(d0, d1, V, sigma=2.0)
        if case["prefix"]:  # position i of sequence b has the i tokens before it
            s["history"] = _tokens((d0, 1, L), V, g).expand(d0, d1, L)
            s["history_len"] = torch.arange(d1, device="cuda", dtype=torch.int32).repeat(d0)
            s["prompt_len"] = (s["history_len"] // 4).to(torch.int32)
        else:  # ragged; the first of several rows has generated nothing yet
            s["history"] = _tokens((d0, d1, L), V, g)
            s["history_len"] = torch.randint(0, L + 1, (N,), generator=g, device="cuda", dtype=torch.int32)
            s["history_len"][0] = 0 if N > 1 else L
            s["prompt_len"] = (s["history_len"].double() * uniform(N, 0, 1)).to(torch.int32)
            past = torch.arange(L, device="cuda") >= s["history_len"].view(d0, d1, 1)
            s["history"].masked_fill_(past, -1)
        s["repetition"], s["temperature"] = uniform(N, 1.0, 1.5), uniform(N, 0.5, 1.5)
        s["mask"] = None
        if case["mask"]:  # a quarter of the columns allowed; the last of several rows has none
            words = [torch.randint(-2 ** 31, 2 ** 31, (d0, d1, (V + 31) // 32), generator=g, device="cuda",
                                   dtype=torch.int32) for _ in range(2)]
            s["mask"] = words[0] & words[1]
            if N > 1:
                s["mask"][-1, -1] = 0
        s["out"] = torch.empty_like(x)
        if op == "process":
            s["x"] = x
            s["frequency"], s["presence"] = uniform(N, 0.0, 0.5), uniform(N, 0.0, 0.5)
            s["bias"] = normal(V, sigma=1.0, dtype=torch.float32).expand(d0, d1, V) if case["bias"] else None
        else:
            s["dz"] = torch.rand(x.shape, generator=g, device="cuda", dtype=dt).mul_(1.0 / V)
            pad = torch.zeros((N, -V % 8), dtype=torch.bool, device="cuda")
            bits = torch.cat([x.view(N, V) > 0, pad], 1).view(N, -1, 8)
            s["signs"] = sum(bits[..., k].to(torch.uint8) << k for k in range(8))
    elif op.startswith("embed"):
        N, V, D = case["N"], case["V"], case["D"]
        s["ids"] = _tokens((N,), V, g)
        s["scale"] = math.sqrt(D)
        if op == "embed":
            s["w"] = normal(V, D, sigma=0.02)
        else:
            s["dout"] = normal(N, D, sigma=1e-3)
            s["dw"] = normal(V, D, sigma=1e-2, dtype=torch.float32) if case["add"] else None
    else:
        N, D = case["N"], case["D"]
        s["w"] = normal(D, sigma=0.1).add_(1.0)
        if op == "norm":
            s["x"] = normal(N, D)
            s["r"] = normal(N, D, sigma=3.0) if case["residual"] else None
        else:
            s["s"], s["dy"] = normal(N, D, sigma=3.0), normal(N, D, sigma=1e-3)
            s["dsum"] = normal(N, D, sigma=1e-3) if case["residual"] else None
    return s


# ---- the plain forms -------------------------------------------------------------------------------------


def _counts(s, V):
    """(seen in prompt or output, occurrences in the output) of every column, [d0, d1, V]."""
    h = s["history"]
    at = torch.arange(h.shape[2], device=h.device)
    n, p = s["history_len"].view(*h.shape[:2], 1), s["prompt_len"].view(*h.shape[:2], 1)
    inside = (at < n) & (h >= 0) & (h < V)
    idx = torch.where(inside, h, 0)
    c = torch.zeros((*h.shape[:2], V), dtype=torch.int32, device=h.device)
    seen = c.scatter_add(2, idx, (inside & (at < p)).int()) > 0
    c.scatter_add_(2, idx, (inside & (at >= p)).int())
    return seen | (c > 0), c


def _allowed(mask, V):
    bits = (mask.unsqueeze(-1) >> torch.arange(32, device=mask.device, dtype=torch.int32)) & 1
    return bits.flatten(2)[..., :V] != 0


def _rows(t, like):
    return t.to(like.dtype).view(like.shape[0], like.shape[1], 1)


def _plain_process(s):
    v = s["x"].float()
    V = v.shape[2]
    seen, c = _counts(s, V)
    theta = _rows(s["repetition"], v)
    v = torch.where(seen, torch.where(v > 0, v / theta, v * theta), v)
    v = v - _rows(s["frequency"], v) * c - _rows(s["presence"], v) * (c > 0)
    if s["bias"] is not None:
        v = v + s["bias"]
    v = v / _rows(s["temperature"], v)
    if s["mask"] is not None:
        v = torch.where(_allowed(s["mask"], V), v, -math.inf)
    return v.to(s["x"].dtype)


def _plain_process_bwd(s):
    v = s["dz"].float()
    V = v.shape[2]
    seen, _ = _counts(s, V)
    theta = _rows(s["repetition"], v)
    up = (s["signs"].unsqueeze(-1) >> torch.arange(8, device=v.device, dtype=torch.uint8)) & 1
    up = up.flatten(1)[:, :V].reshape(v.shape) != 0
    v = torch.where(seen, torch.where(up, v / theta, v * theta), v) / _rows(s["temperature"], v)
    if s["mask"] is not None:
        v = torch.where(_allowed(s["mask"], V), v, 0.0)
    return v.to(s["dz"].dtype)


def _plain_embed(s):
    return (s["w"][s["ids"]].float() * s["scale"]).to(s["w"].dtype)


def _plain_embed_bwd(s):
    rows = s["dout"].float() * s["scale"]
    dw = s["dw"]
    if dw is None:
        dw = torch.zeros((s["case"]["V"], rows.shape[1]), dtype=torch.float32, device=rows.device)
    return dw.index_add_(0, s["ids"], rows)


def _plain_norm(s):
    x, group = s["x"], s["case"]["group"]
    t = x.float() if s["r"] is None else x.float() + s["r"].float()
    y = t * torch.rsqrt(t.square().mean(1, keepdim=True) + EPS) * s["w"].float()
    total = [] if s["r"] is None else [t.to(x.dtype)]
    if group < 0:
        return [y.to(x.dtype)] + total
    N, D = y.shape
    G = group if group else D
    y = torch.cat([y, y.new_zeros((N, -D % G))], 1).view(N, -1, G)
    scale = (y.abs().amax(2) / FP8_MAX).clamp(min=FP32_TINY)
    q = (y / scale.unsqueeze(2)).view(N, -1)[:, :D].to(torch.float8_e4m3fn)
    return [q, scale] + total


def _plain_norm_bwd(s):
    t, dy, w = s["s"].float(), s["dy"].float(), s["w"].float()
    rstd = torch.rsqrt(t.square().mean(1, keepdim=True) + EPS)
    gy = dy * w
    ds = rstd * gy - t * (rstd.pow(3) * (gy * t).mean(1, keepdim=True))
    if s["dsum"] is not None:
        ds = ds + s["dsum"].float()
    return [ds.to(s["s"].dtype), (dy * t * rstd).sum(0)]


_PLAIN = dict(process=_plain_process, process_bwd=_plain_process_bwd, embed=_plain_embed, embed_bwd=_plain_embed_bwd,
              norm=_plain_norm, norm_bwd=_plain_norm_bwd)


# ---- the library's calls ---------------------------------------------------------------------------------


def _own(s):
    import vocab_cross_entropy_amd as vce

    case = s["case"]
    op = case["op"]
    if op == "process":
        return vce.ce_logits_process(s["x"], out=s["out"], history=s["history"], history_len=s["history_len"],
                                     prompt_len=s["prompt_len"], repetition=s["repetition"], presence=s["presence"],
                                     frequency=s["frequency"], bias=s["bias"], mask=s["mask"],
                                     temperature=s["temperature"])
    if op == "process_bwd":
        return vce.ce_logits_process_backward(s["dz"], out=s["out"], signs=s["signs"], history=s["history"],
                                              history_len=s["history_len"], prompt_len=s["prompt_len"],
                                              repetition=s["repetition"], mask=s["mask"],
                                              temperature=s["temperature"])
    if op == "embed":
        return vce.ce_embedding(s["ids"], s["w"], s["scale"])
    if op == "embed_bwd":
        return vce.ce_embedding_backward(s["dout"], s["ids"], case["V"], s["scale"], dw=s["dw"],
                                         accumulate=s["dw"] is not None)
    if op == "norm":
        if case["group"] < 0:
            y, total = vce.ce_rms_norm(s["x"], s["w"], s["r"], EPS)
            return [y] if s["r"] is None else [y, total]
        q, scale, total = vce.ce_rms_norm_quant(s["x"], s["w"], s["r"], EPS, group=case["group"])
        return [q, scale] if s["r"] is None else [q, scale, total]
    dx, dw = vce.ce_rms_norm_backward(s["dy"], s["s"], s["w"], EPS, dsum=s["dsum"])
    return [dx, dw]


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without -----------------------------------------------------------------------


def _unique(N, V):
    """Expected number of different ids among N of _tokens()."""
    edge = (np.arange(V + 1) / V) ** 0.25
    return float(-np.expm1(N * np.log1p(-np.minimum(np.diff(edge), 1 - 1e-12))).sum())


def work(case):
    op, eb = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("process"):
        N, V, L = case["d0"] * case["d1"], case["V"], case["L"]
        tokens = case["d0"] * L if case["prefix"] else N * L // 2
        seen = tokens if op == "process_bwd" else 0  # a sign for each seen column
        return dict(bytes=2 * N * V * eb + 8 * tokens + seen + 24 * N + (N * V // 8 if case["mask"] else 0)
                    + (4 * V if case["bias"] else 0), flops=6 * N * V)
    if op == "embed":
        return dict(bytes=(case["N"] + _unique(case["N"], case["V"])) * case["D"] * eb + 8 * case["N"],
                    flops=case["N"] * case["D"])
    if op == "embed_bwd":
        N, V, D = case["N"], case["V"], case["D"]
        return dict(bytes=N * D * eb + 8 * N + (8 * D * _unique(N, V) if case["add"] else 4 * V * D), flops=2 * N * D)
    N, D = case["N"], case["D"]
    if op == "norm":
        out = eb if case["group"] < 0 else 1 + 4.0 / (case["group"] or D)
        return dict(bytes=N * D * (eb + out + (2 * eb if case["residual"] else 0)) + D * eb, flops=5 * N * D)
    return dict(bytes=N * D * eb * (4 if case["residual"] else 3) + D * (eb + 4), flops=12 * N * D)


# ---- the definitions in 64 bits --------------------------------------------------------------------------


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op.startswith("process"):
        src = s["x"] if op == "process" else s["dz"]
        d0, d1, V = src.shape
        N, L = d0 * d1, case["L"]
        z = src.reshape(N, V).double()
        # one entry per history token that counts, as (row, column, in the output?)
        rows = torch.arange(N, device="cuda").view(N, 1).expand(N, L)
        pos = torch.arange(L, device="cuda").expand(N, L)
        tok = s["history"].reshape(N, L)
        ok = (pos < s["history_len"].view(N, 1)) & (tok >= 0) & (tok < V)
        new = (pos >= s["prompt_len"].view(N, 1))[ok]
        where, times = torch.unique(rows[ok] * V + tok[ok], return_inverse=True)
        times = torch.zeros(len(where), dtype=torch.float64, device="cuda").index_add_(0, times, new.double())
        r = where // V
        theta = s["repetition"].double()[r]
        flat = z.view(-1)
        old = flat[where]
        if op == "process":
            old = torch.where(old > 0, old / theta, old * theta)
            old = old - s["frequency"].double()[r] * times - s["presence"].double()[r] * (times > 0).double()
        else:
            bit = (s["signs"].view(-1)[r * s["signs"].shape[1] + where % V // 8].long() >> (where % V % 8)) & 1
            old = torch.where(bit == 1, old / theta, old * theta)
        flat[where] = old
        if op == "process" and s["bias"] is not None:
            z += s["bias"][0, 0].double()
        z /= s["temperature"].double().view(N, 1)
        if s["mask"] is not None:
            j = torch.arange(V, device="cuda")
            words = s["mask"].reshape(N, -1).long() & 0xffffffff
            z[((words[:, j // 32] >> (j % 32)) & 1) == 0] = -math.inf if op == "process" else 0.0
        return z.view(d0, d1, V)
    if op == "embed":
        return torch.nn.functional.embedding(s["ids"], s["w"]).double() * s["scale"]
    if op == "embed_bwd":
        # sums over each id's run of the sorted tokens, as differences of a running sum
        order = torch.sort(s["ids"], stable=True)
        run_sum = torch.cumsum(s["dout"][order.indices].double() * s["scale"], 0)
        ids, counts = torch.unique_consecutive(order.values, return_counts=True)
        ends = run_sum[torch.cumsum(counts, 0) - 1]
        ends[1:] = ends[1:] - ends[:-1].clone()
        dw = torch.zeros((case["V"], case["D"]), dtype=torch.float64, device="cuda")
        if s["dw"] is not None:
            dw += s["dw"]
        dw[ids] += ends
        return dw
    w = s["w"].double()
    if op == "norm":
        t = s["x"].double() + (0 if s["r"] is None else s["r"].double())
        y = t / ((t * t).sum(1) / case["D"] + EPS).sqrt().view(-1, 1) * w
        total = [] if s["r"] is None else [t]
        if case["group"] < 0:
            return [y] + total
        G = case["group"] or case["D"]
        column = torch.arange(case["D"], device="cuda") // G
        top = torch.zeros((case["N"], int(column[-1]) + 1), dtype=torch.float64, device="cuda")
        top.scatter_reduce_(1, column.expand(case["N"], -1), y.abs(), "amax")
        scale = top / FP8_MAX
        return [y / scale[:, column].clamp(min=FP32_TINY), scale.clamp(min=FP32_TINY)] + total
    t, dy = s["s"].double(), s["dy"].double()
    inv = 1.0 / ((t * t).sum(1, keepdim=True) / case["D"] + EPS).sqrt()
    n = t * inv  # the normalised row; y = n w
    ds = inv * (dy * w - n * (dy * w * n).sum(1, keepdim=True) / case["D"])
    return [ds if s["dsum"] is None else ds + s["dsum"].double(), (dy * n).sum(0)]
