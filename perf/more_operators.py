"""Reading log-probabilities off logits and distilling into them, as they are measured.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges, ``prepare(case, seed)`` makes a
case's inputs on the GPU, ``run(state)`` makes one pass through an operator and ``exact(case, seed)`` gives
the same outputs from the definition in 64 bits.  With ``own`` false ``run`` is the plain form in elementary
torch operations (32 bits, one rounding at the end); with ``own`` true it calls the library.

Per row of logits x, with p = softmax(x):
    logprobs      log p of given tokens, the entropy H = -sum p log p, and the K largest logits' columns
                  (ties: the lower column) with their log p
    logprobs_bwd  dx_v = sum over given tokens of g [v = token] - p_v (sum of g + dH (log p_v + H))
    distill       q = softmax(x / T);  loss = T^2 sum_k p_k (log p_k - log q_k) over a teacher's K columns,
                  with p the teacher's softmax over them at T, or its probabilities at T with what they
                  leave of 1 as one more class, all the other columns together; the gradient of x
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a decoding step of one sequence that returns the sampled token's log-probability and alternatives
        dict(name="logprobs one row", op="logprobs", d0=1, d1=1, V=128000, dtype="bf16", M=1, K=20, entropy=False,
             mask=False),
        # a serving batch on processed FP32 logits: a grammar left a quarter of the words, and three in the last row
        dict(name="logprobs batch", op="logprobs", d0=64, d1=1, V=128000, dtype="f32", M=1, K=5, entropy=False,
             mask=True),
        # scoring a policy's samples for training: every position's token, and the entropy
        dict(name="logprobs train", op="logprobs", d0=4, d1=2048, V=128000, dtype="bf16", M=1, K=0, entropy=True,
             mask=False),
        # a teacher's pass: the alternatives that a student will be distilled from
        dict(name="logprobs teacher", op="logprobs", d0=2, d1=1024, V=32000, dtype="bf16", M=0, K=64, entropy=False,
             mask=False),
        # several candidates a position, everything asked for, rows that start at every alignment
        dict(name="logprobs odd", op="logprobs", d0=3, d1=171, V=32003, dtype="f32", M=7, K=17, entropy=True,
             mask=False),
        # the training step's gradient, of the tokens and of an entropy bonus
        dict(name="logprobs backward", op="logprobs_bwd", d0=4, d1=2048, V=128000, dtype="bf16", M=1, entropy=True),
        # the gradient of several candidates, among them the same twice, FP32, odd rows
        dict(name="logprobs backward odd", op="logprobs_bwd", d0=2, d1=512, V=32003, dtype="f32", M=5,
             entropy=False),
        # the training step of a distillation over a teacher's 64 largest logits
        dict(name="distill train", op="distill", d0=4, d1=2048, V=128000, dtype="bf16", K=64, T=2.0, tail=False,
             ragged=False, reduce="mean", grad=True),
        # log-probabilities of a teacher behind an interface that returns 20, with padded positions
        dict(name="distill tail", op="distill", d0=2, d1=1024, V=32000, dtype="bf16", K=20, T=1.0, tail=True,
             ragged=True, reduce="mean", grad=True),
        # FP32, odd rows, losses of each row
        dict(name="distill odd", op="distill", d0=1, d1=515, V=32003, dtype="f32", K=50, T=1.5, tail=False,
             ragged=True, reduce="none", grad=True),
        # a few rows of a small vocabulary
        dict(name="distill few", op="distill", d0=1, d1=16, V=8192, dtype="bf16", K=16, T=4.0, tail=True,
             ragged=False, reduce="sum", grad=True),
        # the evaluation: the loss alone
        dict(name="distill evaluate", op="distill", d0=2, d1=512, V=128000, dtype="bf16", K=100, T=1.0, tail=False,
             ragged=True, reduce="sum", grad=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs_bwd", "distill", "distill"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    V = rng.choice([128000, 32000, _log(rng, 300, 200000), _log(rng, 300, 200000)])
    # rows up to 2048 x 128000 logits in all
    d0 = _log(rng, 1, 64)
    d1 = max(1, min(rng.choice([1, _log(rng, 1, 2048)]), (2048 * 128000) // (d0 * V)))
    case = dict(op=op, d0=d0, d1=d1, V=V, dtype=dtype)
    if op == "logprobs":
        M = rng.choice([0, 1, 1, _log(rng, 1, 32)])
        K = rng.choice([0, 1, 5, 20, _log(rng, 1, 128)])
        case.update(M=M, K=K, entropy=rng.random() < 0.5 or M + K == 0, mask=rng.random() < 0.3)
    elif op == "logprobs_bwd":
        case.update(M=rng.choice([1, 1, _log(rng, 1, 32)]), entropy=rng.random() < 0.5)
    else:
        case.update(K=_log(rng, 1, 128), T=round(rng.uniform(0.8, 4.0), 2), tail=rng.random() < 0.4,
                    ragged=rng.random() < 0.5, reduce=rng.choice(["mean", "sum", "none"]), grad=rng.random() < 0.8)
    return case


def _rows(N, V, budget=1 << 28):
    """Row ranges that keep a pass of 64-bit intermediates within memory."""
    step = max(1, budget // V)
    return [slice(i, min(N, i + step)) for i in range(0, N, step)]


def _distinct(N, n, V, g):
    """n distinct columns of each of N rows: steps of 1 to V // n from a random start, wrapped."""
    gaps = torch.randint(1, V // n + 1, (N, n), generator=g, device="cuda")
    return (gaps.cumsum(1) + torch.randint(0, V, (N, 1), generator=g, device="cuda")) % V


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)
    d0, d1, V, op = case["d0"], case["d1"], case["V"], case["op"]
    N, dt = d0 * d1, DTYPES[case["dtype"]]

    def normal(*shape, sigma=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(sigma)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(case=case)
    x = normal(N, V, sigma=2.0, dtype=dt)
    if op == "distill":
        K = min(case["K"], V)
        ids = _distinct(N, K, V, g)
        # the teacher's logits fall off with rank; the student has learnt a part of it
        t = 9.0 - 1.5 * torch.arange(1, K + 1, device="cuda").float().log() + normal(N, K, sigma=0.7)
        t = t.sort(1, descending=True).values
        x.scatter_(1, ids, (t * uniform(N, 1, lo=0.5, hi=1.0) + normal(N, K)).to(dt))
        if case["tail"]:  # log-probabilities; 0.1% to 30% of the teacher's mass lies elsewhere
            t = t / case["T"]
            t = t - t.logsumexp(1, keepdim=True) + torch.log1p(-torch.exp(uniform(N, 1, lo=-6.9, hi=-1.2)))
        s["teacher_ids"], s["teacher"] = ids.view(d0, d1, K), t.view(d0, d1, K)
        s["teacher_len"] = None
        if case["ragged"]:  # every tenth row is padding, others have up to K entries
            n = torch.randint((K + 1) // 2, K + 1, (N,), generator=g, device="cuda", dtype=torch.int32)
            n[3::10] = 0
            s["teacher_len"] = n
            s["teacher_ids"] = s["teacher_ids"].masked_fill(
                torch.arange(K, device="cuda") >= n.view(d0, d1, 1), -100)
        s["x"] = x.view(d0, d1, V)
        s["out"] = torch.empty_like(s["x"]) if case["grad"] else None
        s["loss"] = torch.empty(N if case["reduce"] == "none" else 1, device="cuda")
        s["ws"] = None  # made by the library's call, kept for its next
        return s
    M = case["M"]
    if M:
        ids = _distinct(N, M, V, g)
        # tokens are sampled ones: most of them are likely, some nearly certain
        x.scatter_add_(1, ids, uniform(N, M, lo=0.0, hi=14.0).to(dt))
        if op == "logprobs_bwd" and M > 2:
            ids[::2, 2] = ids[::2, 0]
        ids[5::16, 0] = -100  # padding
        s["ids"] = ids.view(d0, d1, M)
    else:
        s["ids"] = None
    s["x"] = x.view(d0, d1, V)
    if op == "logprobs":
        if case["mask"]:
            for r in _rows(N, V):
                x[r].masked_fill_(torch.rand(x[r].shape, generator=g, device="cuda") < 0.75, -math.inf)
            x[:, 0] = 1.0  # something is left in every row
            x[-1, 4:] = -math.inf
            x[-1, :4] = torch.tensor([1.0, -math.inf, 0.5, 1.0])[:V].to(dt)
            if M:  # what is masked was not sampled
                s["ids"] = torch.where(s["ids"] < 0, s["ids"], 0)
        s["ws"] = None
        return s
    s["dlogp"] = normal(d0, d1, M)
    s["dentropy"] = normal(d0, d1, sigma=0.01) if case["entropy"] else None
    # what the forward pass handed over: the largest logit, the log-sum relative to it, 1 - its probability, H
    stats = torch.empty((N, 4), device="cuda")
    for r in _rows(N, V):
        z = x[r].double()
        m = z.amax(1, keepdim=True)
        z -= m
        rest = z.exp().sum(1) - 1.0
        u = torch.log1p(rest)
        h = u - (z.exp() * z).sum(1) / (1.0 + rest)
        stats[r] = torch.stack([m[:, 0], u, rest / (1.0 + rest), h], 1).float()
    s["stats"] = stats
    s["out"] = torch.empty_like(s["x"])
    return s


# ---- the plain forms -------------------------------------------------------------------------------------


def _log_softmax(x):
    z = x.float()
    z = z - z.amax(-1, keepdim=True)
    return z - z.exp().sum(-1, keepdim=True).log()


def _plain_logprobs(s):
    case = s["case"]
    logp = _log_softmax(s["x"])
    out = []
    if s["ids"] is not None:
        ids = s["ids"]
        out.append(torch.where(ids < 0, 0.0, logp.gather(2, ids.clamp(min=0))))
    if case["entropy"]:
        p = logp.exp()
        out.append(-torch.where(p > 0, p * logp, 0.0).sum(-1))
    if case["K"]:
        K = min(case["K"], case["V"])
        order = torch.sort(s["x"].float(), dim=2, descending=True, stable=True).indices[..., :K]
        out += [order, logp.gather(2, order)]
    return out


def _plain_logprobs_bwd(s):
    x, ids = s["x"], s["ids"]
    m, u, _, h = s["stats"].view(*x.shape[:2], 4, 1).unbind(2)
    logp = (x.float() - m) - u
    given = torch.where(ids < 0, 0.0, s["dlogp"])
    slope = given.sum(2, keepdim=True)
    if s["dentropy"] is not None:
        slope = slope + s["dentropy"].unsqueeze(2) * (logp + h)
    dx = -logp.exp() * slope
    return dx.scatter_add_(2, ids.clamp(min=0), given).to(x.dtype)


def _plain_distill(s):
    case = s["case"]
    T, tail = case["T"], case["tail"]
    x, ids, t = s["x"].float() / T, s["teacher_ids"], s["teacher"]
    N, V = x.shape[0] * x.shape[1], x.shape[2]
    have = torch.ones_like(ids, dtype=torch.bool)
    if s["teacher_len"] is not None:
        have = torch.arange(ids.shape[2], device=x.device) < s["teacher_len"].view(*x.shape[:2], 1)
    row = have.any(2)
    n = row.sum()
    ids = torch.where(have, ids, 0)
    if tail:
        p = torch.where(have, t.exp(), 0.0)
        left = (1.0 - p.sum(2)).clamp(min=0.0)
        logt = t
    else:
        logt = torch.where(have, t / T, -math.inf)
        logt = logt - logt.amax(2, keepdim=True)
        logt = logt - logt.exp().sum(2, keepdim=True).log()
        p = torch.where(have, logt.exp(), 0.0)
    logq = _log_softmax(x)
    q = logq.exp()
    loss = torch.where(p > 0, p * (logt - logq.gather(2, ids)), 0.0).sum(2)
    if tail:
        others = torch.ones_like(q).scatter_reduce_(2, ids, (~have).float(), "amin")
        mass = (q * others).sum(2)
        loss = loss + torch.where(left > 0, left * (left.log() - mass.log()), 0.0)
    loss = torch.where(row, loss * (T * T), 0.0)
    total = loss.view(-1) if case["reduce"] == "none" else loss.sum().view(1)
    if case["reduce"] == "mean":
        total = total / n
    if not case["grad"]:
        return [total]
    if tail:
        dx = q * (1.0 - others * (left / mass).unsqueeze(2))
    else:
        dx = q
    dx = dx.scatter_add(2, ids, -p) * T
    if case["reduce"] == "mean":
        dx = dx / n
    return [total, torch.where(row.unsqueeze(2), dx, 0.0).to(s["x"].dtype)]


_PLAIN = dict(logprobs=_plain_logprobs, logprobs_bwd=_plain_logprobs_bwd, distill=_plain_distill)


# ---- the library's calls ---------------------------------------------------------------------------------


def _own(s):
    import vocab_cross_entropy_amd as vce

    case = s["case"]
    if case["op"] == "logprobs":
        K = min(case["K"], case["V"])
        if s["ws"] is None:
            s["ws"] = vce.ce_workspace_init(torch.empty(
                vce.ce_token_logprobs_workspace_bytes(s["x"], top_k=K), dtype=torch.uint8, device="cuda"))
        r = vce.ce_token_logprobs(s["x"], s["ids"], top_k=K, entropy=case["entropy"], ws=s["ws"])
        return [t for t in (r.logprobs, r.entropy, r.top_ids, r.top_logprobs) if t is not None]
    if case["op"] == "logprobs_bwd":
        return vce.ce_token_logprobs_backward(s["x"], s["stats"], s["ids"], s["dlogp"], dentropy=s["dentropy"],
                                              out=s["out"])
    if s["ws"] is None:
        s["ws"] = vce.ce_workspace_init(torch.empty(
            vce.ce_distill_workspace_bytes(s["x"]), dtype=torch.uint8, device="cuda"))
    vce.ce_distill_fwd_bwd(s["x"], s["teacher_ids"], s["teacher"], case["T"], case["reduce"],
                           teacher="logprobs" if case["tail"] else "logits", teacher_len=s["teacher_len"],
                           out=s["out"], want_grad=case["grad"], loss=s["loss"], ws=s["ws"])
    return [s["loss"]] + ([s["out"]] if case["grad"] else [])


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without -----------------------------------------------------------------------


def work(case):
    N, V, eb = case["d0"] * case["d1"], case["V"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "logprobs":
        return dict(bytes=N * (V * eb + 12 * case["M"] + 12 * case["K"] + (4 if case["entropy"] else 0)),
                    flops=(6 if case["entropy"] else 4) * N * V)
    if case["op"] == "logprobs_bwd":
        return dict(bytes=N * (2 * V * eb + 12 * case["M"] + 16 + (4 if case["entropy"] else 0)),
                    flops=(6 if case["entropy"] else 4) * N * V)
    return dict(bytes=N * ((2 if case["grad"] else 1) * V * eb + 12 * case["K"]),
                flops=(8 if case["grad"] else 4) * N * V)


# ---- the definitions in 64 bits --------------------------------------------------------------------------


def _largest(x, K):
    """Columns of the K largest of each row, by whole-number keys: the value's bits in order, then the column."""
    bits = (x.float() + 0.0).view(torch.int32).long()
    key = torch.where(bits >= 0, bits, -(bits & 0x7fffffff)) * (1 << 32)
    key = key + (x.shape[1] - 1 - torch.arange(x.shape[1], device=x.device))
    return x.shape[1] - 1 - (key.topk(K, dim=1).values & 0xffffffff)


def exact(case, seed):
    s = prepare(case, seed)
    op, d0, d1, V = case["op"], case["d0"], case["d1"], case["V"]
    N = d0 * d1
    x = s["x"].view(N, V)
    if op == "logprobs":
        parts = []
        for r in _rows(N, V, 1 << 27):
            z = x[r].double()
            lse = torch.logsumexp(z, 1, keepdim=True)
            part = []
            if s["ids"] is not None:
                ids = s["ids"].view(N, -1)[r]
                part.append((z.gather(1, ids.clamp(min=0)) - lse) * (ids >= 0))
            if case["K"]:
                top = _largest(x[r], min(case["K"], V))
                tops = [top, z.gather(1, top) - lse]
            if case["entropy"]:
                p = torch.softmax(z, 1)
                part.append(lse[:, 0] - (p * z.clamp(min=-1e30)).sum(1))
            parts.append(part + (tops if case["K"] else []))
        return [torch.cat(c).view(d0, d1, *c[0].shape[1:]) for c in zip(*parts)]
    if op == "logprobs_bwd":
        M = case["M"]
        dx = torch.empty((N, V), dtype=torch.float64, device="cuda")
        ids, dlogp = s["ids"].view(N, M), s["dlogp"].view(N, M).double()
        for r in _rows(N, V, 1 << 27):
            z = x[r].double()
            lse = torch.logsumexp(z, 1, keepdim=True)
            p = torch.softmax(z, 1)
            d = torch.zeros_like(z)
            for m in range(M):
                g = (dlogp[r, m] * (ids[r, m] >= 0)).unsqueeze(1)
                d -= g * p
                d.scatter_add_(1, ids[r, m:m + 1].clamp(min=0), g)
            if s["dentropy"] is not None:
                # H = lse - sum p z;  dH/dz = p (E[z] - z)
                d += s["dentropy"].view(N, 1)[r].double() * p * ((p * z).sum(1, keepdim=True) - z)
            dx[r] = d
        return dx.view(d0, d1, V)
    K, T = min(case["K"], V), float(case["T"])
    ids, t = s["teacher_ids"].view(N, K), s["teacher"].view(N, K).double()
    length = torch.full((N,), K, device="cuda") if s["teacher_len"] is None else s["teacher_len"].long()
    n = int((length > 0).sum())
    scale = 1.0 / n if case["reduce"] == "mean" else 1.0
    losses = torch.empty(N, dtype=torch.float64, device="cuda")
    dx = torch.empty((N, V), dtype=torch.float64, device="cuda") if case["grad"] else None
    for r in _rows(N, V, 1 << 27):
        z = x[r].double() / T
        rows, k = torch.nonzero(torch.arange(K, device="cuda") < length[r].unsqueeze(1), as_tuple=True)
        col, lt = ids[r][rows, k], t[r][rows, k]
        target = torch.zeros_like(z)  # the teacher's probabilities in their columns
        if case["tail"]:
            target[rows, col] = lt.exp()
            rest = z.clone()
            rest[rows, col] = -math.inf
            log_rest = torch.logsumexp(rest, 1, keepdim=True)
            left = (1.0 - target.sum(1, keepdim=True)).clamp(min=0.0)
        else:
            w = torch.full_like(z, -math.inf)
            w[rows, col] = lt / T
            target = torch.nan_to_num(torch.softmax(w, 1))  # rows without an entry come out 0
        lse = torch.logsumexp(z, 1, keepdim=True)
        cross = -(target * (z - lse)).sum(1)
        loss = cross + torch.xlogy(target, target).sum(1)
        d = torch.exp(z - lse) - target
        if case["tail"]:
            loss += (torch.xlogy(left, left) - left * (log_rest - lse))[:, 0]
            d -= left * torch.exp(rest - log_rest)
        on = (length[r] > 0).double()
        losses[r] = torch.where(on > 0, loss * T * T, 0.0)
        if dx is not None:
            dx[r] = d * (on * T * scale).unsqueeze(1)
    total = losses if case["reduce"] == "none" else (losses.sum() * scale).view(1)
    return [total] + ([dx] if case["grad"] else [])
