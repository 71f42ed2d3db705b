"""One workspace for a loss that keeps its rows' plain FP32 losses there and for the calls that exchange tagged words: what
the former leaves never passes for a word of the latter."""
import math

import numpy as np
import pytest
import torch

import vocab_cross_entropy_amd as vce
from gpu_util import say

pytestmark = pytest.mark.gpu


def _losses_like_tags(N, ws):
    """A mean over N rows, whose losses' bits are the tag of the next call (set here: that of the 1.06e9th)."""
    x, t = torch.zeros((1, N, 2), device="cuda"), torch.zeros((1, N), dtype=torch.int64, device="cuda")
    vce.ce_forward(x, t, reduce_loss="mean", ws=ws)
    losses = ws.view(torch.int32)[64:64 + N]
    tag = int(losses[0])
    assert bool((losses == tag).all()) and abs(float(losses.view(torch.float32)[0]) - math.log(2)) < 1e-6
    ws.view(torch.int64)[3] = tag


@pytest.mark.parametrize("grad", [True, False], ids=["gradient", "loss_alone"])
def test_distillation_after_a_mean(grad):
    """Row 0 is brought together late (a chunk that publishes nothing, forced from the host, and a bounded wait), so the
    sum has to wait for its NaN."""
    N, V, K = 8, 70001, 6
    g = torch.Generator().manual_seed(1)
    x = torch.randn((1, N, V), generator=g).to(torch.bfloat16).cuda()
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)]).view(1, N, K).cuda()
    t = torch.randn((1, N, K), generator=g).cuda()
    ws = vce.ce_workspace_init(torch.empty(vce.ce_distill_workspace_bytes(x), dtype=torch.uint8, device="cuda"))
    words = ws.view(torch.int64)
    out = dict(out=torch.empty_like(x)) if grad else dict(want_grad=False)
    say("distillation on a workspace with the rows' losses of a mean")
    _losses_like_tags(N, ws)
    words[4] = (0 + 1) << 8 | 1
    total, _ = vce.ce_distill_fwd_bwd(x, ids, t, 1.0, "sum", ws=ws, **out)
    assert math.isnan(float(total))
    with pytest.raises(vce.CeError):
        vce.ce_workspace_check(ws)
    words[4] = 0
    rows, _ = vce.ce_distill_fwd_bwd(x, ids, t, 1.0, "none", ws=ws, **out)
    _losses_like_tags(N, ws)
    total, _ = vce.ce_distill_fwd_bwd(x, ids, t, 1.0, "sum", ws=ws, **out)
    assert float(total) == float(np.float32(rows.double().sum().item()))
    vce.ce_workspace_check(ws)


def test_regions_do_not_meet():
    """The words of both calls lie behind 4 bytes a row: what they leave there starts past them."""
    N, V, K = 6, 70001, 5
    x = torch.randn((1, N, V), device="cuda")
    ids = torch.arange(K, device="cuda").view(1, 1, K).expand(1, N, K)
    t = torch.randn((1, N, K), device="cuda")
    n = max(vce.ce_distill_workspace_bytes(x), vce.ce_token_logprobs_workspace_bytes(x, K))
    say("regions of a shared workspace")
    for call in (lambda ws: vce.ce_distill_fwd_bwd(x, ids, t, 1.0, "mean", out=torch.empty_like(x), ws=ws),
                 lambda ws: vce.ce_token_logprobs(x, ids, top_k=K, ws=ws)):
        ws = vce.ce_workspace_init(torch.empty(n, dtype=torch.uint8, device="cuda"))
        call(ws)
        torch.cuda.synchronize()
        body = ws[256:]
        assert not bool(body[:4 * N].any()) and bool(body[4 * N:].any())
