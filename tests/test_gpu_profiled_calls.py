"""Profiled calls without rows: they run no kernel of their operator's, so they take no pair of events, and the calls
around them are timed."""
import pytest
import torch

import vocab_cross_entropy_amd as vce
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("reduce", ["none", "mean", "sum"])
def test_a_profiled_distillation_without_rows(reduce):
    x = torch.randn((2, 3, 500), device="cuda")
    ids, t = torch.zeros((2, 3, 4), dtype=torch.int64, device="cuda"), torch.randn((2, 3, 4), device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    say(f"[profile] distillation without rows, {reduce}")
    with vce.Profiler(8) as p:
        vce.ce_distill_fwd_bwd(x, ids, t, 1.0, reduce, want_grad=False)
        vce.ce_distill_fwd_bwd(x[:0], ids[:0], t[:0], 1.0, reduce, n_valid=n)
        vce.ce_token_logprobs(x[:0], ids[:0], top_k=2, entropy=True)
        vce.ce_token_logprobs(x, ids)
    assert len(p.ms) == 2 and all(ms > 0 for ms in p.ms)


def test_profiled_losses_without_rows():
    x, t = torch.randn((2, 3, 500), device="cuda"), torch.zeros((2, 3), dtype=torch.int64, device="cuda")
    none, no_t = x[:0], t[:0]
    one = torch.ones(1, device="cuda")
    lse, aux = vce.ce_forward_ex(x, t)[1:3]
    calls = {
        "forward": lambda x, t: vce.ce_forward(x, t, reduce_loss="mean"),
        "fused": lambda x, t: vce.ce_fwd_bwd_fused(x, t, reduce_loss="sum"),
        "shards": lambda x, t: vce.ce_shards_fwd_bwd_fused([x[:, :, :200], x[:, :, 200:]], t),
        "partial statistics": lambda x, t: vce.ce_shard_partial_stats(x, t, 0, 500),
        "backward": lambda x, t: vce.ce_backward_inplace_ex(x, t, lse, aux),
        "scaling": lambda x, t: vce.ce_scale_grad_inplace(x, one, per_row=False),
        "processing": lambda x, t: vce.ce_logits_process(x, temperature=one.expand(6).contiguous()),
    }
    for name, call in calls.items():
        say(f"[profile] {name} without rows")
        with vce.Profiler(4) as p:
            call(none, no_t)
            call(x.clone(), t)
        assert len(p.ms) == 1 and p.ms[0] > 0, name
