"""Several losses on one tensor of logits.  Those that stage their gradient in the logits' storage tell autograd, so a
function that keeps the logits for its backward refuses; on a copy both give the gradient of their sum."""
import numpy as np
import pytest
import torch

import vocab_cross_entropy_amd as vce
from gpu_util import say
from ops_util import assert_within
from score_util import f64, half_step, ref_distill, ref_logprobs_grad

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
D0, D1, V, K, T = 2, 3, 1203, 6, 2.0
N = D0 * D1


def _inputs(dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((D0, D1, V), generator=g) * 2).to(dtype)
    ids = torch.randint(0, V, (D0, D1), generator=g)
    t_ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)]).view(D0, D1, K)
    return x, ids, t_ids, torch.randn((D0, D1, K), generator=g)


LOSSES = {
    "distillation": lambda z, ids, ti, tv: vce.distillation_loss(z, ti, tv, T, "sum"),
    "cross_entropy": lambda z, ids, ti, tv: vce.parallel_cross_entropy(z, ids, 0.0, "sum"),
    "processed": lambda z, ids, ti, tv: vce.processed_cross_entropy(z, ids, 0.0, "sum",
                                                                    temperature=torch.full((N,), 1.5, device="cuda")),
    "sharded": lambda z, ids, ti, tv: vce.sharded_cross_entropy([z[:, :, :600], z[:, :, 600:]], ids, 0.0, "sum"),
}


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", LOSSES)
def test_a_loss_over_kept_logits_is_refused(name, dtype):
    dev = [t.cuda() for t in _inputs(dtype)]
    leaf = dev[0].requires_grad_()
    z = leaf * 1
    say(f"shared logits: token_logprobs, then {name}")
    r = vce.token_logprobs(z, dev[1], entropy=True)
    loss = LOSSES[name](z, *dev[1:])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        (r.logprobs.sum() + r.entropy.sum() + loss).backward()


@pytest.mark.parametrize("first,second", [("distillation", "cross_entropy"), ("cross_entropy", "distillation"),
                                          ("distillation", "distillation"), ("processed", "distillation")])
def test_two_staged_losses_are_refused(first, second):
    dev = [t.cuda() for t in _inputs(BF16)]
    z = dev[0].requires_grad_() * 1
    say(f"shared logits: {first}, then {second}")
    loss = LOSSES[first](z, *dev[1:]) + LOSSES[second](z, *dev[1:])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_raw_calls_over_kept_logits():
    """The calls that write over logits, without autograd: so too; those that leave them as they are do not count."""
    x, ids, ti, tv = (t.cuda() for t in _inputs(F32))
    ti, tv = ti.contiguous(), tv.contiguous()
    lse = vce.ce_forward(x, ids)[1]
    g = torch.ones(N, device="cuda")
    stats = vce.ce_token_logprobs(x, stats=True).stats
    half = torch.full((N,), 0.5, device="cuda")
    loss, nv = torch.empty(N, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    writes = {
        "fused": lambda z: vce.ce_fwd_bwd_fused(z, ids),
        "fused, no allocation": lambda z: vce.ce_fwd_bwd_fused_noalloc(z, ids, loss=loss, n_valid=nv),
        "backward": lambda z: vce.ce_backward_inplace(z, ids, lse),
        "shards": lambda z: vce.ce_shards_fwd_bwd_fused([z[:, :, :600], z[:, :, 600:]], ids),
        "processing": lambda z: vce.ce_logits_process(z, temperature=half),
        "processing into itself": lambda z: vce.ce_logits_process(z, out=z.view(z.shape), temperature=half),
        "distillation": lambda z: vce.ce_distill_fwd_bwd(z, ti, tv),
        "distillation into itself": lambda z: vce.ce_distill_fwd_bwd(z, ti, tv, out=z.view(z.shape)),
        "log-probabilities' gradient": lambda z: vce.ce_token_logprobs_backward(z, stats, ids, g, out=z),
        "the same, into itself": lambda z: vce.ce_token_logprobs_backward(z, stats, ids, g, out=z.view(z.shape)),
    }
    leaves = {
        "forward": lambda z: vce.ce_forward(z, ids),
        "log-probabilities": lambda z: vce.ce_token_logprobs(z, ids, top_k=2),
        "processing elsewhere": lambda z: vce.ce_logits_process(z, out=torch.empty_like(z), temperature=half),
        "the loss alone": lambda z: vce.ce_distill_fwd_bwd(z, ti, tv, want_grad=False),
        "distillation elsewhere": lambda z: vce.ce_distill_fwd_bwd(z, ti, tv, out=torch.empty_like(z)),
        "gradient elsewhere": lambda z: vce.ce_token_logprobs_backward(z, stats, ids, g),
    }
    for name, call in {**writes, **leaves}.items():
        say(f"shared logits: {name}")
        z = x.clone().requires_grad_() * 1
        r = vce.token_logprobs(z, ids)
        with torch.no_grad():
            call(z.detach())
        if name in writes:
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                r.logprobs.sum().backward()
        else:
            r.logprobs.sum().backward()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_a_copy_for_one_of_them(dtype):
    """Log-probabilities with an entropy bonus and a distillation, the latter on a copy: the gradient of the sum."""
    x, ids, ti, tv = _inputs(dtype)
    leaf = x.cuda().requires_grad_()
    z = leaf * 1
    r = vce.token_logprobs(z, ids.cuda(), entropy=True)
    loss = vce.distillation_loss(z.clone(), ti.cuda(), tv.cuda(), T, "sum")
    (r.logprobs.sum() + 0.5 * r.entropy.sum() + loss).backward()
    a, ta = ref_logprobs_grad(f64(x).reshape(N, V), ids.reshape(N, 1).numpy(), np.ones((N, 1)), np.full(N, 0.5), dtype=dtype)
    _, _, b, tb = ref_distill(f64(x).reshape(N, V), ti.reshape(N, K).numpy(), f64(tv).reshape(N, K), np.full(N, K), T, False,
                              np.ones(N), dtype)
    # autograd adds the two in the logits' type
    tol = ta + tb + 1.01 * half_step(dtype) * (np.abs(a + b) + ta + tb)
    assert_within(f64(leaf.grad).reshape(N, V), a + b, tol, "dx")


def test_what_autograd_allows_still_runs():
    """The leaf itself, a view of it, no_grad and inference mode, and a second backward of a kept graph."""
    dev = [t.cuda() for t in _inputs(F32)]
    for name, call in LOSSES.items():
        say(f"shared logits: {name} by itself")
        leaf = dev[0].clone().requires_grad_()
        call(leaf, *dev[1:]).backward()
        want = leaf.grad
        leaf = dev[0].clone().requires_grad_()
        call(leaf.view(D0, D1, V), *dev[1:]).backward()
        assert torch.equal(leaf.grad, want), name
        leaf = dev[0].clone().requires_grad_()
        loss = call(leaf * 1, *dev[1:])
        loss.backward(retain_graph=True)
        loss.backward()
        assert torch.equal(leaf.grad, 2 * want), name
        with torch.inference_mode():
            call(dev[0].clone(), *dev[1:])
        with torch.no_grad():
            call(dev[0].clone(), *dev[1:])
