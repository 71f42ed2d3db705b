"""Alternatives of rows that hold NaN of every kind, signalling ones among them: the largest logits all the same, NaN
last."""
import math

import numpy as np
import pytest
import torch

import vocab_cross_entropy_amd as vce
from gpu_util import say
from score_util import f64, largest

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAMES = {BF16: "bf16", F32: "f32"}
# quiet and signalling, of both signs, of the smallest and the largest payload
PATTERNS = {BF16: (0x7FC0, 0x7F81, 0x7FBF, -0x7F, -0x41, -0x1),
            F32: (0x7FC00000, 0x7F800001, 0x7FBFFFFF, -0x7FFFFF, -0x400001, -0x1)}


def _with_nan(x, at, pattern):
    """The row with a bit pattern in some columns."""
    bits = x.view(torch.int16 if x.dtype is BF16 else torch.int32).clone()
    bits[at] = pattern
    return bits.view(x.dtype)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("N,V", [(40, 700), (40, 1500), (40, 5003), (40, 40001), (600, 5003), (512, 20001)],
                         ids=["wave", "wave_8", "chunks_2", "chunks", "streamed", "streamed_8"])
def test_alternatives_beside_nan(N, V, dtype):
    g = torch.Generator().manual_seed(V)
    assert all(bool(torch.tensor([p], dtype=torch.int16 if dtype is BF16 else torch.int32).view(dtype).isnan())
               for p in PATTERNS[dtype])
    rows = []
    for i, pattern in enumerate(PATTERNS[dtype]):
        for near in (1, -1, 2, -2, 3, 7):
            x = (torch.randn((V,), generator=g) * 2).to(dtype)
            peaks = torch.randperm(V - 20, generator=g)[:30] + 10
            x[peaks] = (torch.rand((30,), generator=g) * 8 + 20).to(dtype)  # the largest
            x[peaks[0]] = 60.0
            at = (peaks + near)[~torch.isin(peaks + near, peaks)]
            rows.append(_with_nan(x, at, pattern))
        rows.append(_with_nan((torch.randn((V,), generator=g) * 2).to(dtype), torch.arange(V) % 2 == i % 2, pattern))
        x = (torch.randn((V,), generator=g)).to(dtype)
        x[V // 2:] = -math.inf
        rows.append(_with_nan(x, torch.arange(5, V, 11), pattern))
    R = len(rows)
    x = torch.stack(rows).cuda()[(torch.arange(N) % R).cuda()].view(1, N, V)
    for K in (1, 20, 128):
        say(f"alternatives beside NaN {NAMES[dtype]} {N}x{V} K{K}")
        got = vce.ce_token_logprobs(x, top_k=K, entropy=True)
        want = largest(f64(torch.stack(rows)), K)
        have = got.top_ids.cpu().numpy()[0]
        for r in range(N):
            assert np.array_equal(have[r], want[r % R]), f"K={K}, row {r}: {have[r][:6]}, not {want[r % R][:6]}"
        assert bool(got.top_logprobs.isnan().all()) and bool(got.entropy.isnan().all())
