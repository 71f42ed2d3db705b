"""Counts that do not fit the C interface's 32 bits are refused, not taken modulo 2^32."""
import pytest
import torch

import vocab_cross_entropy_amd as vce


@pytest.mark.parametrize("top_k", [-1, 129, 1 << 31, (1 << 32) + 5, -(1 << 32) + 5, 1 << 64])
def test_alternatives_out_of_range(top_k):
    x = torch.zeros(1, 2, 500)  # host memory, never read: sizes alone
    assert vce.ce_token_logprobs_workspace_bytes(x, 5) == 256
    with pytest.raises(vce.CeArgumentError) as e:
        vce.ce_token_logprobs_workspace_bytes(x, top_k)
    assert e.value.status == vce._abi.CE_EINVAL
