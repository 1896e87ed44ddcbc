"""What the attention operators decide on the host: no GPU needed."""

import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import row_wise_top_topk_amd as mt


def test_forward_mode_derivatives_are_refused():
    """A tangent would be dropped without a word."""
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    blocks = torch.zeros(4, 2, 1, dtype=torch.int32)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        calls = [lambda: mt.block_means(dual, 16), lambda: mt.block_scores(dual, x.float(), 16, 1),
                 lambda: mt.block_attention(dual, x, x, blocks, 16),
                 lambda: mt.block_attention_backward(x, dual, x, x, x, None, blocks, 16),
                 lambda: mt.kv8_append(dual, x, *[None] * 6), lambda: mt.kv8_attention(dual, *[None] * 6)]
        for call in calls:
            with pytest.raises(ValueError, match="forward-mode"):
                call()
        # the operands themselves are looked at: a primal of a level has no tangent
        with pytest.raises(ValueError, match="GPU"):
            mt.block_means(forward_ad.unpack_dual(dual).primal, 16)
