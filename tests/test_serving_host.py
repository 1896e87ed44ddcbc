"""What the binding of the serving operators decides on the host."""

import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import row_wise_top_topk_amd as mt


@pytest.mark.parametrize("name", ["logits", "repetition", "presence", "frequency", "bias"])
def test_operands_with_a_tangent_are_refused(name):
    """A tangent would be dropped without a word."""
    x = {"logits": torch.zeros(2, 5), "tokens": torch.zeros(2, 3, dtype=torch.int32), "bias_ids": torch.zeros(2, 1, dtype=torch.int32),
         "bias": torch.zeros(2, 1)} | {n: torch.ones(2) for n in ("repetition", "presence", "frequency")}
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="GPU"):    # (of the host: all else is as it should be)
            mt.penalize_logits(**x)
        with pytest.raises(ValueError, match=f"{name} has a tangent"):
            mt.penalize_logits(**(x | {name: forward_ad.make_dual(x[name], torch.ones_like(x[name]))}))
