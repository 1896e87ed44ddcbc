"""GPU: calls of the serving operators and of the 8-bit cache that are refused, and
calls whose operands are next to each other or next to a limit."""

import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import row_wise_top_topk_amd as mt

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_scales_and_means_with_a_tangent_are_refused():
    pages, hk, bs, d = 4, 2, 16, 64
    cache = {n: torch.zeros(pages, hk, bs, d, device=DEV).to(torch.float8_e4m3fn) for n in ("k_cache", "v_cache")}
    scales = {n: torch.ones(pages, hk, device=DEV) for n in ("k_scale", "v_scale")}
    mean = torch.zeros(pages, hk, d, device=DEV)
    x = torch.zeros(1, hk, d, dtype=torch.bfloat16, device=DEV)
    table, lengths = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    calls = {
        "chunk_attention": lambda c, m: mt.chunk_attention(x, x, x, **c, block_table=table, lengths=lengths),
        "kv8_append": lambda c, m: mt.kv8_append(x, x, **c, block_table=table, lengths=lengths, k_mean=m),
        "kv8_attention": lambda c, m: mt.kv8_attention(x, **c, block_table=table, lengths=lengths),
        "pages_copy": lambda c, m: mt.pages_copy(**c, copies=torch.full((1, 2), -1, dtype=torch.int32, device=DEV), k_mean=m),
    }
    with forward_ad.dual_level():
        for what, call in calls.items():
            call(cache | scales, mean)
            for n in scales:
                with pytest.raises(ValueError, match=f"{n} has a tangent"):
                    call(cache | scales | {n: forward_ad.make_dual(scales[n], scales[n])}, mean)
            if what in ("kv8_append", "pages_copy"):
                with pytest.raises(ValueError, match="k_mean has a tangent"):
                    call(cache | scales, forward_ad.make_dual(mean, mean))
