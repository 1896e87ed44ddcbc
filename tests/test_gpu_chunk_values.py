"""GPU: attention of a chunk whose values are small or large as a whole, or not finite.

Tolerances as in test_gpu_chunk.py.  Where all of a result comes from keys of one
value it is also relative to the result: a weight's rounding (u), the result's (u),
and 2 e of the scores; fp16 results below 2^-14 are rounded to multiples of 2^-24.
"""

import math

import pytest
import torch

import row_wise_top_topk_amd as mt
from test_gpu_chunk import build, check, put, want_of

pytestmark = pytest.mark.gpu

F16 = 2 ** -11


def far_ahead(ratio, n, d, bs, v_exponent, in_cache):
    """One key of value 0 far ahead of n others: 2^-ratio each, of one code.  Returns
    the inputs, what the others add up to, and the error of the scores."""
    x = build(1, [n + 1 + in_cache], [1], 1, 1, d, bs, torch.float16)
    for name in ("q", "k", "v"):
        x[name].zero_()
    x["k_cache"].zero_()
    x["k_scale"].fill_(1.0)
    x["v_cache"].fill_(256.0)
    x["v_scale"].fill_(2.0 ** v_exponent)
    x["q"][0, 0, 0] = 16.0
    want = ratio * math.log(2) / 16 * math.sqrt(d)
    if in_cache:  # the key ahead is the cache's first one, in a page whose scale is 1
        page = int(x["block_table"][0, 0])
        x["k"][0, 0, 0] = -60000.0   # the new token has no weight
        x["k_cache"][page, 0, 0, 0], x["k_scale"][page, 0] = 256.0, want / 256
        x["v_cache"][page], x["v_scale"][page, 0] = 0.0, 1.0
        score, some = 16 * float(x["k_scale"][page, 0]) * 256 / math.sqrt(d), n + 1 - bs
    else:
        x["k"][0, 0, 0] = want
        score, some = 16 * float(x["k"][0, 0, 0]) / math.sqrt(d), n
    p = math.exp(-score)
    return x, 256 * 2.0 ** v_exponent * some * p / (1 + n * p), 2 ** -24 * (d + 64) * score + 2 ** -22 * score


@pytest.mark.parametrize("max_length", [1, None])    # the walk in one part, in several
@pytest.mark.parametrize("d,bs", [(64, 16), (64, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("v_exponent", [-24, -17, -16, -15, -13, -5, 7, 8, 20])
def test_fp16_small_weights_of_values_of_any_size(v_exponent, d, bs, max_length):
    n = 32000
    for ratio in (20, 22):
        x, want, e = far_ahead(ratio, n, d, bs, v_exponent, 0)
        got = mt.chunk_attention(**put(x), max_length=max_length)[0].cpu().double()
        if want * (1 - F16) > 65504:
            continue
        # below 2^-15 a scale's rest joins the weight, which is 2^12 times as large and rounded to 2^-24
        rest = n * 2 ** -37 * 256 * 2 ** -15 if v_exponent < -15 else 0.0
        assert ((got - want).abs() <= (4 * F16 + 2 * e) * want + 2 ** -25 + rest).all(), (got.flatten()[0].item(), want)


@pytest.mark.parametrize("max_length", [1, None])
@pytest.mark.parametrize("d,bs", [(64, 32), (128, 128)])
@pytest.mark.parametrize("v_exponent", [-15, -10])
def test_fp16_pages_of_different_scales(v_exponent, d, bs, max_length):
    x, want, e = far_ahead(20, 32000, d, bs, v_exponent, 1)
    got = mt.chunk_attention(**put(x), max_length=max_length)[0].cpu().double()
    assert ((got - want).abs() <= (4 * F16 + 2 * e) * want + 2 ** -25).all(), (got.flatten()[0].item(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,new,heads,hk,d,bs", [([300, 90], [70, 33], 6, 3, 64, 16), ([700], [260], 8, 1, 128, 32), ([1500], [700], 4, 2, 64, 64),
                                                    ([900, 65], [300, 65], 4, 1, 128, 128)], ids=str)
def test_small_values_and_any_scales(dtype, lens, new, heads, hk, d, bs):
    g = torch.Generator().manual_seed(len(lens))
    for low, high, by in ((-22, -13, -8), (-18, 9, 0), (5, 9, 5)):
        x = build(high + 30, lens, new, heads, hk, d, bs, dtype)
        x["v"] = (x["v"].float() * 2.0 ** by).to(dtype)
        x["v_scale"] = torch.exp2(torch.empty(x["v_scale"].shape).uniform_(low, high, generator=g))
        x["v_cache"] = x["v_cache"].clamp(-60, 60)   # (results within fp16's range)
        check(x, bs, mt.chunk_attention(**put(x)))


def agree(x, bs, got):
    """As check(), where the results are finite; infinities and NaN in the same places."""
    out, lse, size = want_of(x, bs)
    got_out, got_lse = (t.cpu().double() for t in got)
    u, d = torch.finfo(x["q"].dtype).eps / 2, x["q"].shape[2]
    big = max(float(t[torch.isfinite(t)].abs().max()) for t in (x["v"], x["v_cache"] * x["v_scale"][..., None, None]) if torch.isfinite(t).any())
    e = 2 ** -24 * (d + 64) * size + 2 ** -22 * size
    assert torch.equal(torch.isnan(got_out), torch.isnan(out))
    for inf in (math.inf, -math.inf):
        assert torch.equal(got_out == inf, out == inf)
    fine = torch.isfinite(out)
    assert not fine.all() and fine.any()
    assert ((got_out - out).abs() <= (2.25 * u + 2 * e[..., None]) * big)[fine].all()
    assert ((got_lse - lse).abs() <= e + 2 ** -23 * lse.abs() + 1e-7).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,hk,d,bs", [(4, 1, 64, 16), (6, 2, 64, 64), (3, 1, 128, 32), (8, 2, 128, 128)])
@pytest.mark.parametrize("score", [0.0, -21.0, -300.0])     # weights that both types have, that fp16 has not, that 32 bits have not
def test_infinities_and_nan_of_any_weight(score, heads, hk, d, bs, dtype):
    for new, context, max_length in ((300, 70, None), (300, 0, 1), (620, 0, None)):
        x = build(new, [new + context, 66], [new, 66], heads, hk, d, bs, dtype)
        x["q"][:, :, 0], x["k"][:, :, 0] = 8.0, 0.0
        x["v"][[10, 150, 290, 20, 40], :, [3, 3, 9, 12, 50]] = torch.tensor([math.inf, -math.inf, math.inf, math.nan, -math.inf]).to(dtype)[:, None]
        x["k"][[10, 150, 290, 20, 40], :, 0] = score * math.sqrt(d) / 8
        x["k_cache"][:, :, :, 0] = 0.0
        agree(x, bs, mt.chunk_attention(**put(x), max_length=max_length))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,bs", [(64, 32), (128, 64)])
def test_infinities_in_a_part_of_no_weight(d, bs, dtype):
    # all new tokens far below the context, whose parts have all of the weight
    x = build(4, [6000 + 140], [140], 2, 1, d, bs, dtype)
    x["q"][:, :, 0], x["k"][:, :, 0] = 8.0, -300 * math.sqrt(d) / 8
    x["k_cache"][:, :, :, 0] = 0.0
    x["v"][[5, 100, 120], 0, [3, 4, 3]] = torch.tensor([math.inf, math.nan, -math.inf]).to(dtype)
    agree(x, bs, mt.chunk_attention(**put(x)))


def test_infinities_and_nan_in_long_prompts():
    # rows of many tiles that all of them see
    x = build(6, [1500], [1500], 2, 1, 64, 64, torch.float16)
    x["v"][[0, 700, 1400], 0, [3, 60, 33]] = torch.tensor([math.inf, math.nan, -math.inf]).to(torch.float16)
    agree(x, 64, mt.chunk_attention(**put(x)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,bs", [(64, 32), (128, 64)])
def test_infinities_beside_a_nan_of_the_cache(d, bs, dtype):
    # the cache's NaN stays, also in a column whose new values hold an infinity of no weight
    x = build(9, [400 + 300, 70], [300, 70], 2, 1, d, bs, dtype)
    x["q"][:, :, 0], x["k"][:, :, 0] = 8.0, 0.0
    x["k"][10, 0, 0] = -300 * math.sqrt(d) / 8
    x["k_cache"][:, :, :, 0] = 0.0
    x["v"][10, 0, 3:5] = math.inf
    x["v_cache"][int(x["block_table"][0, 2]), 0, 5, 3] = math.nan
    agree(x, bs, mt.chunk_attention(**put(x), max_length=1))
    got = mt.chunk_attention(**put(x))[0]
    agree(x, bs, (got, mt.chunk_attention(**put(x))[1]))
    assert torch.isnan(got[:300, :, 3]).all() and (got[10:300, :, 4] == math.inf).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,hk,d,bs", [(3, 1, 64, 32), (4, 2, 128, 64)])
def test_many_infinities_and_nan(heads, hk, d, bs, dtype):
    # in all kinds of tiles at once; a column that is NaN from the first token on, columns without any
    x = build(13, [640 + 90, 130], [640, 130], heads, hk, d, bs, dtype, extra=3)
    g = torch.Generator().manual_seed(2)
    pick = torch.rand(x["v"].shape, generator=g) < 0.003
    pick[..., d // 2:] = False
    values = torch.tensor([math.inf, -math.inf, math.nan]).to(dtype)
    x["v"][pick] = values[torch.randint(0, 3, (int(pick.sum()),), generator=g)]
    x["v"][..., d - 3] = math.nan
    x["v"][:, 0, d - 9] = math.inf
    want = want_of(x, bs)
    out, lse = (t.cpu().double() for t in mt.chunk_attention(**put(x), max_length=1))
    assert (out[-3:] == 0).all() and torch.isneginf(lse[-3:]).all()
    agree({n: t[:-3] if n in ("q", "k", "v") else t for n, t in x.items()}, bs, (out[:-3], lse[:-3]))
    assert torch.equal(torch.isnan(out), torch.isnan(want[0]))
