"""GPU: attention of a chunk behind the 8-bit cache, against a plain 64-bit form.

out: a weight is rounded once to the type of q (u relative, half a step) before
the product with exact codes and 16-bit values, and the result once more: 2 u
max|v|.  A score is a 32-bit sum of d products, off by at most 2^-24 (d + 64) of
the sum of its absolute terms, and by 2^-22 of itself through the exponent's
arguments: e in all; a weight and the sum of the weights are off by e each, which
adds 2 e max|v|, and the 32-bit sums over n keys by n 2^-24 max|v| (2^-24 sqrt n in
practice; a quarter of u covers n up to 4096 for bf16, 1024 for fp16 taken twice).
lse: e, and 2^-23 of itself.
"""

import math

import pytest
import torch

import row_wise_top_topk_amd as mt
import serving_oracle as oracle

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F8 = torch.float8_e4m3fn
BOTH = [torch.bfloat16, torch.float16]


def round8(x):
    return x.clamp(-448, 448).float().to(F8).float()


def build(seed, lens, new, heads, hk, d, bs, dtype, extra=0, cols=None):
    """Inputs on the CPU: pages hold the sequences' context, NaN codes elsewhere."""
    g = torch.Generator().manual_seed(seed)
    held = [max(0, a - b) for a, b in zip(lens, new)]
    need = [-(-n // bs) for n in held]
    pages, wide = sum(need) + 3, max([1] + need) if cols is None else cols
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), wide), -7, dtype=torch.int32)
    kc, vc = (torch.full((pages, hk, bs, d), math.nan) for _ in range(2))
    ks, vs = (torch.exp2(torch.randint(-9, -4, (pages, hk), generator=g).float()) for _ in range(2))
    at = 0
    for i, n in enumerate(held):
        c = min(need[i], wide)
        table[i, :c] = order[at:at + c]
        for j in range(need[i]):
            e = min(bs, n - j * bs)
            for x in (kc, vc):
                x[order[at + j], :, :e] = round8(60 * torch.randn(hk, e, d, generator=g))
        at += need[i]
    t = sum(new) + extra
    q = (1.5 * torch.randn(t, heads, d, generator=g)).to(dtype)
    k, v = (torch.randn(t, hk, d, generator=g).to(dtype) for _ in range(2))
    cu = torch.tensor([0] + [sum(new[:i + 1]) for i in range(len(new))], dtype=torch.int32)
    return dict(q=q, k=k, v=v, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, block_table=table,
                lengths=torch.tensor(lens, dtype=torch.int32), cu_seqlens=cu)


def put(x):
    return {n: (t.to(DEV).to(F8) if n in ("k_cache", "v_cache") else t.to(DEV)) for n, t in x.items() if t is not None}


def want_of(x, bs, scale=None):
    return oracle.chunk_attention(x["q"], x["k"], x["v"], x["k_cache"], x["v_cache"], x["k_scale"], x["v_scale"], x["block_table"],
                                  x["lengths"], bs, x.get("cu_seqlens"), scale)


def check(x, bs, got, scale=None, want=None):
    out, lse, size = want_of(x, bs, scale) if want is None else want
    got_out, got_lse = (t.cpu().double() for t in got)
    u = torch.finfo(x["q"].dtype).eps / 2
    d = x["q"].shape[2]
    finite = [t.double()[torch.isfinite(t.double())].abs() for t in (x["v"], x["v_cache"] * x["v_scale"][..., None, None])]
    big = max([float(t.max()) for t in finite if t.numel()] + [0.0])
    e = 2 ** -24 * (d + 64) * size + 2 ** -22 * size
    assert torch.equal(torch.isneginf(got_lse), torch.isneginf(lse))
    seen = ~torch.isneginf(lse)
    assert torch.all((got_lse - lse)[seen].abs() <= (e + 2 ** -23 * lse.abs() + 1e-7)[seen])
    assert torch.all(got_out[~seen] == 0)
    off = (got_out - out).abs()
    assert torch.all(off <= (2.25 * u + 2 * e[..., None]) * big), (off.max().item(), u * big)


CASES = [  # lengths, new tokens, heads, key heads, dim, block
    ([1], [1], 1, 1, 64, 16),
    ([130], [3], 4, 2, 128, 16),
    ([64], [64], 2, 1, 64, 64),
    ([65, 0, 300, 17], [65, 0, 33, 1], 6, 3, 64, 32),
    ([200], [129], 8, 1, 128, 64),
    ([517, 90], [7, 90], 10, 2, 128, 128),
    ([700], [150], 5, 1, 64, 16),
    ([40, 41, 42, 43, 500], [1, 1, 2, 1, 5], 16, 1, 128, 16),
    ([1100], [20], 128, 1, 64, 64),
    ([333, 260], [66, 200], 3, 3, 128, 32),
]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("lens,new,heads,hk,d,bs", CASES, ids=str)
def test_chunks(dtype, lens, new, heads, hk, d, bs):
    x = build(sum(lens), lens, new, heads, hk, d, bs, dtype, extra=2)
    check(x, bs, mt.chunk_attention(**put(x)))


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("d,bs,heads,hk", [(64, 16, 3, 1), (128, 32, 7, 1), (128, 64, 2, 2), (64, 128, 64, 1), (128, 128, 12, 2), (128, 16, 1, 1)])
def test_lengths_around_tiles(dtype, d, bs, heads, hk):
    lens = [1, 15, 63, 64, 65, 127, 128, 129, 191, 257]
    for ahead in (0, 1, 63, 64, 65, 128):
        new = [min(n, 66) for n in lens]
        x = build(ahead, [n + ahead for n in new], new, heads, hk, d, bs, dtype)
        check(x, bs, mt.chunk_attention(**put(x)))


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("d,bs,heads,hk", [(64, 16, 8, 2), (64, 128, 6, 6), (128, 32, 3, 1), (128, 64, 16, 2)])
def test_one_sequence_in_a_wide_table(dtype, d, bs, heads, hk):
    # room for 200000 keys: workgroups of 256 rows, in parts most of which are empty
    for n, m in ((70, 70), (1, 900), (129, 1500), (300, 301)):
        x = build(n, [m], [n], heads, hk, d, bs, dtype, extra=1, cols=200000 // bs)
        check(x, bs, mt.chunk_attention(**put(x)))
    x = build(5, [4300], [400], heads, hk, d, bs, dtype, cols=60000 // bs)
    check(x, bs, mt.chunk_attention(**put(x)))


@pytest.mark.parametrize("max_length", [None, 1, 100, 5000])
@pytest.mark.parametrize("bs,d", [(16, 64), (128, 128), (64, 128)])
def test_split_walks(max_length, bs, d):
    # few rows, many keys: the walk is split; bounds that are too small are no mistake
    x = build(7, [5001, 2000, 4], [3, 2, 4], 4, 2, d, bs, torch.bfloat16)
    check(x, bs, mt.chunk_attention(**put(x), max_length=max_length))


def test_segments_of_pages():
    # more blocks than are looked up at a time (256), also from inside a block
    for bs, n in ((16, 9000), (32, 17000), (64, 17000)):
        x = build(bs, [n + 5], [5], 2, 1, 64, bs, torch.bfloat16)
        got = mt.chunk_attention(**put(x))
        check(x, bs, got)


def test_one_token_each_without_cu():
    x = build(3, [5, 1, 700, 64], [1, 1, 1, 1], 6, 2, 64, 16, torch.float16)
    del x["cu_seqlens"]
    check(x, 16, mt.chunk_attention(**put(x)))


def test_scale_strides_and_out():
    x = build(9, [90, 41], [33, 41], 4, 2, 64, 16, torch.bfloat16)
    dev = put(x)
    for n in ("q", "k", "v"):      # heads first in memory, 24 columns between rows
        t = dev[n]
        wide = torch.zeros(t.shape[1], t.shape[0], t.shape[2] + 24, dtype=t.dtype, device=DEV)
        wide[:, :, :t.shape[2]] = t.transpose(0, 1)
        dev[n] = wide[:, :, :t.shape[2]].transpose(0, 1)
    table = torch.full((2, 11), 99, dtype=torch.int32, device=DEV)
    table[:, :dev["block_table"].shape[1]] = dev["block_table"]
    dev["block_table"] = table[:, :dev["block_table"].shape[1]]
    out = torch.empty_like(x["q"], device=DEV)
    got = mt.chunk_attention(**dev, scale=0.3, out=out)
    assert got[0] is out
    check(x, 16, got, scale=0.3)


def test_more_new_tokens_than_a_length():
    # the first of them would stand before the sequence's start: hidden, and seeing nothing
    x = build(2, [40, 3, -5, 0], [100, 70, 4, 3], 4, 2, 64, 16, torch.bfloat16)
    x["k"][:60] = math.nan
    x["v"][:60] = math.inf
    x["v"][100:167] = math.nan
    x["v"][170:] = math.inf
    want = want_of(x, 16)
    got = mt.chunk_attention(**put(x))
    assert torch.isneginf(got[1][:60]).all() and torch.isneginf(got[1][170:]).all()
    check(x, 16, got, want=want)


def test_pages_and_columns_that_are_not_there():
    x = build(4, [300, 200], [10, 50], 4, 2, 128, 16, torch.bfloat16)
    x["block_table"][0, 0], x["block_table"][0, 5], x["block_table"][1, 9] = -1, 1 << 30, x["k_cache"].shape[0]
    check(x, 16, mt.chunk_attention(**put(x)))
    x = build(4, [300, 200], [10, 50], 4, 2, 128, 16, torch.float16, cols=6)   # a narrow table
    check(x, 16, mt.chunk_attention(**put(x)))
    x["block_table"][:] = -1
    check(x, 16, mt.chunk_attention(**put(x)))
    x["block_table"] = torch.zeros(2, 0, dtype=torch.int32)
    check(x, 16, mt.chunk_attention(**put(x)))
    x |= {n: x[n][:0] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    check(x, 16, mt.chunk_attention(**put(x)))


@pytest.mark.parametrize("dtype", BOTH)
def test_scales_that_are_no_powers_of_two(dtype):
    x = build(6, [270], [70], 4, 1, 64, 16, dtype)
    g = torch.Generator().manual_seed(1)
    for n in ("k_scale", "v_scale"):
        x[n] = 0.01 + 0.03 * torch.rand(x[n].shape, generator=g)
    check(x, 16, mt.chunk_attention(**put(x)))


@pytest.mark.parametrize("bs", [16, 64])
def test_hidden_infinities_and_nan(bs):
    # each in a place that some rows see and others do not: those get them, these do not
    x = build(8, [130 + 90], [90], 2, 1, 64, bs, torch.bfloat16)
    plain = want_of(x, bs)
    x["v"][40, 0, 3], x["v"][41, 0, 3], x["v"][50, 0, 9], x["v"][80, 0, 5] = math.inf, -math.inf, math.nan, -math.inf
    x["k"][85, 0, 0] = math.nan
    want = want_of(x, bs)
    out, lse = (t.cpu().double() for t in mt.chunk_attention(**put(x)))
    assert torch.equal(torch.isnan(out), torch.isnan(want[0]))
    for inf in (math.inf, -math.inf):
        assert torch.equal(out == inf, want[0] == inf)
    fine = torch.isfinite(want[0])
    u, big = 2 ** -8, 5.0
    assert ((out - plain[0])[fine].abs() <= 2.5 * u * big).all()
    assert torch.equal(torch.isnan(lse), torch.isnan(want[1])) and torch.isnan(lse[85:]).all() and not torch.isnan(lse[:85]).any()


def test_nan_of_the_cache_reaches_its_rows_only():
    x = build(8, [150, 160], [20, 30], 2, 1, 64, 16, torch.bfloat16)
    page = int(x["block_table"][0, 2])
    x["v_cache"][page, 0, 3, 7] = math.nan
    out, lse = mt.chunk_attention(**put(x))
    assert torch.isnan(out[:20, :, 7]).all() and not torch.isnan(out[:20, :, :7]).any() and not torch.isnan(out[20:]).any()
    x["k_cache"][page, 0, 3, 7] = math.nan
    out, lse = mt.chunk_attention(**put(x))
    assert torch.isnan(out[:20]).all() and torch.isnan(lse[:20]).all() and not torch.isnan(out[20:]).any()


def test_fp16_keeps_many_small_weights():
    # one key far ahead of the others: 2^-24 each, which fp16 has no bits for beside 1
    n, d = 60000, 64
    x = build(1, [n + 1], [1], 1, 1, d, 128, torch.float16)
    x["k_cache"].zero_()
    x["k"].zero_()
    x["q"].zero_()
    x["q"][0, 0, 0], x["k"][0, 0, 0] = 16.0, 24 * math.log(2) / 16 * 8
    x["v"].zero_()
    x["v_cache"][:], x["v_scale"][:] = 256.0, 256.0
    got = mt.chunk_attention(**put(x))[0].cpu().double()
    p = math.exp(-float(x["q"][0, 0, 0]) * float(x["k"][0, 0, 0]) / 8)
    want = 65536 * n * p / (1 + n * p)
    assert ((got - want).abs() <= 4 * 2 ** -11 * want).all()


def test_lowest_finite_and_infinite_scores():
    # scores of the type's lowest value and of -inf beside others: no weight, no NaN
    x = build(8, [80], [20], 1, 1, 64, 16, torch.bfloat16)
    x["q"].fill_(1.0)
    x["k"][3], x["k"][5] = torch.finfo(torch.bfloat16).min / 64, -math.inf
    got = mt.chunk_attention(**put(x))
    want = want_of(x, 16)
    size = want_of({**x, "k": x["k"].clone().index_fill_(0, torch.tensor([3, 5]), 0)}, 16)[2]
    check(x, 16, got, want=(want[0], want[1], size))


def test_shared_heads_of_every_number():
    for group in (1, 2, 3, 4, 5, 6, 7, 8, 9, 11, 12, 15, 16, 17, 31, 33, 64, 65, 127, 128):
        x = build(group, [150], [9], group, 1, 64, 16, torch.bfloat16)
        check(x, 16, mt.chunk_attention(**put(x)))


def test_nothing_to_do():
    x = put(build(3, [0, 0], [0, 0], 2, 1, 64, 16, torch.bfloat16))
    out, lse = mt.chunk_attention(**x)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    x = put(build(3, [], [], 2, 1, 64, 16, torch.bfloat16, extra=5) | {"block_table": torch.zeros(0, 1, dtype=torch.int32)})
    out, lse = mt.chunk_attention(**x)   # rows without a sequence
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_same_result_from_run_to_run():
    x = put(build(5, [3000, 2000], [200, 3], 8, 2, 128, 64, torch.bfloat16))
    a, b = mt.chunk_attention(**x), mt.chunk_attention(**x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_as_the_cache_attention_where_the_chunk_is_in_the_cache():
    # a chunk whose own rows are exact in 8 bits gives what kv8_attention gives of the whole cache
    lens, new, bs, hk, d = [150, 70], [20, 70], 16, 2, 64
    x = build(12, lens, new, 4, hk, d, bs, torch.bfloat16)
    x["k"], x["v"] = (round8(16 * x[n].float()).to(torch.bfloat16) for n in ("k", "v"))
    x["q"] = (x["q"] / 16).to(torch.bfloat16)
    dev = put(x)
    refs = torch.zeros(40, dtype=torch.int32, device=DEV)
    pages = 40
    cache = [torch.zeros(pages, hk, bs, d, device=DEV).to(F8) for _ in range(2)] + [torch.ones(pages, hk, device=DEV) for _ in range(2)]
    table, lengths = torch.full((2, 12), -1, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    before = torch.tensor([a - b for a, b in zip(lens, new)], dtype=torch.int32, device=DEV)
    mt.pages_grow(table, lengths, refs, before, bs)
    for i in range(2):
        for j in range(-(-int(before[i]) // bs)):
            at, was = int(table[i, j]), int(x["block_table"][i, j])
            for to, name in zip(cache, ("k_cache", "v_cache", "k_scale", "v_scale")):
                to[at] = dev[name][was]
    mt.pages_grow(table, lengths, refs, torch.tensor(new, dtype=torch.int32, device=DEV), bs)
    chunk = mt.chunk_attention(dev["q"], dev["k"], dev["v"], *cache, table, lengths, cu_seqlens=dev["cu_seqlens"])
    mt.kv8_append(dev["k"], dev["v"], *cache, table, lengths, cu_seqlens=dev["cu_seqlens"])
    whole = mt.kv8_attention(dev["q"], *cache, table, lengths, cu_seqlens=dev["cu_seqlens"])
    want = want_of(x, bs)
    check(x, bs, chunk, want=want)
    assert (chunk[0].float() - whole[0].float()).abs().max() <= 5 * 2 ** -8 * float(x["v"].abs().max())
