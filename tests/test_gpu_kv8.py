"""GPU: the 8-bit paged cache and the attention that reads it, against plain
64-bit forms.

kv8_append is exact: scales are powers of two, a quotient by one is exact, and
the rounding to nearest even is the definition, so codes and scales are equal.
Means: a sum of up to 128 codes times a power of two, a division:
140 * 2^-24 * max.

kv8_attention's out: the weights are rounded to the type of q (u relative, half
a step) before the product with the exact codes and the result once more:
2.25 u max|v|, as for the other attention; fp16 weights below 2^-14 of the
largest one are off by 2^-25 of it, n * 2^-25 max|v| over n keys, within the
quarter for n up to 4096.  lse: 32-bit: 2^-24 (d + 64) (max|s| + 10).
"""

import math

import pytest
import torch

import attention_oracle as oracle
import row_wise_top_topk_amd as mt

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F8 = torch.float8_e4m3fn


def build(seed, lens, hk, d, bs, spare=3, codes=True):
    """A cache on the CPU whose pages hold the sequences, NaN codes elsewhere."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // bs) for n in lens]
    pages, wide = sum(need) + spare, max(1, max(need))
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), wide), -7, dtype=torch.int32)
    kc, vc = (torch.full((pages, hk, bs, d), math.nan) for _ in range(2))
    ks, vs = (torch.exp2(torch.randint(-9, -4, (pages, hk), generator=g).float()) for _ in range(2))
    at = 0
    for i, n in enumerate(lens):
        table[i, :need[i]] = order[at:at + need[i]]
        for j in range(need[i]):
            e = min(bs, n - j * bs)
            for c in (kc, vc):
                c[order[at + j], :, :e] = oracle.round8(60 * torch.randn(hk, e, d, generator=g))
        at += need[i]
    return kc, vc, ks, vs, table


def put(kc, vc, ks, vs, table):
    return [x.to(DEV).to(F8) for x in (kc, vc)] + [x.to(DEV) for x in (ks, vs, table)]


def same(got, want):
    got = got.float().cpu()
    return torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,new,hk,d,bs", [
    ([1], None, 1, 128, 16),
    ([5, 64, 65, 128, 17], None, 3, 64, 64),
    ([200, 31], [200, 31], 2, 128, 32),
    ([300, 0, 40, 129], [150, 0, 1, 129], 2, 64, 128),
    ([77], [30], 1, 128, 16),
])
def test_append(dtype, lens, new, hk, d, bs):
    n = [1] * len(lens) if new is None else new
    before = [a - b for a, b in zip(lens, n)]
    kc, vc, ks, vs, table = build(3, lens, hk, d, bs)
    for i, (b, x) in enumerate(zip(before, lens)):     # what is not yet stored is rubbish
        for pos in range(b, x):
            for c in (kc, vc):
                c[table[i, pos // bs], :, pos % bs] = math.nan
    g = torch.Generator().manual_seed(5)
    t = sum(n) + (0 if new is None else 2)              # rows behind the last sequence
    size = torch.exp2(torch.randint(-12, 5, (t, hk, 1), generator=g).float())
    k, v = ((size * torch.randn(t, hk, d, generator=g)).to(dtype) for _ in range(2))
    if t > 1:
        k[0, 0, 1], v[-1 if new is None else 0, 0, 2] = math.inf, -math.inf
        k[0, 0, 3] = math.nan
        v[1 if new is None else 0] = 0
    cu = None if new is None else torch.tensor([0] + n).cumsum(0).to(torch.int32)
    dev = put(kc, vc, ks, vs, table)
    mean = torch.full((kc.shape[0], hk, d), 7.0)
    mean_dev = mean.to(DEV)
    mt.kv8_append(k.to(DEV), v.to(DEV), *dev[:4], dev[4], torch.tensor(lens, dtype=torch.int32, device=DEV),
                  cu_seqlens=None if cu is None else cu.to(DEV), k_mean=mean_dev)
    oracle.append(k, v, kc, vc, ks, vs, table, lens, bs, cu, mean)
    assert torch.equal(dev[2].cpu(), ks) and torch.equal(dev[3].cpu(), vs)
    assert same(dev[0], kc) and same(dev[1], vc)
    fin = torch.isfinite(mean)
    got = mean_dev.cpu()
    assert torch.equal(torch.isfinite(got), fin)
    top = mean[fin].abs().max().item()
    peak = max(top, (448 * ks).max().item())
    assert (got - mean)[fin].abs().max().item() <= 140 * 2.0 ** -24 * peak


def test_append_one_by_one_grows_scales():
    """Token after token, sizes rising: earlier codes are rounded again under each larger scale."""
    g = torch.Generator().manual_seed(8)
    kc, vc, ks, vs, table = build(1, [40], 2, 64, 16)
    dev = put(kc, vc, ks, vs, table)
    for pos in range(40):
        k, v = ((2.0 ** (pos / 3 - 4) * torch.randn(1, 2, 64, generator=g)).to(torch.bfloat16) for _ in range(2))
        mt.kv8_append(k.to(DEV), v.to(DEV), *dev, torch.tensor([pos + 1], dtype=torch.int32, device=DEV))
        oracle.append(k, v, kc, vc, ks, vs, table, [pos + 1], 16)
    assert torch.equal(dev[2].cpu(), ks) and same(dev[0], kc) and same(dev[1], vc)


def test_append_skips_pages_that_are_not_there():
    kc, vc, ks, vs, table = build(2, [64, 64], 1, 64, 16)
    table[0, 1], table[1, 2] = -1, kc.shape[0]
    dev = put(kc, vc, ks, vs, table)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(128, 1, 64, generator=g).to(torch.float16) for _ in range(2))
    cu = torch.tensor([0, 64, 128], dtype=torch.int32)
    mt.kv8_append(k.to(DEV), v.to(DEV), *dev, torch.tensor([64, 80], dtype=torch.int32, device=DEV), cu_seqlens=cu.to(DEV))
    oracle.append(k, v, kc, vc, ks, vs, table, [64, 80], 16, cu)
    assert torch.equal(dev[2].cpu(), ks) and same(dev[0], kc) and same(dev[1], vc)


CASES = [
    # lens, new, heads, kv_heads, dim, block, dtype
    ([1], None, 1, 1, 128, 16, torch.bfloat16),
    ([33, 0, 700, 64], None, 8, 1, 128, 64, torch.bfloat16),
    ([1000, 17, 129], None, 10, 2, 64, 16, torch.float16),
    ([700, 1, 250], [3, 1, 2], 12, 3, 64, 32, torch.bfloat16),
    ([900], [5], 16, 1, 128, 128, torch.float16),               # 80 rows: two tiles of 64
    ([300, 40], [70, 40], 4, 2, 128, 16, torch.bfloat16),       # a prompt behind a cache
    ([500, 130], None, 40, 1, 128, 32, torch.bfloat16),         # more heads than a tile of 32
    ([260], None, 128, 1, 64, 64, torch.float16),               # more than a tile of 64
    ([3000], None, 2, 2, 64, 16, torch.bfloat16),               # several chunks
    ([20, 2], [3, 5], 4, 1, 128, 16, torch.float16),            # more new tokens than length: empty rows
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("select", [0, 1, 5])
def test_attention(case, select):
    lens, new, h, hk, d, bs, dtype = case
    g = torch.Generator().manual_seed(4)
    kc, vc, ks, vs, table = build(6, lens, hk, d, bs)
    n = [1] * len(lens) if new is None else new
    tail = 0 if new is None else 2
    t = sum(n) + tail
    q = (2 * torch.randn(t, h, d, generator=g)).to(dtype)
    cu = None if new is None else torch.tensor([0] + n).cumsum(0).to(torch.int32)
    blocks = None
    if select:
        blocks = torch.randint(-1, table.shape[1] + 1, (t, hk, select), generator=g).to(torch.int32)
        blocks[0, 0] = torch.arange(select).to(torch.int32)
    want, want_lse = oracle.cache_attention(q, kc, vc, ks, vs, table, lens, bs, cu, blocks)
    dev = put(kc, vc, ks, vs, table)
    for bound in (None, 1):                                      # a bound that is too small changes the split only
        out, lse = mt.kv8_attention(q.to(DEV), *dev, torch.tensor(lens, dtype=torch.int32, device=DEV),
                                    cu_seqlens=None if cu is None else cu.to(DEV),
                                    blocks=None if blocks is None else blocks.to(DEV), max_length=bound)
        check(out, lse, want, want_lse, q, kc, vc, ks, vs, d, dtype)
        if tail:
            assert (out[-tail:] == 0).all() and (lse[-tail:] == -math.inf).all()


def check(out, lse, want, want_lse, q, kc, vc, ks, vs, d, dtype):
    u = torch.finfo(dtype).eps / 2
    top = (vc.nan_to_num() * vs[:, :, None, None]).abs().max().item()
    assert torch.isfinite(out).all()
    err = (out.cpu().double() - want).abs().max().item()
    assert err <= 2.25 * u * top, (err, 2.25 * u * top)
    fin = torch.isfinite(want_lse)
    assert (lse.cpu()[~fin] == -math.inf).all()
    smax = (q.double().norm(dim=2).max() * (kc.nan_to_num() * ks[:, :, None, None]).double().norm(dim=3).max() / math.sqrt(d)).item()
    if fin.any():
        off = (lse.cpu().double() - want_lse)[fin].abs().max().item()
        assert off <= 2.0 ** -24 * (d + 64) * (smax + 10), off


def test_attention_without_some_pages_and_with_any_scales():
    kc, vc, ks, vs, table = build(9, [400, 300], 2, 128, 32)
    g = torch.Generator().manual_seed(2)
    ks = 0.003 + 0.02 * torch.rand(ks.shape, generator=g)
    vs = torch.exp(6 * torch.randn(vs.shape, generator=g) - 6)   # from page to page by factors of thousands
    table[0, 3], table[0, 12], table[1, 0] = -1, kc.shape[0], 1 << 30
    q = torch.randn(2, 8, 128, generator=g).to(torch.bfloat16)
    want, want_lse = oracle.cache_attention(q, kc, vc, ks, vs, table, [400, 300], 32)
    dev = put(kc, vc, ks, vs, table)
    out, lse = mt.kv8_attention(q.to(DEV), *dev, torch.tensor([400, 300], dtype=torch.int32, device=DEV))
    check(out, lse, want, want_lse, q, kc, vc, ks, vs, 128, torch.bfloat16)
    table[:] = -1
    out, lse = mt.kv8_attention(q.to(DEV), *put(kc, vc, ks, vs, table), torch.tensor([400, 300], dtype=torch.int32, device=DEV))
    assert (out == 0).all() and (lse == -math.inf).all()


def test_repeated_and_unordered_blocks():
    kc, vc, ks, vs, table = build(3, [1500], 2, 64, 16)
    g = torch.Generator().manual_seed(3)
    q = torch.randn(1, 8, 64, generator=g).to(torch.float16).to(DEV)
    dev = put(kc, vc, ks, vs, table)
    lens = torch.tensor([1500], dtype=torch.int32, device=DEV)
    row = torch.randperm(94, generator=g)[:40].to(torch.int32)
    plain = torch.stack([row.sort()[0], row.sort()[0]])[None].to(DEV)
    wild = torch.cat([row, row[:30], torch.tensor([-5, 94, 1 << 30])]).to(torch.int32)
    wild = torch.stack([wild, wild.flip(0)])[None].contiguous().to(DEV)
    a, la = mt.kv8_attention(q, *dev, lens, blocks=plain)
    b, lb = mt.kv8_attention(q, *dev, lens, blocks=wild)
    # the same keys in another order: two roundings of the same sums
    assert (la - lb).abs().max().item() <= 2.0 ** -24 * 128 * 50
    top = (vc.nan_to_num() * vs[:, :, None, None]).abs().max().item()
    assert (a.double() - b.double()).abs().max().item() <= 2 * 2.25 * 2.0 ** -11 * top


def test_serving_run():
    """Prompt into the cache, then steps: append, score the cached means, select, attend."""
    g = torch.Generator().manual_seed(12)
    hk, h, d, bs = 2, 8, 128, 16
    lens = [200, 77]
    kc, vc, ks, vs, table = build(4, [210, 90], hk, d, bs)
    dev = put(kc, vc, ks, vs, table)
    mean = torch.zeros(kc.shape[0], hk, d, device=DEV)
    mean_cpu = torch.zeros(kc.shape[0], hk, d, dtype=torch.float64)
    k, v = (torch.randn(sum(lens), hk, d, generator=g).to(torch.bfloat16) for _ in range(2))
    cu = torch.tensor([0, 200, 277], dtype=torch.int32)
    mt.kv8_append(k.to(DEV), v.to(DEV), *dev, torch.tensor(lens, dtype=torch.int32, device=DEV), cu_seqlens=cu.to(DEV), k_mean=mean)
    oracle.append(k, v, kc, vc, ks, vs, table, lens, bs, cu, mean_cpu)
    for _ in range(5):
        lens = [n + 1 for n in lens]
        lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
        q = (2 * torch.randn(2, h, d, generator=g)).to(torch.bfloat16)
        k, v = (torch.randn(2, hk, d, generator=g).to(torch.bfloat16) for _ in range(2))
        mt.kv8_append(k.to(DEV), v.to(DEV), *dev, lengths, k_mean=mean)
        scores, counts = mt.block_scores(q.to(DEV), mean, bs, table.shape[1], lengths=lengths, block_table=dev[4])
        blocks = mt.topk_indices(scores.flatten(0, 1), counts.flatten(), 4).view(2, hk, 4)
        out, lse = mt.kv8_attention(q.to(DEV), *dev, lengths, blocks=blocks)
        oracle.append(k, v, kc, vc, ks, vs, table, lens, bs, None, mean_cpu)
        picked = blocks.cpu()
        for i, n in enumerate(lens):
            assert (picked[i] >= 0).all() and (picked[i, :, 0] == 0).all() and (picked[i, :, -1] == (n - 1) // bs).all()
        want, want_lse = oracle.cache_attention(q, kc, vc, ks, vs, table, lens, bs, None, picked)
        check(out, lse, want, want_lse, q, kc, vc, ks, vs, d, torch.bfloat16)
