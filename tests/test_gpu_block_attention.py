"""GPU: block means, block scores and block sparse attention against plain
64-bit forms.

Tolerances.  u is half a step of the type, relative (bf16 2^-8, fp16 2^-11;
``torch.finfo(t).eps / 2``).  Inputs are exact in both.
* out: the probabilities are rounded to the type before the product with v
  (each by u of itself, so the sum moves by at most u * sum p |v| <= u max|v|)
  and the result once more (u |out| <= u max|v|); the scores and the sums are
  held in 32 bits, whose share is below u max|v| / 8 for bf16 and fp16 at these
  lengths (scores up to 40: an error of 40 * 2^-22 in the exponent).  Allowed:
  2.25 u max|v| over the visible keys, taken over the whole tensor.
* lse: 32-bit scores, sums and logarithm: 2^-24 * (d + 64) * (max|s| + 10).
* means: a sum of up to 128 values in 32 bits: 130 * 2^-24 * max|k|.
* scores: 24-bit terms (two of 2^-23 for fp16) and 32-bit sums of up to 3 d
  products: (3 d + 8) * 2^-23 * sum |q||mean| * scale.
"""

import math

import pytest
import torch

import attention_oracle as oracle
import row_wise_top_topk_amd as mt

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def make(seed, lens_q, lens_k, h, hk, d, bs, select, dtype, tail=0, spread=1.0):
    """Random packed inputs on the CPU with ``tail`` rows behind the last sequence."""
    g = torch.Generator().manual_seed(seed)
    t, tk = sum(lens_q) + tail, sum(lens_k) + tail
    q = (spread * torch.randn(t, h, d, generator=g)).to(dtype)
    k = torch.randn(tk, hk, d, generator=g).to(dtype)
    v = torch.randn(tk, hk, d, generator=g).to(dtype)
    cu_q = torch.tensor([0] + lens_q).cumsum(0).to(torch.int32)
    cu_k = torch.tensor([0] + lens_k).cumsum(0).to(torch.int32)
    blocks = torch.full((t, hk, select), -1, dtype=torch.int32)
    for n, m, a in zip(lens_q, lens_k, cu_q.tolist()):
        nb = max(1, -(-m // bs))
        for r in range(n):
            for c in range(hk):
                last = max(0, (m - n + r) // bs)
                pick = torch.randperm(nb, generator=g)[:max(0, select - 1)].tolist()
                row = sorted(set(pick + [last]))[:select]
                blocks[a + r, c, :len(row)] = torch.tensor(row, dtype=torch.int32)
    return q, k, v, blocks, cu_q, cu_k


def check_out(got, want, lse, want_lse, v, smax, d, dtype):
    u = half_step(dtype)
    top = v.abs().double().max().item()
    assert torch.isfinite(got).all()
    err = (got.cpu().double() - want).abs().max().item()
    assert err <= 2.25 * u * top, f"out off by {err}, allowed {2.25 * u * top}"
    fin = torch.isfinite(want_lse)
    assert torch.equal(torch.isfinite(lse.cpu()), fin)
    assert (lse.cpu()[~fin] == -math.inf).all()
    if fin.any():
        off = (lse.cpu().double() - want_lse)[fin].abs().max().item()
        assert off <= 2.0 ** -24 * (d + 64) * (smax + 10), off


def gpu(*ts):
    return [t.to(DEV) for t in ts]


CASES = [
    # lens_q, lens_k, heads, kv_heads, dim, block, select, dtype, tail
    ([1], [1], 1, 1, 128, 64, 1, torch.bfloat16, 0),
    ([1], [77], 16, 1, 128, 16, 3, torch.bfloat16, 0),
    ([65], [65], 4, 2, 64, 32, 2, torch.float16, 0),
    ([130], [130], 8, 1, 128, 64, 2, torch.bfloat16, 0),
    ([257], [257], 2, 2, 64, 16, 5, torch.bfloat16, 0),         # one head a group: 128 tokens a tile
    ([200], [200], 10, 2, 128, 32, 4, torch.float16, 3),        # five heads a group, rows behind the end
    ([90, 0, 1, 33], [90, 0, 1, 33], 6, 3, 64, 128, 1, torch.bfloat16, 0),
    ([17, 40], [300, 41], 32, 1, 64, 64, 3, torch.float16, 5),  # fewer queries than keys
    ([50, 9], [20, 9], 4, 1, 128, 16, 2, torch.bfloat16, 0),    # more queries than keys: empty rows
    ([12], [12], 128, 1, 128, 16, 1, torch.bfloat16, 0),        # a whole tile for each token
    ([300], [300], 3, 3, 128, 128, 2, torch.float16, 0),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("causal", [True, False])
def test_forward(case, causal):
    lq, lk, h, hk, d, bs, select, dtype, tail = case
    q, k, v, blocks, cu_q, cu_k = make(7, lq, lk, h, hk, d, bs, select, dtype, tail)
    want, want_lse = oracle.attention(q, k, v, blocks, bs, cu_q, cu_k, causal=causal)
    out, lse = mt.block_attention(*gpu(q, k, v, blocks), bs, cu_seqlens=cu_q.to(DEV), cu_seqlens_k=cu_k.to(DEV), causal=causal)
    smax = (q.double().norm(dim=2).max() * k.double().norm(dim=2).max() / math.sqrt(d)).item() if k.numel() else 0
    check_out(out, want, lse, want_lse, v, smax, d, dtype)
    if tail:
        assert (out[-tail:] == 0).all() and (lse[-tail:] == -math.inf).all()
    if len(lq) == 1 and lq == lk and not tail:
        again, lse2 = mt.block_attention(*gpu(q, k, v, blocks), bs, causal=causal)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_many_blocks_and_windows():
    # one head a group and 16-key blocks: 600 blocks pass the window of 512 block numbers
    q, k, v, blocks, _, _ = make(3, [40], [9600], 2, 2, 64, 16, 40, torch.bfloat16)
    cu_q, cu_k = torch.tensor([0, 40], dtype=torch.int32), torch.tensor([0, 9600], dtype=torch.int32)
    want, want_lse = oracle.attention(q, k, v, blocks, 16, cu_q, cu_k)
    out, lse = mt.block_attention(*gpu(q, k, v, blocks), 16, cu_seqlens=cu_q.to(DEV), cu_seqlens_k=cu_k.to(DEV))
    check_out(out, want, lse, want_lse, v, 40, 64, torch.bfloat16)


def test_order_repeats_and_bad_numbers_of_blocks():
    q, k, v, blocks, _, _ = make(5, [150], [150], 4, 2, 64, 16, 6, torch.bfloat16)
    wild = blocks.clone()
    g = torch.Generator().manual_seed(1)
    for t in range(150):
        for c in range(2):
            wild[t, c] = wild[t, c][torch.randperm(6, generator=g)]
    wild = torch.cat([wild, wild[:, :, :2], torch.full((150, 2, 1), 10_000, dtype=torch.int32),
                      torch.full((150, 2, 1), -(1 << 31), dtype=torch.int32),
                      torch.full((150, 2, 1), (1 << 31) - 1, dtype=torch.int32)], 2)
    a, la = mt.block_attention(*gpu(q, k, v, blocks), 16)
    b, lb = mt.block_attention(*gpu(q, k, v, wild), 16)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_empty_rows():
    q, k, v, blocks, _, _ = make(6, [100], [100], 4, 1, 128, 32, 2, torch.float16)
    blocks[10:40] = -1
    blocks[60] = 3  # a block behind the query: nothing of it is visible
    want, want_lse = oracle.attention(q, k, v, blocks, 32)
    out, lse = mt.block_attention(*gpu(q, k, v, blocks), 32)
    check_out(out, want, lse, want_lse, v, 40, 128, torch.float16)
    assert (out[10:40] == 0).all() and (lse[60] == -math.inf).all()


def test_strided_operands():
    q, k, v, blocks, _, _ = make(8, [140], [140], 8, 2, 64, 32, 3, torch.bfloat16)
    want, wl = mt.block_attention(*gpu(q, k, v, blocks), 32)
    packed = torch.cat([x.flatten(1) for x in (q, k, v)], 1).to(DEV)        # one buffer, as a projection gives it
    qs, ks, vs = packed[:, :512].view(140, 8, 64), packed[:, 512:640].view(140, 2, 64), packed[:, 640:].view(140, 2, 64)
    out, lse = mt.block_attention(qs, ks, vs, blocks.to(DEV), 32)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    kt = k.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)             # heads first in memory
    out, lse = mt.block_attention(q.to(DEV), kt, v.to(DEV), blocks.to(DEV), 32)
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bs,d,lens", [(16, 64, [1]), (64, 128, [64, 0, 63, 130]), (128, 64, [300, 1]), (32, 128, [31, 33])])
def test_means(dtype, bs, d, lens):
    g = torch.Generator().manual_seed(4)
    k = torch.randn(sum(lens) + 2, 3, d, generator=g).to(dtype)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    got = mt.block_means(k.to(DEV), bs, cu_seqlens=cu.to(DEV)).cpu().double()
    want = oracle.means(k, bs, cu)
    assert got.shape == want.shape
    assert (got - want).abs().max().item() <= 130 * 2.0 ** -24 * k.abs().double().max().item()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens_q,lens_k,h,hk,d,bs,first,last", [
    ([1], [1], 1, 1, 128, 16, 1, 1),
    ([333], [333], 8, 2, 128, 16, 1, 1),
    ([40, 0, 77], [400, 0, 77], 10, 2, 64, 32, 0, 0),
    ([30, 20], [10, 20], 16, 1, 64, 16, 2, 3),
    ([70], [2000], 128, 1, 128, 16, 1, 2),
])
def test_scores_packed(dtype, lens_q, lens_k, h, hk, d, bs, first, last):
    g = torch.Generator().manual_seed(9)
    t, tk = sum(lens_q) + 2, sum(lens_k)
    q = torch.randn(t, h, d, generator=g).to(dtype)
    # blocks of very different sizes, down to where a 16-bit term has no bits left
    k = (torch.randn(tk, hk, d, generator=g) * torch.exp2(torch.randint(-9, 4, (tk, 1, 1), generator=g).float())).to(dtype)
    cu_q = torch.tensor([0] + lens_q).cumsum(0).to(torch.int32)
    cu_k = torch.tensor([0] + lens_k).cumsum(0).to(torch.int32)
    means = mt.block_means(k.to(DEV), bs, cu_seqlens=cu_k.to(DEV))
    nb = max(1, -(-max(lens_k) // bs))
    got, counts = mt.block_scores(q.to(DEV), means, bs, nb, cu_seqlens=cu_q.to(DEV), cu_seqlens_k=cu_k.to(DEV), first=first, last=last)
    m = means.cpu().double()
    placed = [(a + r, i, (e - c) - (b - a) + r) for i, (a, b, c, e) in enumerate(oracle.spans(t, tk, cu_q, cu_k)) for r in range(b - a)]
    want, want_counts = oracle.scores(q, lambda i, b: m[int(cu_k[i]) // bs + i + b], bs, nb, placed, hk, first, last)
    assert torch.equal(counts.cpu(), want_counts)
    size = q.double().norm(dim=2).max() * m.norm(dim=2).max() / math.sqrt(d)
    compare_scores(got, want, (3 * d + 8) * 2.0 ** -23 * size.item())


def compare_scores(got, want, allowed):
    got = got.cpu().double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin) and torch.equal(got[~fin], want[~fin])
    assert not fin.any() or (got - want)[fin].abs().max().item() <= allowed


@pytest.mark.parametrize("new", [None, [1, 3, 0, 2]])
@pytest.mark.parametrize("h,hk,d,bs,dtype", [(8, 1, 128, 64, torch.bfloat16), (12, 4, 64, 16, torch.float16), (40, 2, 128, 32, torch.bfloat16)])
def test_scores_paged(new, h, hk, d, bs, dtype):
    g = torch.Generator().manual_seed(2)
    lens = [1, 700, 0, 129] if new is None else [5, 700, 64, 2]
    nb = -(-max(lens) // bs)
    pages = 4 * nb
    means = torch.randn(pages, hk, d, generator=g)
    table = torch.randperm(pages, generator=g).view(4, nb).to(torch.int32)
    table[1, 2], table[1, 3] = -1, pages                # pages that are none
    n = [1] * 4 if new is None else new
    t = sum(n)
    q = torch.randn(t, h, d, generator=g).to(dtype)
    cu = torch.tensor([0] + n).cumsum(0).to(torch.int32)
    got, counts = mt.block_scores(q.to(DEV), means.to(DEV), bs, nb, cu_seqlens=None if new is None else cu.to(DEV),
                                  lengths=torch.tensor(lens, dtype=torch.int32, device=DEV), block_table=table.to(DEV))
    placed = [(int(cu[i]) + r, i, lens[i] - n[i] + r) for i in range(4) for r in range(n[i])]
    mean_of = lambda i, b: means[table[i, b]] if 0 <= table[i, b] < pages else None  # noqa: E731
    want, want_counts = oracle.scores(q, mean_of, bs, nb, placed, hk, 1, 1)
    assert torch.equal(counts.cpu(), want_counts)
    size = q.double().norm(dim=2).max() * means.double().norm(dim=2).max() / math.sqrt(d)
    compare_scores(got, want, (3 * d + 8) * 2.0 ** -23 * size.item())


def test_selection_run():
    """Means, scores, the selection and attention, one after the other."""
    q, k, v, _, cu, _ = make(11, [700, 129], [700, 129], 8, 2, 128, 32, 1, torch.bfloat16)
    q, k, v, cu = gpu(q, k, v, cu)
    means = mt.block_means(k, 32, cu_seqlens=cu)
    scores, counts = mt.block_scores(q, means, 32, 22, cu_seqlens=cu)
    blocks = mt.topk_indices(scores.flatten(0, 1), counts.flatten(), 6).view(829, 2, 6)
    out, lse = mt.block_attention(q, k, v, blocks, 32, cu_seqlens=cu)
    picked = blocks.cpu()
    for t, pos in ((0, 0), (31, 31), (32, 32), (699, 699), (700, 0), (828, 128)):
        row = picked[t, 0][picked[t, 0] >= 0].tolist()
        assert row == sorted(set(row)) and row[0] == 0 and row[-1] == pos // 32 and len(row) == min(6, pos // 32 + 1)
    want, want_lse = oracle.attention(q.cpu(), k.cpu(), v.cpu(), picked, 32, cu.cpu())
    check_out(out, want, lse, want_lse, v.cpu(), 40, 128, torch.bfloat16)
