"""GPU: block attention over many rows, where a workgroup takes 128 of them: the
cases of the other tests, repeated as packed sequences until there are enough.
The copies' arithmetic is the same, so their results are equal; one of them is
compared with the 64-bit form, within the tolerances of those tests."""

import math

import pytest
import torch

import attention_oracle as oracle
import row_wise_top_topk_amd as mt
from test_gpu_attention_hidden import agree, inputs
from test_gpu_block_attention import CASES, check_out, make
from test_gpu_block_attention_grad import check

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def copies_for(lens, heads, kv_heads):
    """Enough of them for 700 workgroups of 128 rows."""
    per = 128 // (heads // kv_heads)
    return -(-700 // (kv_heads * sum(max(1, n // per) for n in lens)))


def cu_of(lens, copies):
    return torch.tensor([0] + lens * copies).cumsum(0).to(torch.int32).to(DEV)


def repeat(x, copies):
    return x.repeat(copies, *[1] * (x.dim() - 1)).to(DEV)


def same(x, copies, rows):
    """The first copy, after a look at whether all are equal."""
    x = x.detach().view(copies, rows, *x.shape[1:])
    assert torch.equal(torch.nan_to_num(x, 7.0), torch.nan_to_num(x[:1], 7.0).expand_as(x))
    return x[0]


@pytest.mark.parametrize("case", [c for c in CASES if not c[-1]], ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_forward_and_gradient(case, causal):
    lq, lk, h, hk, d, bs, select, dtype, _ = case
    q, k, v, blocks, cu_q, cu_k = make(21, lq, lk, h, hk, d, bs, select, dtype)
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(1)).to(dtype)
    want, want_lse, *grads, sizes = oracle.attention(q, k, v, blocks, bs, cu_q, cu_k, causal=causal, dout=dout)
    n = copies_for(lq, h, hk)
    t, tk = sum(lq), sum(lk)
    leaves = [repeat(x, n).requires_grad_() for x in (q, k, v)]
    rest = dict(cu_seqlens=cu_of(lq, n), cu_seqlens_k=cu_of(lk, n), causal=causal)
    out, lse = mt.block_attention(*leaves, repeat(blocks, n), bs, **rest)
    with torch.no_grad():
        plain, plain_lse = mt.block_attention(*leaves, repeat(blocks, n), bs, **rest)
    smax = (q.double().norm(dim=2).max() * k.double().norm(dim=2).max() / math.sqrt(d)).item()
    for o, l in ((out, lse), (plain, plain_lse)):
        check_out(same(o, n, t), want, same(l, n, t), want_lse, v, smax, d, dtype)
    got = torch.autograd.grad(out, leaves, repeat(dout, n))
    got = [same(g, n, r) for g, r in zip(got, (t, tk, tk))]
    factor = max(x.abs().max().item() for x in (q, k, dout))
    check(got, grads, sizes, dtype, (h // hk) * max(max(lq), max(lk)), factor)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bs,d", [(16, 64), (32, 128), (64, 128), (64, 64)])
@pytest.mark.parametrize("where", ["k", "v"])
def test_hidden_nan(dtype, bs, d, where):
    q, k, v, blocks, g = inputs(bs, d, dtype)
    x = k if where == "k" else v
    x[bs + 3, 0, 5] = x[140, 1, 7] = math.nan
    dout = torch.randn(q.shape, generator=g).to(dtype)
    want, _, *grads, sizes = oracle.attention(q, k, v, blocks, bs, dout=dout)
    n = copies_for([150], 4, 2)
    leaves = [repeat(y, n).requires_grad_() for y in (q, k, v)]
    u = torch.finfo(dtype).eps / 2
    out, _ = mt.block_attention(*leaves, repeat(blocks, n), bs, cu_seqlens=cu_of([150], n))
    with torch.no_grad():
        plain, _ = mt.block_attention(*leaves, repeat(blocks, n), bs, cu_seqlens=cu_of([150], n))
    top = v[torch.isfinite(v)].abs().max().item()
    for o in (out, plain):
        agree(same(o, n, 150), want, 2.25 * u * top)
    few = 2.0 ** -25 * 200 * 16 if dtype == torch.float16 else 0.0
    for got, w, size in zip(torch.autograd.grad(out, leaves, repeat(dout, n)), grads, sizes):
        agree(same(got, n, 150), w, 1.25 * u * (size + w.abs()) + few)


def test_without_the_rest_of_the_rounding():
    """The explicit gradient without ``rest``: delta from the rounded output, the tolerances count that."""
    q, k, v, blocks, _, _ = make(5, [200], [200], 8, 2, 64, 32, 3, torch.bfloat16)
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    _, _, *grads, sizes = oracle.attention(q, k, v, blocks, 32, dout=dout)
    q, k, v, blocks, dout = (x.to(DEV) for x in (q, k, v, blocks, dout))
    out = torch.empty_like(q)
    got, lse = mt.block_attention(q, k, v, blocks, 32, out=out)
    assert got is out
    check(mt.block_attention_backward(dout, q, k, v, out, lse, blocks, 32), grads, sizes, torch.bfloat16, 0, 0)


@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 9, 16, 17, 31, 33, 40, 63, 64, 65, 100, 127, 128])
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 64)])
def test_any_group(group, d, bs):
    """Heads a key head from 1 to 128: attention, gradient, scores and the cache's step."""
    from test_gpu_kv8 import build, check as check_cache, put
    dtype = torch.float16 if group % 2 else torch.bfloat16
    q, k, v, blocks, cu, _ = make(group, [23, 9], [23, 9], group, 1, d, bs, 2, dtype)
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(4)).to(dtype)
    want, want_lse, *grads, sizes = oracle.attention(q, k, v, blocks, bs, cu, cu, dout=dout)
    leaves = [x.to(DEV).requires_grad_() for x in (q, k, v)]
    out, lse = mt.block_attention(*leaves, blocks.to(DEV), bs, cu_seqlens=cu.to(DEV))
    smax = (q.double().norm(dim=2).max() * k.double().norm(dim=2).max() / math.sqrt(d)).item()
    check_out(out.detach(), want, lse, want_lse, v, smax, d, dtype)
    got = torch.autograd.grad(out, leaves, dout.to(DEV))
    check(got, grads, sizes, dtype, group * 23, max(x.abs().max().item() for x in (q, k, dout)))
    means = mt.block_means(k.to(DEV), bs, cu_seqlens=cu.to(DEV))
    scores, counts = mt.block_scores(q.to(DEV), means, bs, 2, cu_seqlens=cu.to(DEV), first=0, last=0)
    m = means.cpu().double()
    placed = [(a + r, i, r) for i, (a, n) in enumerate(((0, 23), (23, 9))) for r in range(n)]
    ws, wc = oracle.scores(q, lambda i, b: m[int(cu[i]) // bs + i + b], bs, 2, placed, 1, 0, 0)
    assert torch.equal(counts.cpu(), wc)
    fin = torch.isfinite(ws)
    size = (q.double().norm(dim=2).max() * m.norm(dim=2).max() / math.sqrt(d)).item()
    assert torch.equal(scores.cpu()[~fin].double(), ws[~fin])
    assert (scores.cpu().double() - ws)[fin].abs().max().item() <= (3 * d + 8) * 2.0 ** -23 * size
    lens = [130, 31]
    kc, vc, ks, vs, table = build(3, lens, 1, d, bs)
    for new in (1, 3):
        cu = torch.tensor([0, new, 2 * new], dtype=torch.int32)
        one = q[:2 * new].contiguous()
        want, want_lse = oracle.cache_attention(one, kc, vc, ks, vs, table, lens, bs, cu)
        out, lse = mt.kv8_attention(one.to(DEV), *put(kc, vc, ks, vs, table), torch.tensor(lens, dtype=torch.int32, device=DEV), cu_seqlens=cu.to(DEV))
        check_cache(out, lse, want, want_lse, one, kc, vc, ks, vs, d, dtype)
