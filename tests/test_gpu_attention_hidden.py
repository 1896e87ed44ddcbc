"""GPU: infinities and NaN that a query does not see do not reach its results.

Results that are not finite in the 64-bit form are not finite, all others are
within the tolerances of the finite tests (2.25 u max|v| for out; for the
gradients 1.25 u of their terms, see those tests)."""

import math

import pytest
import torch

import attention_oracle as oracle
import row_wise_top_topk_amd as mt

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAN, INF = math.nan, math.inf


def agree(got, want, allowed):
    got = got.cpu().double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin), (torch.isfinite(got) ^ fin).nonzero()[:5]
    allowed = allowed[fin] if isinstance(allowed, torch.Tensor) else allowed
    assert ((got[fin] - want[fin]).abs() <= allowed).all()


def inputs(bs, d, dtype, h=4, hk=2, t=150, seed=3):
    """Tokens select their own block and block 0; two of three also block 1, from token 100 on also block 2."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(t, h, d, generator=g).to(dtype)
    k, v = (torch.randn(t, hk, d, generator=g).to(dtype) for _ in range(2))
    blocks = torch.full((t, hk, 4), -1, dtype=torch.int32)
    blocks[:, :, 0] = 0
    blocks[:, :, 1] = (torch.arange(t) // bs).to(torch.int32)[:, None]
    blocks[torch.arange(t) % 3 != 0, 0, 2] = 1
    blocks[100:, :, 3] = 2
    return q, k, v, blocks, g


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bs,d", [(16, 64), (32, 128), (64, 128)])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_forward_and_gradient(dtype, bs, d, where, value):
    q, k, v, blocks, g = inputs(bs, d, dtype)
    x = k if where == "k" else v
    if where == "k" and math.isinf(value):      # scores of -inf, weights of 0
        x[145, 0, 0] = value
        q[145:, :2, 0] = -math.copysign(1.0, value)
    else:
        x[bs + 3, 0, 5] = value                 # in block 1: some tokens do not select it
        x[140, 1, 7] = value                    # hidden from the tokens before it
    dout = torch.randn(q.shape, generator=g).to(dtype)
    want, want_lse, wq, wk, wv, (sq, sk, sv) = oracle.attention(q, k, v, blocks, bs, dout=dout)
    assert torch.isfinite(want).any() and not torch.isfinite(wq).all()
    u = torch.finfo(dtype).eps / 2
    leaves = [t.to(DEV).requires_grad_() for t in (q, k, v)]
    out, lse = mt.block_attention(*leaves, blocks.to(DEV), bs)
    with torch.no_grad():
        plain, plain_lse = mt.block_attention(*leaves, blocks.to(DEV), bs)
    top = v[torch.isfinite(v)].abs().max().item()
    for o, l in ((out, lse), (plain, plain_lse)):
        agree(o.detach(), want, 2.25 * u * top)
        assert torch.equal(torch.isfinite(l.detach().cpu()), torch.isfinite(want_lse))
    dq, dk, dv = torch.autograd.grad(out, leaves, dout.to(DEV))
    few = 2.0 ** -25 * 200 * 16 if dtype == torch.float16 else 0.0    # fp16's smallest step, over the terms
    agree(dq, wq, 1.25 * u * (sq + wq.abs()) + few)
    agree(dk, wk, 1.25 * u * (sk + wk.abs()) + few)
    agree(dv, wv, 1.25 * u * (sv + wv.abs()) + few)


def test_gradient_of_output_rows():
    """A NaN in one row's output gradient reaches that row's dq and the keys it sees."""
    q, k, v, blocks, g = inputs(32, 64, torch.bfloat16)
    dout = torch.randn(q.shape, generator=g).to(torch.bfloat16)
    dout[70, 1, 3] = NAN
    dout[20, 2, 9] = INF
    _, _, wq, wk, wv, (sq, sk, sv) = oracle.attention(q, k, v, blocks, 32, dout=dout)
    leaves = [t.to(DEV).requires_grad_() for t in (q, k, v)]
    grads = torch.autograd.grad(mt.block_attention(*leaves, blocks.to(DEV), 32)[0], leaves, dout.to(DEV))
    for got, want, size in zip(grads, (wq, wk, wv), (sq, sk, sv)):
        agree(got, want, 1.25 * 2.0 ** -8 * (size + want.abs()))


def test_scores_of_infinite_means():
    g = torch.Generator().manual_seed(1)
    for dtype in (torch.bfloat16, torch.float16):
        q = torch.randn(200, 4, 64, generator=g).to(dtype)
        k = torch.randn(200, 2, 64, generator=g).to(dtype)
        k[20, 0, 3], k[70, 1, 5], k[90, 0, 0] = INF, -INF, NAN
        means = mt.block_means(k.to(DEV), 16)
        scores, counts = mt.block_scores(q.to(DEV), means, 16, 13)
        m = oracle.means(k, 16)
        want, want_counts = oracle.scores(q, lambda i, b: m[b], 16, 13, [(r, 0, r) for r in range(200)], 2, 1, 1)
        assert torch.equal(counts.cpu(), want_counts)
        got = scores.cpu().double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        odd = ~torch.isfinite(want) & ~torch.isnan(want)
        assert torch.equal(got[odd], want[odd]) and torch.equal(torch.isfinite(got), torch.isfinite(want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("h,hk,d,bs,new", [(8, 2, 128, 16, 3), (8, 1, 64, 64, 1), (16, 1, 128, 32, 2), (24, 1, 64, 16, 5), (4, 4, 128, 128, 9)])
@pytest.mark.parametrize("where", ["k", "v"])
def test_cache(dtype, h, hk, d, bs, new, where):
    """NaN codes in the new tokens: those before do not see them; and behind the lengths: nobody does."""
    from test_gpu_kv8 import build, put
    lens = [333, 70, 16]
    kc, vc, ks, vs, table = build(5, lens, hk, d, bs)
    g = torch.Generator().manual_seed(2)
    x = kc if where == "k" else vc
    for i, n in enumerate(lens):
        if i < 2:
            x[table[i, (n - 1) // bs], 0, (n - 1) % bs, 4 + i] = NAN       # the last token
        x[table[i, 0], hk - 1, 2, 17] = NAN if i == 1 else 1.0             # a token that all see
    q = torch.randn(new * 3, h, d, generator=g).to(dtype)
    cu = torch.tensor([0, new, 2 * new, 3 * new], dtype=torch.int32)
    want, _ = oracle.cache_attention(q, kc, vc, ks, vs, table, lens, bs, cu)
    dev = put(kc, vc, ks, vs, table)
    top = (vc.nan_to_num() * vs[:, :, None, None]).abs().max().item()
    for bound in (None, 1):
        out, _ = mt.kv8_attention(q.to(DEV), *dev, torch.tensor(lens, dtype=torch.int32, device=DEV), cu_seqlens=cu.to(DEV), max_length=bound)
        agree(out, want, 2.25 * torch.finfo(dtype).eps / 2 * top)
    # the step for single tokens, one before the NaN and one at it
    for back in (1, 0):
        short = [n - back for n in lens]
        one = q[:3].contiguous()
        want, _ = oracle.cache_attention(one, kc, vc, ks, vs, table, short, bs)
        out, _ = mt.kv8_attention(one.to(DEV), *dev, torch.tensor(short, dtype=torch.int32, device=DEV))
        agree(out, want, 2.25 * torch.finfo(dtype).eps / 2 * top)
