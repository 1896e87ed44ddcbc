"""GPU: the gradient of block sparse attention against the formulas in 64 bits
and against differences.

Tolerances, u half a step of the type, relative.  dv: the probabilities are
rounded (u of each term) and the result (u).  dq and dk: the scores' gradients
are rounded (u of each term); delta comes from the rounded out, which moves a
score's gradient by at most u p sum |dout out|; the result is rounded.  So an
element may be off by u (sum of the absolute terms, counted so) + u |result|;
a quarter more for the 32-bit scores and exponentials (fp16: their relative
error of 2^-15 at scores up to 100 against u = 2^-11, twice), and fp16's smallest
step 2^-25 for each of the n terms times the largest factor.
"""

import math

import pytest
import torch

import attention_oracle as oracle
import row_wise_top_topk_amd as mt
from test_gpu_block_attention import CASES, gpu, make

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def check(got, want, sizes, dtype, terms, factor):
    u = torch.finfo(dtype).eps / 2
    for name, g, w, s in zip(("dq", "dk", "dv"), got, want, sizes):
        assert torch.isfinite(g).all(), name
        allowed = 1.25 * u * (s + w.abs()) + (2.0 ** -24 * terms * factor if dtype == torch.float16 else 0) + 1e-30
        off = (g.cpu().double() - w).abs()
        assert (off <= allowed).all(), (name, (off / allowed).max().item(), off.max().item())


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("causal", [True, False])
def test_gradient(case, causal):
    lq, lk, h, hk, d, bs, select, dtype, tail = case
    q, k, v, blocks, cu_q, cu_k = make(17, lq, lk, h, hk, d, bs, select, dtype, tail)
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(1)).to(dtype)
    _, _, *want, sizes = oracle.attention(q, k, v, blocks, bs, cu_q, cu_k, causal=causal, dout=dout)
    leaves = [x.to(DEV).requires_grad_() for x in (q, k, v)]
    out, lse = mt.block_attention(*leaves, blocks.to(DEV), bs, cu_seqlens=cu_q.to(DEV), cu_seqlens_k=cu_k.to(DEV), causal=causal)
    assert not lse.requires_grad
    got = torch.autograd.grad(out, leaves, dout.to(DEV))
    factor = max(x.abs().max().item() for x in (q, k, dout))
    check(got, want, sizes, dtype, (h // hk) * max(lq) if max(lq) > max(lk) else (h // hk) * max(lk), factor)
    if tail:
        assert all((x[-tail:] == 0).all() for x in got)
    again = torch.autograd.grad(mt.block_attention(*leaves, blocks.to(DEV), bs, cu_seqlens=cu_q.to(DEV),
                                                   cu_seqlens_k=cu_k.to(DEV), causal=causal)[0], leaves, dout.to(DEV))
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_blocks_in_many_pieces():
    # every token selects block 0: with 16 heads a group it is cut into pieces of 128 tokens
    q, k, v, blocks, _, _ = make(2, [700], [700], 16, 1, 64, 64, 2, torch.bfloat16)
    blocks[:, :, 0] = 0
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    _, _, *want, sizes = oracle.attention(q, k, v, blocks, 64, dout=dout)
    leaves = [x.to(DEV).requires_grad_() for x in (q, k, v)]
    out, _ = mt.block_attention(*leaves, blocks.to(DEV), 64)
    check(torch.autograd.grad(out, leaves, dout.to(DEV)), want, sizes, torch.bfloat16, 700 * 16, 6)


def test_repeated_blocks_count_once():
    q, k, v, blocks, _, _ = make(4, [100], [100], 4, 2, 64, 16, 3, torch.float16)
    twice = torch.cat([blocks, blocks.flip(2)], 2)
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(3)).to(torch.float16).to(DEV)
    q, k, v, blocks, twice = gpu(q, k, v, blocks, twice)
    grads = []
    for b in (blocks, twice):
        out, lse = mt.block_attention(q, k, v, b, 16)
        grads.append(mt.block_attention_backward(dout, q, k, v, out, lse, b, 16))
    assert all(torch.equal(a, b) for a, b in zip(*grads))


def test_differences():
    """sum(out * w) moves by grad . step along a random direction of each input.
    The steps are multiples of a power of two that keep the inputs exact in
    bfloat16's 8 bits; the 64-bit form of the moved inputs gives the difference,
    central, so of second order in the step: 2^-6 of inputs of size 1 leaves
    about 2^-12 of the change's size; the gradient's own rounding 1.25 u of the
    absolute terms."""
    g = torch.Generator().manual_seed(6)
    q, k, v, blocks, _, _ = make(5, [40], [40], 4, 2, 64, 16, 2, torch.bfloat16)
    w = torch.randn(q.shape, generator=g).to(torch.bfloat16)
    leaves = [x.to(DEV).requires_grad_() for x in (q, k, v)]
    out, _ = mt.block_attention(*leaves, blocks.to(DEV), 16)
    grads = [x.cpu().double() for x in torch.autograd.grad(out, leaves, w.to(DEV))]
    _, _, _, _, _, sizes = oracle.attention(q, k, v, blocks, 16, dout=w)
    for i in range(3):
        step = torch.randn(leaves[i].shape, generator=g, dtype=torch.float64) * 2.0 ** -6
        up, down = [x.double() for x in (q, k, v)], [x.double() for x in (q, k, v)]
        up[i], down[i] = up[i] + step, down[i] - step
        change = ((oracle.attention(*up, blocks, 16)[0] - oracle.attention(*down, blocks, 16)[0]) * w.double()).sum() / 2
        predicted = (grads[i] * step).sum()
        allowed = 1.25 * 2.0 ** -8 * ((sizes[i] + grads[i].abs()) * step.abs()).sum() + 2.0 ** -10 * (grads[i].abs() * step.abs()).sum()
        assert abs(change - predicted) <= allowed, (i, change.item(), predicted.item(), allowed.item())


def test_shared_and_broadcast_inputs():
    """One key head expanded to all, keys that are the values, a summed loss (an expanded gradient)."""
    g = torch.Generator().manual_seed(7)
    q = torch.randn(70, 4, 64, generator=g).to(torch.bfloat16).to(DEV).requires_grad_()
    x = torch.randn(70, 1, 64, generator=g).to(torch.bfloat16).to(DEV).requires_grad_()
    blocks = torch.zeros(70, 4, 1, dtype=torch.int32, device=DEV)
    kv = x.expand(70, 4, 64)
    out, _ = mt.block_attention(q, kv, kv, blocks, 128)
    dq, dx = torch.autograd.grad(out.float().sum(), (q, x))
    one = torch.zeros(70, 1, 1, dtype=torch.int32)
    ones = torch.ones(70, 4, 64)
    _, _, wq, wk, wv, (sq, sk, sv) = oracle.attention(q.detach().cpu(), x.detach().cpu(), x.detach().cpu(), one, 128, dout=ones)
    u = 2.0 ** -8
    # the four heads' and both uses' gradients are rounded each, and the sums of them twice
    assert ((dx.cpu().double() - (wk + wv)).abs() <= 1.25 * u * (sk + sv + 4 * (wk.abs() + wv.abs()) + sk + sv)).all()
    assert ((dq.cpu().double() - wq).abs() <= 1.25 * u * (sq + wq.abs())).all()


def test_only_some_gradients():
    q, k, v, blocks, _, _ = make(5, [40], [40], 4, 2, 64, 16, 2, torch.bfloat16)
    q, k, v, blocks = gpu(q, k, v, blocks)
    k.requires_grad_()
    out, _ = mt.block_attention(q, k, v, blocks, 16)
    out.float().square().sum().backward()
    assert k.grad is not None and q.grad is None and v.grad is None
    with torch.no_grad():
        assert not mt.block_attention(q, k, v, blocks, 16)[0].requires_grad


def test_training_step_falls_nowhere_but_runs():
    """Selection and attention in one differentiable step over packed documents; gradients reach all leaves."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn(300, 64, generator=g).to(torch.bfloat16).to(DEV)
    wq, wk, wv = (((torch.randn(64, n, generator=g) / 8).to(torch.bfloat16).to(DEV)).requires_grad_() for n in (512, 128, 128))
    cu = torch.tensor([0, 170, 300], dtype=torch.int32, device=DEV)
    q, k, v = (x @ wq).view(300, 8, 64), (x @ wk).view(300, 2, 64), (x @ wv).view(300, 2, 64)
    with torch.no_grad():
        means = mt.block_means(k, 16, cu_seqlens=cu)
        scores, counts = mt.block_scores(q, means, 16, 11, cu_seqlens=cu)
        blocks = mt.topk_indices(scores.flatten(0, 1), counts.flatten(), 4).view(300, 2, 4)
    out, _ = mt.block_attention(q, k, v, blocks, 16, cu_seqlens=cu)
    out.float().square().mean().backward()
    for w in (wq, wk, wv):
        assert torch.isfinite(w.grad).all() and w.grad.abs().max() > 0
