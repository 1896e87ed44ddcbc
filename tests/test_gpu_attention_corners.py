"""GPU: calls at the corners of the attention operators: head strides past 4 GiB,
caches and means of no rows, loops that only long inputs enter.

Where two calls have to agree they do the same arithmetic and their results are
equal; against the 64-bit forms the tolerances are those of the other tests."""

import math

import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import attention_oracle as oracle
import row_wise_top_topk_amd as mt
from test_gpu_attention_hidden import agree
from test_gpu_block_attention import check_out, gpu, make
from test_gpu_kv8 import build, check, put, same

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F16 = torch.bfloat16, torch.float16


def test_head_strides_past_4_gib():
    """Heads of q and dout that lie 4 GiB and more apart."""
    t, step = 70, (1 << 31) + (1 << 13)
    q, k, v, blocks, _, _ = make(9, [t], [t], 2, 1, 64, 16, 3, BF)
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(0)).to(BF)
    store = torch.zeros(step + 2 * t * 64, dtype=BF, device=DEV)
    far = [store[i * t * 64:].as_strided((t, 2, 64), (64, step, 1)) for i in range(2)]
    for view, x in zip(far, (q, dout)):
        view.copy_(x)
    near = gpu(q, dout)
    k, v, blocks = gpu(k, v, blocks)
    results = []
    for x, g in (near, far):
        rest = torch.empty_like(q, device=DEV)
        out, lse = mt.block_attention(x, k, v, blocks, 16, rest=rest)
        results.append((out, lse, rest, *mt.block_attention_backward(g, x, k, v, out, lse, blocks, 16, rest=rest)))
    assert all(torch.equal(a, b) for a, b in zip(*results))
    means = mt.block_means(k, 16)
    for a, b in zip(*(mt.block_scores(x, means, 16, 5) for x in (near[0], far[0]))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("h,hk", [(8, 2), (24, 1), (128, 1)])
def test_scores_of_no_means(dtype, h, hk):
    """Means of no rows: a block of none of them has -inf, and the counts are the positions'."""
    means = torch.empty(0, hk, 128, device=DEV)
    q = torch.randn(5, h, 128, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    lengths = torch.tensor([1, 700, 0, 64, 65], dtype=torch.int32, device=DEV)
    table = torch.zeros(5, 11, dtype=torch.int32, device=DEV)
    cu = torch.arange(6, dtype=torch.int32, device=DEV)
    for c in (None, cu):
        scores, counts = mt.block_scores(q, means, 64, 11, cu_seqlens=c, lengths=lengths, block_table=table)
        assert (scores == -math.inf).all() and counts.tolist() == [[n] * hk for n in (1, 11, 0, 1, 2)]
    two = torch.tensor([0, 2, 5], dtype=torch.int32, device=DEV)
    keys = torch.tensor([0, 100, 350], dtype=torch.int32, device=DEV)
    scores, counts = mt.block_scores(q, means, 64, 4, cu_seqlens=two, cu_seqlens_k=keys)
    assert (scores == -math.inf).all() and counts.tolist() == [[n] * hk for n in (2, 2, 4, 4, 4)]


@pytest.mark.parametrize("tail", [0, 3])
def test_scores_of_an_empty_batch(tail):
    """A paged call without sequences, alone or with rows behind the last one."""
    means = torch.randn(4, 2, 64, device=DEV)
    q = torch.randn(tail, 4, 64, device=DEV).to(BF)
    table, lengths = (torch.zeros(*n, dtype=torch.int32, device=DEV) for n in ((3, 6), (3,)))
    cu = torch.zeros(1, dtype=torch.int32, device=DEV)
    for c in (cu,) if tail else (None, cu):
        for x, n in ((table[:0], lengths[:0]), (table[:0].clone(), lengths[:0].clone()), (table[:0], lengths[:0].clone())):
            scores, counts = mt.block_scores(q, means, 16, 6, cu_seqlens=c, lengths=n, block_table=x)
            assert scores.shape == (tail, 2, 6) and (scores == -math.inf).all() and (counts == 0).all() and counts.shape == (tail, 2)


def test_more_forced_blocks_than_32_bits_count():
    k = torch.randn(70, 2, 64, generator=torch.Generator().manual_seed(2)).to(BF).to(DEV)
    means = mt.block_means(k, 16)
    want, _ = mt.block_scores(k, means, 16, 5, first=5, last=0)
    for n in (1 << 31, 1 << 32, 1 << 70):
        for kw in (dict(first=n, last=0), dict(first=0, last=n)):
            assert torch.equal(mt.block_scores(k, means, 16, 5, **kw)[0], want)


def test_forward_mode_derivatives_are_refused():
    q, b = torch.zeros(10, 2, 64, dtype=BF, device=DEV), torch.zeros(10, 2, 1, dtype=torch.int32, device=DEV)
    means, lse = torch.zeros(1, 2, 64, device=DEV), torch.zeros(10, 2, device=DEV)
    with forward_ad.dual_level():
        calls = [(mt.block_attention, (q, q, q, b, 16), 3), (mt.block_attention_backward, (q, q, q, q, q, lse, b, 16), 4),
                 (mt.block_scores, (q, means, 16, 1), 2), (mt.block_means, (q, 16), 1)]
        for fn, args, operands in calls:
            fn(*args)
            for i in range(operands):
                dual = forward_ad.make_dual(args[i], torch.ones_like(args[i]))
                with pytest.raises(ValueError, match="forward-mode"):
                    fn(*args[:i], dual, *args[i + 1:])
                if fn is mt.block_attention and i < 3:
                    with pytest.raises((ValueError, RuntimeError, NotImplementedError)):
                        fn(*(t.clone().requires_grad_() if j < 3 and j != i else t for j, t in enumerate((*args[:i], dual, *args[i + 1:]))))


def test_capture_on_a_stream_of_later_graphs():
    """Leaves whose first graph was another stream's: the later graphs' stream does not make them fit for a capture on it."""
    q, k, v, blocks, _, _ = make(3, [40], [40], 4, 2, 64, 16, 2, BF)
    blocks = blocks.to(DEV)
    leaves = [x.to(DEV).requires_grad_() for x in (q, k, v)]
    stream = torch.cuda.Stream()
    first = mt.block_attention(*leaves, blocks, 16)[0]
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        second = mt.block_attention(*leaves, blocks, 16)[0]
    torch.cuda.synchronize()
    del first                                               # the second keeps the node that the first made
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        with pytest.raises(RuntimeError, match="captured"):
            mt.block_attention(*leaves, blocks, 16)
        with torch.no_grad():
            plain = mt.block_attention(*leaves, blocks, 16)[0]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.isfinite(plain).all() and plain.abs().max() > 0
    del second
    with torch.cuda.stream(stream):
        want = torch.autograd.grad(mt.block_attention(*leaves, blocks, 16)[0], leaves, torch.ones_like(leaves[0]))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph := torch.cuda.CUDAGraph(), stream=stream):
        got = torch.autograd.grad(mt.block_attention(*leaves, blocks, 16)[0], leaves, torch.ones_like(leaves[0]))
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_bounds_of_the_lengths_past_64_bits():
    lens = [700]
    dev = put(*build(1, lens, 1, 64, 16))
    q = torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    want = mt.kv8_attention(q, *dev, torch.tensor(lens, dtype=torch.int32, device=DEV))
    for n in ((1 << 63) - 1, 1 << 63, 1 << 70):
        got = mt.kv8_attention(q, *dev, torch.tensor(lens, dtype=torch.int32, device=DEV), max_length=n)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("selected", [False, True])
def test_nan_of_a_key_that_weighs_nothing(dtype, selected):
    """A visible NaN counts in whatever chunk it lies: its weight is 0 in 64 bits too, and 0 times it is NaN."""
    lens = [700]
    kc, vc, ks, vs, table = build(1, lens, 1, 64, 16, spare=0)
    kc[:] = 0.0
    ks[:] = 1.0
    vc = vc.nan_to_num()
    kc[table[0, 0], 0, 5] = 30.0
    vc[table[0, 37], 0, 8, 3] = math.nan                       # key 600
    q = torch.full((1, 4, 64), 8.0, dtype=dtype)               # the score of key 5 is 1920, all others' 0
    blocks = torch.arange(44, dtype=torch.int32).expand(1, 1, 44).contiguous() if selected else None
    want, want_lse = oracle.cache_attention(q, kc, vc, ks, vs, table, lens, 16, blocks=blocks)
    assert torch.isnan(want[0, :, 3]).all() and torch.isfinite(want).sum() == 4 * 63
    dev = put(kc, vc, ks, vs, table)
    top = (vc.nan_to_num() * vs[:, :, None, None]).abs().max().item()
    for bound in (None, 1):                                    # six chunks, one chunk
        out, lse = mt.kv8_attention(q.to(DEV), *dev, torch.tensor(lens, dtype=torch.int32, device=DEV),
                                    blocks=None if blocks is None else blocks.to(DEV), max_length=bound)
        agree(out, want, 2.25 * torch.finfo(dtype).eps / 2 * top)
        assert (lse.cpu().double() - want_lse).abs().max().item() <= 2.0 ** -24 * 128 * 1930


def test_many_small_weights():
    """800000 keys that each weigh 2^-26 of the first one, in one chunk: together more than fp16's step.  Weights are
    held to 2^-39 of a wavefront's largest one, which over 2^20 keys is 2^-19 max|v|, within the quarter.  A wavefront adds
    up 12500 groups of weights in 32 bits: 12500 * 2^-24, relative, of the sum."""
    lens = [800_000]
    pages = lens[0] // 128
    kc, vc = torch.zeros(pages, 1, 128, 64), torch.ones(pages, 1, 128, 64)
    kc[0, 0, 0], vc[0, 0, 0] = 2.25, 0.0
    ks = vs = torch.ones(pages, 1)
    table = torch.arange(pages, dtype=torch.int32)[None]
    q = torch.ones(1, 1, 64, dtype=F16)                        # scores 18 and 0: 2^26 to 1
    want, want_lse = oracle.cache_attention(q, kc, vc, ks, vs, table, lens, 128)
    dev = put(kc, vc, ks, vs, table)
    for bound in (1, None):
        out, lse = mt.kv8_attention(q.to(DEV), *dev, torch.tensor(lens, dtype=torch.int32, device=DEV), max_length=bound)
        allowed = (2.25 * 2.0 ** -11 + 12500 * 2.0 ** -24) * want
        assert ((out.cpu().double() - want).abs() <= allowed).all(), (out[0, 0, 0].item(), want[0, 0, 0].item())
        assert (lse.cpu().double() - want_lse).abs().max().item() <= 2.0 ** -24 * (128 * 28 + 12500)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("scale", [2.0 ** -80, 2.0 ** -60, 2.0 ** 100])
def test_the_least_and_largest_value_scales(dtype, scale):
    """Sums of weights that are divided by the scale, over 20000 keys in one chunk: in fp32's range."""
    lens = [20000]
    kc, vc, ks, vs, table = build(3, lens, 1, 64, 128)
    vs[:] = scale
    q = (2 * torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(5))).to(dtype)
    want, want_lse = oracle.cache_attention(q, kc, vc, ks, vs, table, lens, 128)
    dev = put(kc, vc, ks, vs, table)
    top = (vc.nan_to_num() * vs[:, :, None, None]).abs().max().item()
    smax = (q.double().norm(dim=2).max() * (kc.nan_to_num() * ks[:, :, None, None]).double().norm(dim=3).max() / 8).item()
    for bound in (None, 1):
        out, lse = mt.kv8_attention(q.to(DEV), *dev, torch.tensor(lens, dtype=torch.int32, device=DEV), max_length=bound)
        if dtype == BF:
            assert (out.cpu().double() - want).abs().max().item() <= 2.25 * 2.0 ** -8 * top
        else:
            assert ((out == 0) if scale < 1 else torch.isinf(out)).all()      # fp16 has neither these values nor a step that near 0
        # the logarithm of the sum and the maximum carry that of the scale: up to 80 ln 2 beside the score
        assert (lse.cpu().double() - want_lse).abs().max().item() <= 2.0 ** -24 * 128 * (smax + 10 + 70)


@pytest.mark.parametrize("heads", [1, 128])
def test_many_small_weights_of_selected_blocks(heads):
    """131072 keys that each weigh 2^-26 of the first one, the most that a query can select: together more than fp16's
    step.  Weights are held to 2^-32 of the largest one, which over 2^17 keys is 2^-15 max|v|; a lane adds up 8192
    groups of weights in 32 bits."""
    t = 131072
    q = torch.ones(1, heads, 64, dtype=F16)
    k, v = torch.zeros(t, 1, 64, dtype=F16), torch.ones(t, 1, 64, dtype=F16)
    k[0], v[0] = 2.25, 0.0                                     # scores 18 and 0
    blocks = torch.arange(1024, dtype=torch.int32).expand(1, 1, 1024).contiguous()
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (1, t))
    want = (t - 1) / (math.exp(18) + t - 1)
    want_lse = math.log(math.exp(18) + t - 1)
    leaves = [x.to(DEV).requires_grad_() for x in (q, k, v)]
    out, lse = mt.block_attention(*leaves, blocks.to(DEV), 128, cu_seqlens=cu_q, cu_seqlens_k=cu_k)
    with torch.no_grad():
        plain, plain_lse = mt.block_attention(*leaves, blocks.to(DEV), 128, cu_seqlens=cu_q, cu_seqlens_k=cu_k)
    allowed = (2.25 * 2.0 ** -11 + 8192 * 2.0 ** -24) * want + 2.0 ** -15
    for o, l in ((out, lse), (plain, plain_lse)):
        assert ((o.detach().cpu().double() - want).abs() <= allowed).all(), (o[0, 0, 0].item(), want)
        assert ((l.cpu().double() - want_lse).abs() <= 2.0 ** -24 * (128 * 28 + 8192)).all()


def windows(seed, t, h, hk, d, few, dtype):
    """t queries at the end of 17600 keys in blocks of 16: 1100 block numbers, more than a workgroup's window of them
    at any number of tokens (2048 words of token bits, one a block for 32 tokens).  Only the tokens of ``few`` select
    anything, half of it on each side of the borders at 512 and 1024."""
    keys = 17600
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(t, h, d, generator=g).to(dtype)
    k, v = (torch.randn(keys, hk, d, generator=g).to(dtype) for _ in range(2))
    dout = torch.randn(t, h, d, generator=g).to(dtype)
    blocks = torch.full((t, hk, 12), -1, dtype=torch.int32)
    for r in few:
        for c in range(hk):
            pick = [511, 512, 1023, 1024, 1055] + torch.randint(0, 1056, (6,), generator=g).tolist()
            blocks[r, c, :11] = torch.tensor(pick, dtype=torch.int32)[torch.randperm(11, generator=g)]
            blocks[r, c, 11] = (keys - t + r) // 16
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32) for n in (t, keys))
    return q, k, v, dout, blocks, cu_q, cu_k


WINDOWS = [
    # tokens, heads, kv_heads, dim, tokens that select, type
    (40, 2, 2, 64, range(40), BF),                             # 64 rows a workgroup: windows of 1024 block numbers
    (600, 1, 1, 128, range(0, 600, 37), F16),
    (70, 16, 2, 128, range(0, 70, 3), BF),                     # several heads a group: one window
    (3200, 16, 16, 128, range(2005, 3200, 149), BF),              # 416 workgroups of 128 rows: windows of 512
]


@pytest.mark.parametrize("hidden", [False, True])
@pytest.mark.parametrize("case", WINDOWS, ids=[str(i) for i in range(len(WINDOWS))])
def test_windows_of_block_numbers(case, hidden):
    """Blocks in several windows, forward and gradient; with NaN at a key that few see, so that the walk key by key
    passes the borders too."""
    t, h, hk, d, few, dtype = case
    q, k, v, dout, blocks, cu_q, cu_k = windows(3, t, h, hk, d, few, dtype)
    few = list(few)
    if hidden:
        blocks[few[1:]] = torch.where(blocks[few[1:]] == 1024, -1, blocks[few[1:]])
        blocks[few[0], :, 0] = 1024
        k[1024 * 16 + 3, 0, 5], v[1024 * 16 + 9, hk - 1, 7] = math.nan, math.nan
    dout[[r for r in range(t) if r not in set(few)]] = 0.0
    want, want_lse, *wants, sizes = oracle.attention(q, k, v, blocks, 16, cu_q, cu_k, dout=dout)
    leaves = [x.to(DEV).requires_grad_() for x in (q, k, v)]
    args = dict(cu_seqlens=cu_q.to(DEV), cu_seqlens_k=cu_k.to(DEV))
    out, lse = mt.block_attention(*leaves, blocks.to(DEV), 16, **args)
    with torch.no_grad():
        plain, plain_lse = mt.block_attention(*leaves, blocks.to(DEV), 16, **args)
    u = torch.finfo(dtype).eps / 2
    if not hidden:
        for o, l in ((out, lse), (plain, plain_lse)):
            check_out(o.detach(), want, l, want_lse, v, 80, d, dtype)
    else:
        assert torch.isnan(want).any() and torch.isfinite(want[few[1:]]).all()
        for o in (out, plain):
            agree(o.detach(), want, 2.25 * u * v.nan_to_num().abs().max().item())
    step = 2.0 ** -24 * (h // hk) * len(few) * 8 if dtype == F16 else 0.0
    for got, w, s in zip(torch.autograd.grad(out, leaves, dout.to(DEV)), wants, sizes):
        agree(got, w, 1.25 * u * (s + w.abs()) + step + 1e-30)


def picks(g, select, nb, rows, hk):
    """Rows of ``select`` entries: block numbers in any order with repeats, and some that name no block."""
    out = torch.empty(rows, hk, select, dtype=torch.int32)
    for r in range(rows):
        for c in range(hk):
            row = torch.randperm(nb, generator=g)[:select]
            if r % 2 == 0:
                row[select // 2:] = row[torch.randint(0, select // 2, (select - select // 2,), generator=g)]
                row[torch.randperm(select, generator=g)[:7]] = torch.tensor([-1, nb, -(1 << 31), (1 << 31) - 1, -5, nb + 3, 0])
            elif r % 4 == 1:
                row = row.sort()[0]
            out[r, c] = row.to(torch.int32)
    return out


@pytest.mark.parametrize("select", [255, 256, 257, 700, 1024])
@pytest.mark.parametrize("dtype", [BF, F16])
def test_many_selected_blocks_of_a_cache(select, dtype):
    """Selections of more entries than a workgroup has threads, up to the limit; many chunks and one."""
    lens = [20000, 17001]
    kc, vc, ks, vs, table = build(6, lens, 2, 64, 16)
    g = torch.Generator().manual_seed(select)
    q = (2 * torch.randn(5, 4, 64, generator=g)).to(dtype)
    cu = torch.tensor([0, 2, 5], dtype=torch.int32)
    blocks = picks(g, select, 1250, 5, 2)
    want, want_lse = oracle.cache_attention(q, kc, vc, ks, vs, table, lens, 16, cu, blocks)
    dev = put(kc, vc, ks, vs, table)
    for bound in (None, 1):
        out, lse = mt.kv8_attention(q.to(DEV), *dev, torch.tensor(lens, dtype=torch.int32, device=DEV), cu_seqlens=cu.to(DEV),
                                    blocks=blocks.to(DEV), max_length=bound)
        check(out, lse, want, want_lse, q, kc, vc, ks, vs, 64, dtype)


@pytest.mark.parametrize("select", [257, 1024])
@pytest.mark.parametrize("h,hk,dtype", [(4, 2, BF), (32, 1, F16)])
def test_many_selected_blocks(select, h, hk, dtype):
    g = torch.Generator().manual_seed(select)
    q, k, v, _, cu_q, cu_k = make(2, [5, 3], [20000, 17001], h, hk, 64, 16, 1, dtype)
    dout = torch.randn(q.shape, generator=g).to(dtype)
    blocks = picks(g, select, 1250, 8, hk)
    want, want_lse, *wants, sizes = oracle.attention(q, k, v, blocks, 16, cu_q, cu_k, dout=dout)
    leaves = [x.to(DEV).requires_grad_() for x in (q, k, v)]
    out, lse = mt.block_attention(*leaves, blocks.to(DEV), 16, cu_seqlens=cu_q.to(DEV), cu_seqlens_k=cu_k.to(DEV))
    # fp16: 2^-25 of the largest weight for each of 16384 keys at most: 2^-11 max|v|, one half step beside the 2.25
    u = torch.finfo(dtype).eps / 2
    top = v.abs().double().max().item()
    assert (out.detach().cpu().double() - want).abs().max().item() <= (2.25 if dtype == BF else 3.25) * u * top
    assert (lse.cpu().double() - want_lse).abs().max().item() <= 2.0 ** -24 * 128 * 60
    # and of each term of the gradients: 16384 keys of dq, with the scale; 8 tokens and a group's heads of dk and dv
    for got, w, s, terms in zip(torch.autograd.grad(out, leaves, dout.to(DEV)), wants, sizes, (16384 / 8, 8 * h // hk, 8 * h // hk)):
        agree(got, w, 1.25 * u * (s + w.abs()) + (2.0 ** -25 * 6 * terms if dtype == F16 else 0.0) + 1e-30)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("lens,new,h,hk,d,bs", [
    ([9000, 4097], None, 8, 2, 128, 16),                        # three segments of 256 pages in one chunk; one page over
    ([9000], [3], 24, 1, 64, 16),
    ([40000, 300], None, 4, 1, 64, 16),                         # 313 chunks: more than the join's 4 x 64
    ([70000], [2], 40, 1, 128, 32),
])
def test_long_caches(lens, new, h, hk, d, bs, dtype):
    """Chunks of several segments of pages, joins of several rounds of chunks.  Over more than 4096 keys fp16's smallest
    weights (2^-25 of the largest one, over n keys) add n * 2^-25 max|v| where one wavefront has them all."""
    kc, vc, ks, vs, table = build(7, lens, hk, d, bs)
    g = torch.Generator().manual_seed(4)
    n = [1] * len(lens) if new is None else new
    q = (2 * torch.randn(sum(n), h, d, generator=g)).to(dtype)
    cu = None if new is None else torch.tensor([0] + n).cumsum(0).to(torch.int32)
    want, want_lse = oracle.cache_attention(q, kc, vc, ks, vs, table, lens, bs, cu)
    dev = put(kc, vc, ks, vs, table)
    u = torch.finfo(dtype).eps / 2
    top = (vc.nan_to_num() * vs[:, :, None, None]).abs().max().item()
    smax = (q.double().norm(dim=2).max() * (kc.nan_to_num() * ks[:, :, None, None]).double().norm(dim=3).max() / math.sqrt(d)).item()
    for bound in (None, 1):
        out, lse = mt.kv8_attention(q.to(DEV), *dev, torch.tensor(lens, dtype=torch.int32, device=DEV),
                                    cu_seqlens=None if cu is None else cu.to(DEV), max_length=bound)
        allowed = 2.25 * u * top + (max(lens) / 4 * 2.0 ** -25 * top if dtype == F16 else 0.0)
        assert (out.cpu().double() - want).abs().max().item() <= allowed
        assert (lse.cpu().double() - want_lse).abs().max().item() <= 2.0 ** -24 * (d + 64) * (smax + 10)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_low_scores_and_a_part_of_a_block(dtype, bs):
    """Finite inputs whose scores are all far below 0, where the last block has few keys: right, and no slower by it."""
    t, h, hk, d = 1037, 16, 2, 64
    times = []
    for low in (0.0, 120.0):
        g = torch.Generator().manual_seed(bs)
        q, k, v, dout = (torch.randn(t, n, d, generator=g) for n in (h, hk, hk, h))
        q[..., 0], k[..., 0] = 16.0, -low / 2                   # all scores lower by low
        q, k, v, dout = (x.to(dtype) for x in (q, k, v, dout))
        blocks = torch.zeros(t, hk, 2, dtype=torch.int32)
        blocks[..., 1] = (t - 1) // bs
        want, want_lse, *wants, sizes = oracle.attention(q, k, v, blocks, bs, causal=False, dout=dout)
        assert low == 0 or want_lse.max() < -100
        args = gpu(q, k, v, blocks)
        rest = torch.empty_like(args[0])
        out, lse = mt.block_attention(*args, bs, causal=False, rest=rest)

        def run():
            return mt.block_attention_backward(dout.to(DEV), *args[:3], out, lse, args[3], bs, causal=False, rest=rest)

        got = run()
        u = torch.finfo(dtype).eps / 2
        # 32-bit scores of up to 130 and their exponentials: 2^-15, relative, of each term, twice, beside the types' roundings;
        # fp16's smallest step for each of the terms, a probability's times dout and a score's gradient's times q or k
        step = 2.0 ** -25 * t * (h // hk) * max(16.0, low / 2) if dtype == F16 else 0.0
        for x, w, s in zip(got, wants, sizes):
            agree(x, w, (1.25 * u + 2.0 ** -14) * (s + w.abs()) + step + 1e-30)
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        best = math.inf
        for _ in range(5):
            a.record()
            for _ in range(5):
                run()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
    assert times[1] < 4 * times[0], times


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("bs,d", [(16, 64), (128, 128)])
def test_append_of_more_tokens_than_lengths_or_table(dtype, bs, d):
    """More new tokens than a sequence's length (the first ones have no place), more than its table holds (the last ones
    have none), keys with strides of other tensors, one tensor for keys and values."""
    lens, new = [20, 2, 40 * bs, 5], [30, 5, 2 * bs + 3, 5]
    kc, vc, ks, vs, table = build(3, [20, 2, 3 * bs, 5], 2, d, bs)
    lens[2] = table.shape[1] * bs + 7                           # seven past the table
    g = torch.Generator().manual_seed(5)
    x = torch.randn(sum(new) + 1, 5, d, generator=g).to(dtype)
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    k = x[:, 1:4:2]
    for one in (False, True):
        v = k if one else x[:, 3:].contiguous()
        dev = put(kc, vc, ks, vs, table)
        mean = torch.full((kc.shape[0], 2, d), 7.0)
        mean_dev = mean.to(DEV)
        far = x.to(DEV)
        mt.kv8_append(far[:, 1:4:2], far[:, 1:4:2] if one else v.to(DEV), *dev, torch.tensor(lens, dtype=torch.int32, device=DEV),
                      cu_seqlens=cu.to(DEV), k_mean=mean_dev)
        want = [t.clone() for t in (kc, vc, ks, vs)]
        oracle.append(k, v, *want, table, lens, bs, cu, mean)
        assert all(same(a, b) for a, b in zip(dev[:2], want[:2])) and all(torch.equal(a.cpu(), b) for a, b in zip(dev[2:4], want[2:]))
        fin = torch.isfinite(mean)
        assert torch.equal(torch.isfinite(mean_dev.cpu()), fin)
        assert (mean_dev.cpu() - mean)[fin].abs().max().item() <= 140 * 2.0 ** -24 * (448 * want[2]).max().item()


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("lens,new,h,hk,d,bs,cols", [
    ([4300], 4200, 64, 1, 64, 128, 600),                        # a prompt: one chunk
    ([17500], 1100, 64, 1, 64, 128, 140),                       # four chunks, the last one short
    ([8000, 300], 1000, 32, 2, 128, 64, 2048),                  # the table holds far more than the sequences: later chunks empty
    ([40 + 7 * (i % 40) for i in range(300)], 4, 64, 4, 64, 64, 1000),   # few tokens a sequence: eight chunks, most of them empty
    ([9000 + i for i in range(5)] + [64] * 600, 2, 40, 1, 64, 128, 1000),
])
def test_calls_whose_chunks_are_limited(lens, new, h, hk, d, bs, cols, dtype):
    """So many rows that the partial results' limit decides the chunks: some rows against 64 bits, all against the same
    call with a bound of the lengths that gives other chunks (the same sums in another order: twice the tolerance)."""
    seqs = len(lens)
    g = torch.Generator().manual_seed(seqs + new)
    lens = [max(n, new) for n in lens] if seqs > 1 and new < 10 else lens
    kc, vc, ks, vs, table = build(7, lens, hk, d, bs)
    wide = torch.full((seqs, cols), -7, dtype=torch.int32)
    wide[:, :min(cols, table.shape[1])] = table[:, :cols]
    q = (2 * torch.randn(new * seqs, h, d, generator=g)).to(dtype)
    cu = (torch.arange(seqs + 1) * new).to(torch.int32).to(DEV)
    dev = put(kc, vc, ks, vs, wide)
    lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse = mt.kv8_attention(q.to(DEV), *dev, lengths, cu_seqlens=cu)
    other, lse2 = mt.kv8_attention(q.to(DEV), *dev, lengths, cu_seqlens=cu, max_length=1)
    u = torch.finfo(dtype).eps / 2
    top = (vc.nan_to_num() * vs[:, :, None, None]).abs().max().item()
    smax = (q.double().norm(dim=2).max() * (kc.nan_to_num() * ks[:, :, None, None]).double().norm(dim=3).max() / math.sqrt(d)).item()
    assert torch.isfinite(out[lengths.repeat_interleave(new) >= new]).all()
    assert (out.double() - other.double()).abs().max().item() <= 2 * 2.25 * u * top
    few = torch.isfinite(lse)
    assert torch.equal(few, torch.isfinite(lse2)) and (lse.double() - lse2.double())[few].abs().max().item() <= 2.0 ** -23 * (d + 64) * (smax + 10)
    rows = sorted({0, 1, new * seqs // 2, new * seqs - 1} | set(torch.randint(0, new * seqs, (20,), generator=g).tolist()))
    at = [r // new for r in rows]
    each = [lens[i] - new + r % new + 1 for i, r in zip(at, rows)]
    want, want_lse = oracle.cache_attention(q[rows], kc, vc, ks, vs, wide[at], [max(0, n) for n in each], bs)
    for r, n in zip(range(len(rows)), each):
        if n <= 0:
            want[r], want_lse[r] = 0.0, -math.inf
    assert (out[rows].cpu().double() - want).abs().max().item() <= 2.25 * u * top
    fin = torch.isfinite(want_lse)
    got = lse[rows].cpu().double()
    assert torch.equal(torch.isfinite(got), fin) and (got - want_lse)[fin].abs().max().item() <= 2.0 ** -24 * (d + 64) * (smax + 10)
