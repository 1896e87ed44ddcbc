"""GPU: how the attention operators are called: refusals, empty and many
sequences, streams, captured graphs, caches and tensors past 32-bit offsets.

Where two calls have to agree they do the same arithmetic and their results are
equal; against the 64-bit forms the tolerances are those of the other tests."""

import math

import pytest
import torch

import attention_oracle as oracle
import row_wise_top_topk_amd as mt
from test_gpu_block_attention import check_out, gpu, make
from test_gpu_kv8 import build, put, same

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F16 = torch.bfloat16, torch.float16


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype, device=DEV)


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


# ---- refusals ----

def test_block_attention_refuses():
    q, k, b = z(10, 4, 64), z(10, 2, 64), torch.zeros(10, 2, 1, dtype=torch.int32, device=DEV)
    good = dict(q=q, k=k, v=k, blocks=b, block_size=16)
    mt.block_attention(**good)
    base = z(12 * 4 * 64 + 8)
    for bad in (dict(q=q.float()), dict(q=q.half()), dict(q=q[:, :, :32]), dict(q=q[0]), dict(k=k[:, :1].expand(10, 3, 64), v=k[:, :1].expand(10, 3, 64)),
                dict(v=k[:9]), dict(k=k.half()), dict(k=k.cpu()), dict(q=base[1:10 * 4 * 64 + 1].view(10, 4, 64)),
                dict(q=z(10, 64, 4).transpose(1, 2)), dict(q=base[:10 * 260].as_strided((10, 4, 64), (252, 64, 1))), dict(q=z(10, 4, 32)),
                dict(blocks=b[:9]), dict(blocks=b.long()), dict(blocks=b.cpu()), dict(blocks=z(10, 2, 0, dtype=torch.int32)),
                dict(blocks=z(10, 2, 1025, dtype=torch.int32)), dict(blocks=z(10, 2, 2, dtype=torch.int32)[:, :, :1]), dict(block_size=8),
                dict(block_size=256), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf),
                dict(cu_seqlens_k=i32(0, 10)), dict(cu_seqlens=i32(0, 10).long()), dict(cu_seqlens=i32(0, 10).cpu()),
                dict(cu_seqlens=i32(0, 10), cu_seqlens_k=i32(0, 5, 10)), dict(q=q[:5], blocks=b[:5], cu_seqlens=i32(0, 5)),
                dict(out=z(10, 4, 64, dtype=F16)), dict(out=z(9, 4, 64)), dict(rest=z(10, 4, 128)[:, :, :64])):
        with pytest.raises(ValueError):
            mt.block_attention(**{**good, **bad})
        if not {"out", "rest"} & set(bad) and bad.get("q", q).is_floating_point():
            with pytest.raises(ValueError):
                args = {**good, **bad}
                args["q"] = args["q"].detach().requires_grad_()
                mt.block_attention(**args)
    with pytest.raises(ValueError):
        mt.block_attention(**{**good, "q": q.clone().requires_grad_()}, out=z(10, 4, 64))
    out, lse = mt.block_attention(**good)
    for bad in (dict(dout=q[:9]), dict(dout=q.half()), dict(out=out.half()), dict(lse=lse.double()), dict(lse=lse[:9]), dict(rest=out[:9])):
        with pytest.raises(ValueError):
            mt.block_attention_backward(**{**dict(dout=q, q=q, k=k, v=k, out=out, lse=lse, blocks=b, block_size=16), **bad})


def test_scores_and_means_refuse():
    q, k = z(10, 4, 64), z(10, 2, 64)
    with pytest.raises(ValueError):
        mt.block_means(k, 16, out=z(1, 2, 64))
    with pytest.raises(ValueError):
        mt.block_means(k, 16, cu_seqlens=i32())
    means = mt.block_means(k, 16)
    good = dict(q=q, means=means, block_size=16, max_blocks=1)
    mt.block_scores(**good)
    table = torch.zeros(10, 1, dtype=torch.int32, device=DEV)
    n = torch.ones(10, dtype=torch.int32, device=DEV)
    for bad in (dict(means=means.half()), dict(means=means[:0]), dict(means=means[:, :, :32]), dict(means=z(1, 3, 64, dtype=torch.float32)),
                dict(max_blocks=0), dict(max_blocks=1 << 22), dict(first=-1), dict(last=-1), dict(scale=0.0), dict(lengths=n),
                dict(block_table=table), dict(block_table=table, lengths=n[:9]), dict(block_table=table, lengths=n, max_blocks=2),
                dict(block_table=table[:9], lengths=n[:9]), dict(block_table=table, lengths=n, cu_seqlens_k=i32(0, 10)),
                dict(block_table=table, lengths=n, cu_seqlens=i32(0, 10)), dict(block_table=table.long(), lengths=n),
                dict(block_table=z(1, 10, dtype=torch.int32).t().expand(10, 2)[:, :1].t(), lengths=n)):
        with pytest.raises(ValueError):
            mt.block_scores(**{**good, **bad})


def test_cache_refuses():
    f8 = torch.float8_e4m3fn
    cache = torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device=DEV).view(f8)
    scale, table, lengths = z(4, 2, dtype=torch.float32), z(3, 2, dtype=torch.int32), i32(1, 2, 3)
    x = z(3, 2, 64)
    good = dict(k=x, v=x, k_cache=cache, v_cache=cache.clone(), k_scale=scale, v_scale=scale.clone(), block_table=table, lengths=lengths)
    common = (dict(k_cache=cache.view(torch.uint8)), dict(v_cache=cache[:3]), dict(k_cache=cache.transpose(0, 1)), dict(k_scale=scale[:3]),
              dict(v_scale=scale.half()), dict(lengths=lengths.long()), dict(lengths=lengths[:2]), dict(block_table=table.long()),
              dict(block_table=table[:2]), dict(block_table=z(2, 3, dtype=torch.int32).t()), dict(cu_seqlens=i32(0, 3)),
              dict(cu_seqlens=i32(0, 1, 2, 3).long()), dict(k_scale=scale.cpu()))
    for bad in common + (dict(k=x[:2]), dict(k=x.half()), dict(k=z(3, 1, 64), v=z(3, 1, 64)), dict(k=z(3, 2, 128), v=z(3, 2, 128)),
                         dict(k=x[:2], v=x[:2]), dict(k_mean=z(4, 2, 64)), dict(k_mean=z(3, 2, 64, dtype=torch.float32))):
        with pytest.raises(ValueError):
            mt.kv8_append(**{**good, **bad})
    good = {n: t for n, t in good.items() if n not in ("k", "v")}
    good["q"] = z(3, 4, 64)
    mt.kv8_attention(**good)
    blocks = z(3, 2, 1, dtype=torch.int32)
    for bad in common + (dict(q=z(3, 3, 64)), dict(q=z(2, 4, 64)), dict(q=z(3, 4, 128)), dict(q=z(3, 4, 64, dtype=torch.float32)),
                         dict(blocks=blocks[:2]), dict(blocks=blocks.long()), dict(blocks=z(3, 2, 0, dtype=torch.int32)), dict(max_length=-1),
                         dict(scale=0.0), dict(out=z(3, 4, 128)), dict(block_table=table[:, :1].expand(3, 1 << 26))):
        with pytest.raises(ValueError):
            mt.kv8_attention(**{**good, **bad})


# ---- nothing, and many ----

@pytest.mark.parametrize("dtype", [BF, F16])
def test_nothing(dtype):
    """No tokens, no keys, no sequences, no pages."""
    b = lambda t: torch.zeros(t, 2, 3, dtype=torch.int32, device=DEV)  # noqa: E731
    for t, tk, cu, cu_k in ((0, 0, None, None), (0, 0, i32(0), i32(0)), (5, 5, i32(0), i32(0)), (0, 40, i32(0, 0), i32(0, 40)),
                            (7, 0, i32(0, 7), i32(0, 0)), (7, 0, None, None), (7, 9, i32(0, 0, 0), i32(0, 9, 9))):
        q, k, v = (torch.randn(n, h, 64, device=DEV).to(dtype).requires_grad_() for n, h in ((t, 4), (tk, 2), (tk, 2)))
        out, lse = mt.block_attention(q, k, v, b(t), 16, cu_seqlens=cu, cu_seqlens_k=cu_k)
        assert out.shape == q.shape and (out == 0).all() and (lse == -math.inf).all()
        for g in torch.autograd.grad(out, (q, k, v), torch.ones_like(out)):
            assert (g == 0).all()
        means = mt.block_means(k.detach(), 16, cu_seqlens=cu_k)
        assert means.shape[0] == tk // 16 + (1 if cu_k is None else cu_k.numel() - 1)
        if t == tk or cu is not None:
            scores, counts = mt.block_scores(q.detach(), means, 16, 3, cu_seqlens=cu, cu_seqlens_k=cu_k)
            if cu is not None:
                assert (scores == -math.inf).all() and (counts == 0).all()
    f8 = torch.float8_e4m3fn
    for pages, cols, n in ((0, 2, 3), (4, 0, 3), (4, 2, 0)):
        cache = torch.zeros(pages, 2, 16, 64, dtype=torch.uint8, device=DEV).view(f8)
        scale = torch.ones(pages, 2, device=DEV)
        table, lengths = torch.zeros(n, cols, dtype=torch.int32, device=DEV), torch.ones(n, dtype=torch.int32, device=DEV)
        x = torch.randn(n, 2, 64, device=DEV).to(dtype)
        before = cache.clone().view(torch.uint8)
        mt.kv8_append(x, x, cache, cache.clone(), scale, scale.clone(), table, lengths)
        assert torch.equal(cache.view(torch.uint8), before)
        out, lse = mt.kv8_attention(torch.randn(n, 4, 64, device=DEV).to(dtype), cache, cache, scale, scale, table, lengths)
        assert (out == 0).all() and (lse == -math.inf).all()
    # lengths of 0 and less
    cache = torch.full((4, 2, 16, 64), 0x7f, dtype=torch.uint8, device=DEV).view(f8)
    scale = torch.ones(4, 2, device=DEV)
    table = torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    out, lse = mt.kv8_attention(torch.randn(3, 4, 64, device=DEV).to(dtype), cache, cache, scale, scale, table, i32(0, -5, -(1 << 31)))
    assert (out == 0).all() and (lse == -math.inf).all()
    mt.kv8_append(torch.randn(3, 2, 64, device=DEV).to(dtype), torch.randn(3, 2, 64, device=DEV).to(dtype), cache, cache, scale, scale, table, i32(0, -5, -(1 << 31)))
    assert (cache.view(torch.uint8) == 0x7f).all()


def test_rows_without_keys_among_others():
    """Selections of nothing, more queries than keys: out 0, lse -inf, no gradient, whatever q and dout hold there."""
    q, k, v, blocks, cu_q, cu_k = make(4, [50, 20], [30, 20], 4, 2, 64, 16, 2, BF)
    blocks[55] = -1
    blocks[60, 0] = 99
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(0)).to(BF)
    _, _, *want, sizes = oracle.attention(q, k, v, blocks, 16, cu_q, cu_k, dout=dout)
    q[:20] = math.nan
    dout[55], q[55] = math.inf, math.nan
    leaves = [x.to(DEV).requires_grad_() for x in (q, k, v)]
    out, lse = mt.block_attention(*leaves, blocks.to(DEV), 16, cu_seqlens=cu_q.to(DEV), cu_seqlens_k=cu_k.to(DEV))
    empty = [*range(20), 55]
    assert (out[empty] == 0).all() and (lse[empty] == -math.inf).all() and (out[60, :2] == 0).all()
    got = torch.autograd.grad(out, leaves, dout.to(DEV))
    assert (got[0][empty] == 0).all()
    for g, w, s in zip(got, want, sizes):
        assert ((g.cpu().double() - w).abs() <= 1.25 * 2.0 ** -8 * (s + w.abs()) + 1e-30).all()


@pytest.mark.parametrize("count", [63, 64, 65, 200])
def test_many_sequences(count):
    """More sequences than a wavefront looks at in one step, empty ones among them."""
    g = torch.Generator().manual_seed(count)
    lens = torch.randint(0, 9, (count,), generator=g).tolist()
    lens[3], lens[-1] = 130, 40
    q, k, v, blocks, cu, _ = make(6, lens, lens, 4, 2, 64, 16, 2, BF, tail=3)
    want, want_lse, wq, wk, wv, sizes = oracle.attention(q, k, v, blocks, 16, cu, cu, dout=torch.ones(q.shape))
    leaves = [x.to(DEV).requires_grad_() for x in (q, k, v)]
    cu_dev = cu.to(DEV)
    out, lse = mt.block_attention(*leaves, blocks.to(DEV), 16, cu_seqlens=cu_dev)
    check_out(out.detach(), want, lse, want_lse, v, 40, 64, BF)
    for got, w, s in zip(torch.autograd.grad(out.float().sum(), leaves), (wq, wk, wv), sizes):
        assert ((got.cpu().double() - w).abs() <= 1.25 * 2.0 ** -8 * (s + w.abs()) + 1e-30).all()
    means = mt.block_means(k.to(DEV), 16, cu_seqlens=cu_dev)
    m = oracle.means(k, 16, cu)
    assert (means.cpu().double() - m).abs().max().item() <= 130 * 2.0 ** -24 * k.abs().double().max().item()
    got, counts = mt.block_scores(q.to(DEV), means, 16, 9, cu_seqlens=cu_dev)
    placed = [(int(cu[i]) + r, i, r) for i in range(count) for r in range(lens[i])]
    want, want_counts = oracle.scores(q, lambda i, b: m[int(cu[i]) // 16 + i + b], 16, 9, placed, 2, 1, 1)
    assert torch.equal(counts.cpu(), want_counts)
    fin = torch.isfinite(want)
    assert torch.equal(got.cpu()[~fin].double(), want[~fin])
    size = (q.double().norm(dim=2).max() * m.norm(dim=2).max() / 8).item()
    assert (got.cpu().double() - want)[fin].abs().max().item() <= 200 * 2.0 ** -23 * size + 130 * 2.0 ** -24 * size
    # the cache: each sequence's last tokens
    have = [n + 5 for n in lens]
    kc, vc, ks, vs, table = build(2, have, 2, 64, 16)
    dev = put(kc, vc, ks, vs, table)
    lengths = torch.tensor(have, dtype=torch.int32, device=DEV)
    mt.kv8_append(k.to(DEV), v.to(DEV), *dev, lengths, cu_seqlens=cu_dev)
    oracle.append(k, v, kc, vc, ks, vs, table, have, 16, cu)
    assert torch.equal(dev[2].cpu(), ks) and same(dev[0], kc) and same(dev[1], vc)
    want, _ = oracle.cache_attention(q, kc, vc, ks, vs, table, have, 16, cu)
    out, _ = mt.kv8_attention(q.to(DEV), *dev, lengths, cu_seqlens=cu_dev)
    top = (vc.nan_to_num() * vs[:, :, None, None]).abs().max().item()
    assert (out.cpu().double() - want).abs().max().item() <= 2.25 * 2.0 ** -8 * top


def test_scales_that_are_no_powers_of_two():
    """A cache that came from elsewhere: its scale grows to the next power of two at least."""
    g = torch.Generator().manual_seed(1)
    for size in (0.001, 1000.0):
        kc, vc, ks, vs, table = build(1, [21], 2, 64, 16)
        ks, vs = ks * 1.25, vs * 1.5                          # few bits: the products are exact
        dev = put(kc, vc, ks, vs, table)
        k, v = ((size * torch.randn(1, 2, 64, generator=g)).to(BF) for _ in range(2))
        mt.kv8_append(k.to(DEV), v.to(DEV), *dev, i32(21))
        page = int(table[0, 1])
        for x, cache, scale, got, got_scale in ((k, kc, ks, dev[0], dev[2]), (v, vc, vs, dev[1], dev[3])):
            for c in range(2):
                old = float(scale[page, c])
                s = max(oracle.scale_for(x[0, c].abs().max().item()), 2.0 ** math.ceil(math.log2(old)))
                cache[page, c, :4] = oracle.round8(cache[page, c, :4].double() * old / s)
                cache[page, c, 4] = oracle.round8(x[0, c].double() / s)
                scale[page, c] = s
            assert torch.equal(got_scale.cpu(), scale) and same(got, cache)


# ---- streams and graphs ----

def prompt_run(q, k, v, cu, top):
    means = mt.block_means(k, 16, cu_seqlens=cu)
    scores, counts = mt.block_scores(q, means, 16, 20, cu_seqlens=cu)
    blocks = mt.topk_indices(scores.flatten(0, 1), counts.flatten(), top).view(q.shape[0], k.shape[1], top)
    return mt.block_attention(q, k, v, blocks, 16, cu_seqlens=cu), blocks


def test_other_streams():
    q, k, v, _, cu, _ = make(3, [300, 77], [300, 77], 8, 2, 64, 16, 1, BF)
    q, k, v, cu = gpu(q, k, v, cu)
    (want, want_lse), blocks = prompt_run(q, k, v, cu, 4)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    grads = torch.autograd.grad(mt.block_attention(*leaves, blocks, 16, cu_seqlens=cu)[0], leaves, torch.ones_like(q))
    streams = [torch.cuda.Stream() for _ in range(3)]
    results = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            (out, lse), _ = prompt_run(q, k, v, cu, 4)
            mine = [x.clone().requires_grad_() for x in (q, k, v)]
            got = torch.autograd.grad(mt.block_attention(*mine, blocks, 16, cu_seqlens=cu)[0], mine, torch.ones_like(q))
        results.append((out, lse, got))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for out, lse, got in results:
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert all(torch.equal(a, b) for a, b in zip(got, grads))


def capture(fn):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            fn()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fn()
    return graph, out


def test_graphs_of_a_prompt_and_a_training_step():
    """Two captured graphs, replayed in turn with eager work and other inputs between the replays."""
    g = torch.Generator().manual_seed(5)
    q, k, v, _, cu, _ = make(3, [300, 77], [300, 77], 8, 2, 64, 16, 1, BF)
    q, k, v, cu = gpu(q, k, v, cu)
    dout = torch.randn(q.shape, generator=g).to(BF).to(DEV)
    blocks = prompt_run(q, k, v, cu, 4)[1].clone()
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]

    def train():
        return torch.autograd.grad(mt.block_attention(*leaves, blocks, 16, cu_seqlens=cu)[0], leaves, dout)

    def explicit():
        rest = torch.empty_like(q)
        out, lse = mt.block_attention(q, k, v, blocks, 16, cu_seqlens=cu, rest=rest)
        return mt.block_attention_backward(dout, q, k, v, out, lse, blocks, 16, cu_seqlens=cu, rest=rest)

    g1, (o1, b1) = capture(lambda: prompt_run(q, k, v, cu, 4))
    g2, o2 = capture(train)
    alive = mt.block_attention(*leaves, blocks, 16, cu_seqlens=cu)[0]        # an eager graph that lives on
    q.requires_grad_()
    too = mt.block_attention(q, k, v, blocks, 16, cu_seqlens=cu)[0]
    q.requires_grad_(False)
    g3, o3 = capture(explicit)
    for seed in range(4):
        g.manual_seed(seed)
        new = [torch.randn(x.shape, generator=g).to(BF).to(DEV) for x in (q, k, v)]
        new_dout = torch.randn(q.shape, generator=g).to(BF).to(DEV)
        del alive, too
        with torch.no_grad():
            for x, leaf, y in zip((q, k, v), leaves, new):
                x.copy_(y)
                leaf.copy_(y)
            dout.copy_(new_dout)
        g1.replay()
        (out, lse), picked = prompt_run(*new, cu, 4)
        assert torch.equal(b1, picked) and torch.equal(o1[0], out) and torch.equal(o1[1], lse)
        g2.replay()
        g1.replay()
        g3.replay()
        fresh = [x.clone().requires_grad_() for x in new]
        alive = mt.block_attention(*fresh, blocks, 16, cu_seqlens=cu)[0]
        too = torch.autograd.grad(alive, fresh, new_dout)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o2, too))
        assert all(torch.equal(a, b) for a, b in zip(o3, too))
        assert torch.equal(o1[0], out)


def test_capture_refuses_leaves_of_living_graphs():
    """The refusal comes before the gradient's machinery sees the capture; afterwards all works."""
    q, k, v, blocks, _, _ = make(3, [40], [40], 4, 2, 64, 16, 2, BF)
    blocks = blocks.to(DEV)
    leaves = [x.to(DEV).requires_grad_() for x in (q, k, v)]
    alive = mt.block_attention(*leaves, blocks, 16)[0]
    graph = torch.cuda.CUDAGraph()
    x = torch.zeros(4, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        x.add_(1)
        with pytest.raises(RuntimeError, match="captured"):
            mt.block_attention(*leaves, blocks, 16)
    graph.replay()
    assert (x == 1).all()
    want = torch.autograd.grad(alive, leaves, torch.ones_like(alive))
    del alive
    graph, got = capture(lambda: torch.autograd.grad(mt.block_attention(*leaves, blocks, 16)[0], leaves, torch.ones_like(leaves[0])))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graphs_of_decode_steps():
    """A captured serving step, its lengths rising from replay to replay, against the same steps run eagerly."""
    g = torch.Generator().manual_seed(3)
    lens = [100, 37, 250]
    kc, vc, ks, vs, table = build(8, [n + 40 for n in lens], 2, 128, 16)
    one, two = put(kc, vc, ks, vs, table), put(kc, vc, ks, vs, table)
    means = [torch.zeros(kc.shape[0], 2, 128, device=DEV) for _ in range(2)]
    q = torch.randn(3, 8, 128, generator=g).to(F16).to(DEV)
    k, v = (torch.randn(3, 2, 128, generator=g).to(F16).to(DEV) for _ in range(2))
    lengths = [torch.tensor(lens, dtype=torch.int32, device=DEV) for _ in range(2)]

    def step(dev, mean, n):
        n.add_(1)
        mt.kv8_append(k, v, *dev, n, k_mean=mean)
        scores, counts = mt.block_scores(q, mean, 16, table.shape[1], lengths=n, block_table=dev[4])
        blocks = mt.topk_indices(scores.flatten(0, 1), counts.flatten(), 4).view(3, 2, 4)
        some = mt.kv8_attention(q, *dev, n, blocks=blocks)
        return *some, *mt.kv8_attention(q, *dev, n)

    graph, out = capture(lambda: step(one, means[0], lengths[0]))
    other, out2 = capture(lambda: mt.kv8_attention(q, *one, lengths[0]))
    for _ in range(2):                                  # the capture's own eager runs
        step(two, means[1], lengths[1])
    for i in range(5):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g).to(F16))
        graph.replay()
        other.replay()
        want = step(two, means[1], lengths[1])
        torch.cuda.synchronize()
        assert torch.equal(lengths[0], lengths[1])
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
        assert all(torch.equal(a, b) for a, b in zip(out2, want[2:])), i
        assert all(same(a.float(), b.float().cpu()) for a, b in zip(one[:4], two[:4]))


# ---- past 32 bits ----

@pytest.mark.parametrize("dtype", [BF, F16])
def test_cache_past_4_gib(dtype):
    pages, bs, d = (1 << 32) // (128 * 128) + 40, 128, 128
    lens = [1500, 129]
    kc, vc, ks, vs, table = build(5, lens, 1, d, bs, spare=0)
    at = (pages - 1 - torch.arange(kc.shape[0])).to(torch.int32)
    at[::2] -= pages // 2                                        # some behind, some before the border
    f8 = torch.float8_e4m3fn
    k_big, v_big = (torch.empty(pages, 1, bs, d, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks_big, vs_big = (torch.ones(pages, 1, device=DEV) for _ in range(2))
    where = at.long().to(DEV)
    k_big[where], v_big[where] = (x.to(f8).view(torch.uint8).to(DEV) for x in (kc, vc))
    ks_big[where], vs_big[where] = ks.to(DEV), vs.to(DEV)
    big = torch.where(table >= 0, at[table.long().clamp(min=0)], table).to(DEV)
    dev = (k_big.view(f8), v_big.view(f8), ks_big, vs_big, big)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(2, 1, d, generator=g).to(dtype) for _ in range(2))
    q = torch.randn(2, 8, d, generator=g).to(dtype)
    lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
    mean = torch.zeros(pages, 1, d, device=DEV)
    mt.kv8_append(k.to(DEV), v.to(DEV), *dev, lengths, k_mean=mean)
    oracle.append(k, v, kc, vc, ks, vs, table, lens, bs)
    assert same(k_big[where].view(f8), kc) and same(v_big[where].view(f8), vc) and torch.equal(ks_big[where].cpu(), ks)
    want, _ = oracle.cache_attention(q, kc, vc, ks, vs, table, lens, bs)
    out, _ = mt.kv8_attention(q.to(DEV), *dev, lengths)
    top = (vc.nan_to_num() * vs[:, :, None, None]).abs().max().item()
    assert (out.cpu().double() - want).abs().max().item() <= 2.25 * torch.finfo(dtype).eps / 2 * top


def test_strides_past_4_gib():
    """Rows of q, k, v and dout that lie 16 MiB apart, 300 of them."""
    t, step = 300, (1 << 23) - 8
    q, k, v, blocks, _, _ = make(9, [t], [t], 2, 1, 64, 16, 3, BF)
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(0)).to(BF)
    store = torch.empty(t * step, dtype=BF, device=DEV)
    views, at = [], 0
    for x in (q, k, v, dout):
        h = x.shape[1]
        view = store[at:].as_strided((t, h, 64), (step, 64, 1))
        view.copy_(x)
        views.append(view)
        at += h * 64
    want = mt.block_attention(*gpu(q, k, v, blocks), 16, rest=(rest := torch.empty(q.shape, dtype=BF, device=DEV)))
    other = torch.empty_like(rest)
    got = mt.block_attention(*views[:3], blocks.to(DEV), 16, rest=other)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]) and torch.equal(rest, other)
    a = mt.block_attention_backward(dout.to(DEV), *gpu(q, k, v), *want, blocks.to(DEV), 16, rest=rest)
    b = mt.block_attention_backward(views[3], *views[:3], *got, blocks.to(DEV), 16, rest=other)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.equal(mt.block_means(views[1], 16), mt.block_means(k.to(DEV), 16))


def test_scores_past_4_gib():
    t, nb = 17000, 1 << 16
    g = torch.Generator().manual_seed(1)
    q = torch.randn(t, 1, 64, generator=g).to(BF).to(DEV)
    k = torch.randn(t, 1, 64, generator=g).to(BF).to(DEV)
    means = mt.block_means(k, 16)
    big, counts = mt.block_scores(q, means, 16, nb)
    small, counts2 = mt.block_scores(q, means, 16, 1063)
    assert big.numel() * 4 > 1 << 32 and torch.equal(counts, counts2)
    assert torch.equal(big[:, :, :1063], small)
    assert (big[::97, :, 1063:] == -math.inf).all() and (big[-50:, :, 1063:] == -math.inf).all()


def test_padded_batch():
    """A decode batch filled up with requests of length 0, whose table rows hold anything."""
    g = torch.Generator().manual_seed(6)
    lens = [40, 0, 7, 0]
    kc, vc, ks, vs, table = build(2, [40, 1, 7, 1], 2, 64, 16)
    table[1], table[3] = torch.tensor([5, 1 << 30, -9]), torch.tensor([0, 1, 2])
    dev = put(kc, vc, ks, vs, table)
    lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
    mean = torch.zeros(kc.shape[0], 2, 64, device=DEV)
    q = torch.randn(4, 8, 64, generator=g).to(BF)
    k, v = (torch.randn(4, 2, 64, generator=g).to(BF) for _ in range(2))
    q[1], k[3], v[1] = math.nan, math.inf, math.nan
    mt.kv8_append(k.to(DEV), v.to(DEV), *dev, lengths, k_mean=mean)
    oracle.append(k, v, kc, vc, ks, vs, table, lens, 16)
    assert same(dev[0], kc) and same(dev[1], vc) and torch.equal(dev[2].cpu(), ks)
    mean[:] = torch.randn(mean.shape, generator=g).to(DEV)
    scores, counts = mt.block_scores(q.to(DEV), mean, 16, 3, lengths=lengths, block_table=dev[4])
    assert counts[:, 0].tolist() == [3, 0, 1, 0] and (scores[[1, 3]] == -math.inf).all()
    blocks = mt.topk_indices(scores.flatten(0, 1), counts.flatten(), 2).view(4, 2, 2)
    assert (blocks[[1, 3]] == -1).all()
    for b in (None, blocks):
        out, lse = mt.kv8_attention(q.to(DEV), *dev, lengths, blocks=b)
        want, want_lse = oracle.cache_attention(q, kc, vc, ks, vs, table, lens, 16, None, None if b is None else b.cpu())
        assert (out[[1, 3]] == 0).all() and (lse[[1, 3]] == -math.inf).all()
        top = (vc.nan_to_num() * vs[:, :, None, None]).abs().max().item()
        assert (out.cpu().double() - want).abs().max().item() <= 2.25 * 2.0 ** -8 * top


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, do not disturb each other."""
    lens = [3000, 2000]
    kc, vc, ks, vs, table = build(7, lens, 2, 128, 16)
    dev = put(kc, vc, ks, vs, table)
    lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(9)
    qs = [torch.randn(2, 8, 128, generator=g).to(BF).to(DEV) for _ in range(8)]
    want = [mt.kv8_attention(q, *dev, lengths)[0] for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [None] * 8
    for i, q in enumerate(qs):
        with torch.cuda.stream(streams[i % 2]):
            got[i] = mt.kv8_attention(q, *dev, lengths)[0]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
