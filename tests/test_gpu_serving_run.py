"""GPU: the serving operators together with the selection and the 8-bit cache, as a
serving loop uses them; captured graphs, streams, calls at once."""

import math

import pytest
import torch

import row_wise_top_topk_amd as mt

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F8 = torch.float8_e4m3fn
HK, D, BS, HEADS = 2, 64, 16, 6


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def codes(t):
    return t.view(torch.uint8)


class Cache:
    """One layer's cache and its means."""

    def __init__(self, pages):
        self.k, self.v = (torch.zeros(pages, HK, BS, D, device=DEV).to(F8) for _ in range(2))
        self.ks, self.vs = (torch.ones(pages, HK, device=DEV) for _ in range(2))
        self.mean = torch.zeros(pages, HK, D, device=DEV)

    def parts(self):
        return self.k, self.v, self.ks, self.vs

    def held(self, table, length, row):
        """What the row's tokens are in the cache: codes and scales of its pages."""
        n = int(length[row])
        out = []
        for j, page in enumerate(table[row, :-(-n // BS)].tolist()):
            e = min(BS, n - j * BS)
            out += [codes(self.k)[page, :, :e], codes(self.v)[page, :, :e], self.ks[page], self.vs[page], self.mean[page]]
        return [t.clone() for t in out]


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def tokens(g, n, heads):
    return torch.randn(n, heads, D, generator=g, device=DEV).to(torch.bfloat16)


def test_prompts_in_chunks_beams_and_requests_that_end():
    """Two layers over one table; beside them a twin without sharing, whose rows own
    fixed pages and are copied whole where the first one forks.  All rows read the
    same codes, scales and means, and attention over both gives the same bits."""
    g = torch.Generator(device=DEV).manual_seed(3)
    rows, cols, pages, vocab = 4, 12, 40, 5000
    table, lengths, refs = torch.full((rows, cols), -1, dtype=torch.int32, device=DEV), ints([0] * rows), ints([0] * pages)
    layers = [Cache(pages) for _ in range(2)]
    twin_table = torch.arange(rows * cols, dtype=torch.int32, device=DEV).view(rows, cols)
    twins = [Cache(rows * cols) for _ in range(2)]
    said = torch.full((rows, cols * BS), -1, dtype=torch.int32, device=DEV)

    def check():
        for a, b in zip(layers, twins):
            for r in range(rows):
                assert same(a.held(table, lengths, r), b.held(twin_table, lengths, r))
        used = [p for r in range(rows) for p in table[r, :-(-int(lengths[r]) // BS)].tolist()]
        assert refs.tolist() == [used.count(p) for p in range(pages)]

    def read(new):
        cu = ints([0] + [sum(new[:i + 1]) for i in range(rows)])
        assert mt.pages_grow(table, lengths, refs, ints(new), BS).tolist() == new
        for a, b in zip(layers, twins):
            q, k, v = tokens(g, sum(new), HEADS), tokens(g, sum(new), HK), tokens(g, sum(new), HK)
            out = mt.chunk_attention(q, k, v, *a.parts(), table, lengths, cu_seqlens=cu)
            twin = mt.chunk_attention(q, k, v, *b.parts(), twin_table, lengths, cu_seqlens=cu)
            assert same(out, twin) and torch.isfinite(out[0]).all()
            mt.kv8_append(k, v, *a.parts(), table, lengths, cu_seqlens=cu, k_mean=a.mean)
            mt.kv8_append(k, v, *b.parts(), twin_table, lengths, cu_seqlens=cu, k_mean=b.mean)
            # a second time behind the append: the chunk's own rows come from k and v
            assert same(out, mt.chunk_attention(q, k, v, *a.parts(), table, lengths, cu_seqlens=cu))
        check()

    def fork(parents):
        before = lengths.tolist()
        copies = mt.pages_fork(table, lengths, refs, ints(parents), BS)
        for a in layers:
            mt.pages_copy(*a.parts(), copies, k_mean=a.mean)
        for b in twins:
            old = [t.clone() for t in (codes(b.k), codes(b.v), b.ks, b.vs, b.mean)]
            for r, p in enumerate(parents):
                if 0 <= p < rows:
                    for new, t in zip((codes(b.k), codes(b.v), b.ks, b.vs, b.mean), old):
                        new[r * cols:(r + 1) * cols] = t[p * cols:(p + 1) * cols]
        assert lengths.tolist() == [before[p] if 0 <= p < rows else 0 for p in parents]
        check()

    read([70, 0, 37, 0])            # two prompts, in chunks
    read([25, 0, 1, 0])
    fork([0, 0, 2, 0])              # three samples of the first one
    for step in range(6):
        read([1, 1, 1, 1])          # a decode step's tokens go the same way
        at = lengths.long()
        q = tokens(g, rows, HEADS)
        outs = [mt.kv8_attention(q, *a.parts(), t, lengths, max_length=cols * BS)
                for a, t in ((layers[0], table), (twins[0], twin_table))]
        assert same(*outs)
        logits = (outs[0][0].reshape(rows, -1).float() @ torch.randn(HEADS * D, vocab, generator=g, device=DEV)).to(torch.bfloat16)
        said.scatter_(1, at[:, None] - 1, torch.randint(0, vocab, (rows, 1), generator=g, device=DEV).to(torch.int32))
        scores = mt.penalize_logits(logits, said, lengths, repetition=torch.full((rows,), 1.2, device=DEV))
        best = mt.topk_indices(scores, ints([vocab] * rows), 2, order="value")
        assert torch.equal(scores.gather(1, best[:, :1].long())[:, 0], scores.amax(1))
        total = scores.gather(1, best.long())
        parents = (total[[0, 1, 3]].flatten().topk(3)[1] // 2).tolist()   # a beam step of the three samples
        parents = [[0, 1, 3][p] for p in parents]
        fork([parents[0], parents[1], 2, parents[2]])
        if step == 2:
            copies = mt.pages_compact(table, lengths, refs, BS)
            for a in layers:
                mt.pages_copy(*a.parts(), copies, k_mean=a.mean)
            check()
            live = int((refs > 0).sum())
            assert (refs[:live] > 0).all()
    fork([-1, 1, 2, -1])            # requests end
    read([30, 0, 5, 64])            # others take their place
    assert mt.pages_grow(table, lengths, refs, ints([0, 0, 0, 10 ** 6]), BS).tolist() == [0, 0, 0, 0]
    fork([-1] * rows)
    assert refs.tolist() == [0] * pages


def chunk_inputs(seed, lens, new, dtype=torch.bfloat16, pages=60):
    g = torch.Generator(device=DEV).manual_seed(seed)
    cols = 20
    table = torch.randperm(pages, generator=g, device=DEV)[:len(lens) * cols].view(len(lens), cols).to(torch.int32)
    a = Cache(pages)
    a.k, a.v = (torch.randn(pages, HK, BS, D, generator=g, device=DEV).to(F8) for _ in range(2))
    t = sum(new)
    q, k, v = (torch.randn(t, h, D, generator=g, device=DEV).to(dtype) for h in (HEADS, HK, HK))
    return [q, k, v, *a.parts(), table, ints(lens)], ints([0] + [sum(new[:i + 1]) for i in range(len(new))])


def test_captured_chunk():
    args, cu = chunk_inputs(1, [300, 77], [40, 3])
    for _ in range(2):
        mt.chunk_attention(*args, cu_seqlens=cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = mt.chunk_attention(*args, cu_seqlens=cu)
    for i in range(4):   # other contents, lengths and cuts, the same launch
        other, _ = chunk_inputs(10 + i, [300 - 50 * i, 77 + 30 * i], [40, 3])
        for a, b in zip(args, other):
            a.copy_(b)
        cu.copy_(ints([0, 43 - i, 43]))
        graph.replay()
        want = mt.chunk_attention(*other, cu_seqlens=cu)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("big", [False, True])
def test_captured_pages(big):
    pages = 20000 if big else 60
    table, lengths, refs = torch.full((4, 9), -1, dtype=torch.int32, device=DEV), ints([0] * 4), ints([0] * pages)
    grow, parents = ints([0] * 4), ints([0, 1, 2, 3])
    a = Cache(60)
    twin = [t.clone() for t in (table, lengths, refs)]
    twin_a = Cache(60)

    def step(table, lengths, refs, a):
        grown = mt.pages_grow(table, lengths, refs, grow, BS)
        copies = mt.pages_fork(table, lengths, refs, parents, BS)
        mt.pages_copy(*a.parts(), copies, k_mean=a.mean)
        moves = mt.pages_compact(table, lengths, refs, BS)
        mt.pages_copy(*a.parts(), moves, k_mean=a.mean)
        return grown, copies, moves

    step(table, lengths, refs, a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(table, lengths, refs, a)
    g = torch.Generator().manual_seed(1)
    for i in range(6):
        grow.copy_(torch.randint(0, 40, (4,), generator=g))
        parents.copy_(torch.randint(-1, 4, (4,), generator=g))
        graph.replay()
        want = step(*twin, twin_a)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert all(torch.equal(x, y) for x, y in zip((table, lengths, refs), twin))
        assert all(torch.equal(codes(x) if x.dtype == F8 else x, codes(y) if y.dtype == F8 else y) for x, y in zip(a.parts(), twin_a.parts()))


def test_captured_logits():
    g = torch.Generator(device=DEV).manual_seed(1)
    logits, tokens_ = torch.randn(5, 4001, generator=g, device=DEV), torch.randint(0, 4001, (5, 70), generator=g, device=DEV).to(torch.int32)
    lengths, r = ints([70, 0, 5, 69, 33]), torch.rand(5, generator=g, device=DEV) + 0.5
    call = lambda: mt.penalize_logits(logits, tokens_, lengths, repetition=r, frequency=r)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(4):
        logits.normal_(generator=g)
        lengths.copy_(ints([3 * i, 70, 0, 1, 10]))
        graph.replay()
        want = call()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_two_graphs_and_two_streams_at_once():
    # each call has a workspace of its own: walks split over both, replayed and enqueued together
    a, cu_a = chunk_inputs(1, [310, 200], [4, 2])
    b, cu_b = chunk_inputs(2, [290, 310], [2, 5])
    want = [mt.chunk_attention(*a, cu_seqlens=cu_a), mt.chunk_attention(*b, cu_seqlens=cu_b)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for args, cu in ((a, cu_a), (b, cu_b)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(mt.chunk_attention(*args, cu_seqlens=cu))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        eager = []
        for (args, cu), stream in zip(((a, cu_a), (b, cu_b)), streams):
            with torch.cuda.stream(stream):
                eager.append(mt.chunk_attention(*args, cu_seqlens=cu))
        torch.cuda.synchronize()
        for got in (outs, eager):
            assert all(torch.equal(x, y) for p, q in zip(got, want) for x, y in zip(p, q))


def test_on_a_stream_of_its_own():
    side = torch.cuda.Stream()
    args, cu = chunk_inputs(5, [100, 250], [30, 30])
    want = mt.chunk_attention(*args, cu_seqlens=cu)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        late = torch.zeros_like(args[0])
        for _ in range(20):      # q is there only after this stream's work
            late.add_(args[0] / 20)
        late.copy_(args[0])
        got = mt.chunk_attention(late, *args[1:], cu_seqlens=cu)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_caches_past_4_gib():
    # pages whose codes lie behind 2^32 bytes
    pages = (1 << 32) // (HK * BS * D) + 40
    a = Cache.__new__(Cache)
    a.k, a.v = (torch.zeros(pages, HK, BS, D, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2))
    a.ks, a.vs = (torch.ones(pages, HK, device=DEV) for _ in range(2))
    small, cu = chunk_inputs(4, [300, 310], [7, 20], pages=40)
    table = torch.arange(40, dtype=torch.int32, device=DEV).view(2, 20)
    high = table + (pages - 40)
    small[7] = table
    for x, y in zip(a.parts(), small[3:7]):
        (codes(x) if x.dtype == F8 else x)[pages - 40:] = (codes(y) if y.dtype == F8 else y)[:40]
    want = mt.chunk_attention(*small, cu_seqlens=cu)
    got = mt.chunk_attention(*small[:3], *a.parts(), high, small[8], cu_seqlens=cu)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    mt.pages_copy(*a.parts(), torch.stack([high.flatten(), table.flatten()], 1).contiguous())
    got = mt.chunk_attention(*small[:3], *a.parts(), table, small[8], cu_seqlens=cu)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_heads_and_rows_past_32_bits():
    # tokens 2^22 elements apart: offsets pass 2^31 elements
    n, apart = 700, 1 << 22
    buf = torch.zeros(n * apart, dtype=torch.bfloat16, device=DEV)
    args, cu = chunk_inputs(6, [700 + 90], [700])
    args[7] = args[7][:, :20]
    want = mt.chunk_attention(*args, cu_seqlens=cu)
    wide = buf.as_strided((n, HK, D), (apart, D, 1))
    wide.copy_(args[1])
    got = mt.chunk_attention(args[0], wide, *args[2:], cu_seqlens=cu)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_many_sequences():
    # more sequences than a wavefront looks at together, with empty ones
    lens = [(37 * i) % 90 + 3 for i in range(300)]
    new = [(11 * i) % 4 for i in range(300)]
    g = torch.Generator(device=DEV).manual_seed(8)
    table, lengths, refs = torch.full((300, 6), -1, dtype=torch.int32, device=DEV), ints([0] * 300), ints([0] * 2000)
    assert mt.pages_grow(table, lengths, refs, ints(lens), BS).tolist() == lens
    a = Cache(2000)
    a.k, a.v = (torch.randn(2000, HK, BS, D, generator=g, device=DEV).to(F8) for _ in range(2))
    q, k, v = tokens(g, sum(new), HEADS), tokens(g, sum(new), HK), tokens(g, sum(new), HK)
    cu = ints([0] + [sum(new[:i + 1]) for i in range(300)])
    out, lse = mt.chunk_attention(q, k, v, *a.parts(), table, lengths, cu_seqlens=cu)
    at = 0
    for i in (0, 1, 63, 64, 65, 128, 200, 299):
        at, n = int(cu[i]), new[i]
        if n:
            one = mt.chunk_attention(q[at:at + n], k[at:at + n], v[at:at + n], *a.parts(), table[i:i + 1], lengths[i:i + 1], cu_seqlens=ints([0, n]))
            assert (one[0].float() - out[at:at + n].float()).abs().max() <= 4 * 2 ** -8 * 4 and (one[1] - lse[at:at + n]).abs().max() < 1e-4
    assert torch.isfinite(out).all()


def test_refusals_of_chunks():
    args, cu = chunk_inputs(1, [30, 40], [3, 4])
    q, k, v, kc, vc, ks, vs, table, lengths = args

    def refused(match=None, **kw):
        base = dict(q=q, k=k, v=v, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, block_table=table, lengths=lengths, cu_seqlens=cu)
        with pytest.raises(ValueError, match=match):
            mt.chunk_attention(**{**base, **kw})

    refused(q=q[:, :5])
    refused(q=q.float())
    refused(q=q.half())
    refused(q=q[:5])
    refused(k=k[:, :1])
    refused(k=k[:6])
    refused(v=v[..., ::2])
    refused(v=v.cpu())
    refused(k_cache=kc.float())
    refused(k_cache=kc[:, :1])
    refused(v_cache=vc[:5])
    refused(k_scale=ks[:5])
    refused(v_scale=vs.double())
    refused(block_table=table.long())
    refused(block_table=table.t())
    refused(lengths=lengths[:1])
    refused(lengths=lengths.float())
    refused(cu_seqlens=cu[:2])
    refused(cu_seqlens=None)
    refused(max_length=-1)
    refused(scale=0.0)
    refused(scale=math.inf)
    refused(out=torch.empty_like(q, dtype=torch.float16))
    refused(out=torch.empty(7, 6, 128, dtype=q.dtype, device=DEV)[..., ::2])
    with torch.autograd.forward_ad.dual_level():
        refused("tangent", q=torch.autograd.forward_ad.make_dual(q, q))
    # no gradient goes back, whatever is asked for
    out, lse = mt.chunk_attention(q.clone().requires_grad_(), *args[1:], cu_seqlens=cu)
    assert not out.requires_grad and not lse.requires_grad
