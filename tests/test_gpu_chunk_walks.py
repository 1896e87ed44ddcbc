"""GPU: the walks that a chunk's workgroups take over long contexts.  A workgroup
looks up 256 blocks at a time; it has four or eight wavefronts; a walk in several
parts is joined.  Sizes are such that each of these is reached with each kind of
page: a bound of the lengths that is too small leaves all that lies behind it to
the last part.  Against a plain form in 64 bits; tolerances as in test_gpu_chunk.py.
"""

import math

import pytest
import torch

import row_wise_top_topk_amd as mt
from test_gpu_chunk import BOTH, DEV, build, check, put

pytestmark = pytest.mark.gpu

SCALE = 1.0   # a few keys, anywhere in the walk, have most of a row's weight: a wrong one shows


def dense(x, bs):
    """What check() takes as ``want``: all rows of a key head at once."""
    t, heads, d = x["q"].shape
    hk = x["k"].shape[1]
    g = heads // hk
    out, lse, size = (torch.zeros(s, dtype=torch.float64) for s in ((t, heads, d), (t, heads), (t, heads)))
    cu = x["cu_seqlens"].tolist()
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        n = b - a
        context = int(x["lengths"][i]) - n
        pages = x["block_table"][i, :-(-context // bs)].long()
        for c in range(hk):
            k, v = (torch.cat([(x[f"{z}_cache"][pages, c].double() * x[f"{z}_scale"][pages, c].double()[:, None, None]).reshape(-1, d)[:context],
                               x[z][a:b, c].double()]).to(DEV) for z in ("k", "v"))
            q = x["q"][a:b, c * g:(c + 1) * g].double().reshape(n * g, d).to(DEV)
            s = q @ k.T.contiguous() * SCALE
            most = q.abs() @ k.abs().T.contiguous() * SCALE
            hidden = torch.arange(context + n, device=DEV) > context + torch.arange(n, device=DEV).repeat_interleave(g)[:, None]
            s.masked_fill_(hidden, -math.inf)
            size[a:b, c * g:(c + 1) * g] = most.masked_fill_(hidden, 0).amax(1).view(n, g).cpu()
            lse[a:b, c * g:(c + 1) * g] = torch.logsumexp(s, 1).view(n, g).cpu()
            out[a:b, c * g:(c + 1) * g] = (torch.softmax(s, 1) @ v).view(n, g, d).cpu()
    return out, lse, size


def run(lens, new, heads, hk, d, bs, dtype, **kw):
    x = build(sum(lens), lens, new, heads, hk, d, bs, dtype, cols=kw.pop("cols", None))
    check(x, bs, mt.chunk_attention(**put(x), scale=SCALE, **kw), want=dense(x, bs))


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_more_blocks_than_are_looked_up_at_once(bs, d, dtype):
    for blocks in (256, 257, 600):                     # the whole walk in one part
        run([blocks * bs + 3], [3], 3, 1, d, bs, dtype, max_length=1)
    run([520 * bs + 7 + 70], [70], 6, 2, d, bs, dtype, max_length=1)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("d,bound", [(64, 1764), (128, 2148)])
def test_a_part_from_inside_a_block_on(d, bound, dtype):
    # parts of three tiles; the last one begins in the middle of a block of 128 keys and has 265 of them
    for n in (36000, 36037):
        run([n + 3], [3], 3, 1, d, 128, dtype, max_length=bound, cols=400)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("d,bs,n", [(128, 32, 26000), (128, 64, 26011), (128, 128, 42003), (64, 64, 26001), (64, 128, 42000), (64, 16, 11000)])
def test_eight_wavefronts_over_many_blocks(d, bs, n, dtype):
    # six parts, of which the last one has more than 256 blocks; pages of 128: from inside a block on
    run([n + 1203], [1203], 8, 1, d, bs, dtype, max_length=7000)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("bs", [16, 64, 128])
def test_eight_wavefronts_and_several_sequences(bs, dtype):
    # twelve parts of 35 tiles; one sequence's walk lies in one part
    for lens, new in (([26500, 9500], [600, 600]), ([2000, 20700, 30], [700, 471, 29])):
        run(lens, new, 8, 1, 128, bs, dtype, cols=25600 // bs if max(lens) < 26000 else None)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("heads,hk,new,n", [(24, 2, 501, 30001), (20, 1, 303, 50003), (32, 2, 97, 100003)])
def test_eight_wavefronts_over_wide_pages_joined(heads, hk, new, n, dtype):
    # groups of 12, 20 and 16 heads: workgroups of 252, 240 and 256 rows
    run([n + new], [new], heads, hk, 128, 128, dtype, cols=100352 // 128)
