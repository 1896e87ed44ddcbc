"""Plain 64-bit forms of the block-attention and 8-bit-cache operators, for the
tests: one sequence, head and query at a time, from the definitions."""

import math

import torch


def spans(total_q, total_k, cu_q=None, cu_k=None):
    """(q0, q1, k0, k1) of every sequence."""
    if cu_q is None:
        return [(0, total_q, 0, total_k)]
    cu_q, cu_k = cu_q.tolist(), (cu_q if cu_k is None else cu_k).tolist()
    return [(cu_q[i], cu_q[i + 1], cu_k[i], cu_k[i + 1]) for i in range(len(cu_q) - 1)]


def visible(blocks_row, bs, keys, pos, causal=True):
    """Boolean [keys]: the keys that a query at ``pos`` with these blocks sees."""
    see = torch.zeros(keys, dtype=torch.bool)
    for b in blocks_row.tolist():
        if b >= 0:
            see[b * bs:(b + 1) * bs] = True
    if causal:
        see[max(pos + 1, 0):] = False
    return see


def attention(q, k, v, blocks, bs, cu_q=None, cu_k=None, scale=None, causal=True, dout=None):
    """(out, lse) in 64 bits, or (out, lse, dq, dk, dv) with ``dout``.  CPU tensors."""
    t, h, d = q.shape
    hk = k.shape[1]
    g = h // hk
    scale = 1 / math.sqrt(d) if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    out, lse = torch.zeros(t, h, d, dtype=torch.float64), torch.full((t, h), -math.inf, dtype=torch.float64)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for a, b, c, e in spans(t, k.shape[0], cu_q, cu_k):
        for r in range(a, b):
            for hh in range(hk):
                see = visible(blocks[r, hh], bs, e - c, (e - c) - (b - a) + r - a, causal)
                at = c + torch.nonzero(see)[:, 0]
                if at.numel() == 0:
                    continue
                heads = slice(hh * g, (hh + 1) * g)
                s = q[r, heads] @ k[at, hh].T * scale
                lse[r, heads] = torch.logsumexp(s, 1)
                p = torch.softmax(s, 1)
                out[r, heads] = p @ v[at, hh]
                if dout is not None:
                    do = dout[r, heads].double()
                    dv[at, hh] += p.T @ do
                    ds = p * (do @ v[at, hh].T - (do * out[r, heads]).sum(1, keepdim=True)) * scale
                    dq[r, heads] = ds @ k[at, hh]
                    dk[at, hh] += ds.T @ q[r, heads]
    return (out, lse) if dout is None else (out, lse, dq, dk, dv)


def means(k, bs, cu=None):
    """block_means in 64 bits."""
    t, hk, d = k.shape
    n = 1 if cu is None else cu.shape[0] - 1
    out = torch.zeros(t // bs + n, hk, d, dtype=torch.float64)
    for i, (a, b, _, _) in enumerate(spans(t, t, cu, cu)):
        for j in range(-(-(b - a) // bs)):
            out[a // bs + i + j] = k[a + j * bs:min(b, a + (j + 1) * bs)].double().mean(0)
    return out


def scores(q, mean_of, bs, max_blocks, placed, hk, first, last, scale=None):
    """block_scores in 64 bits.  ``mean_of(sequence, block)`` gives [hk, dim] or
    None; ``placed``: (row, sequence, position) of every query with a sequence."""
    t, h, d = q.shape
    g = h // hk
    scale = 1 / math.sqrt(d) if scale is None else scale
    out = torch.full((t, hk, max_blocks), -math.inf, dtype=torch.float64)
    counts = torch.zeros(t, hk, dtype=torch.int32)
    for row, seq, pos in placed:
        n = min(pos // bs + 1, max_blocks) if pos >= 0 else 0
        counts[row] = n
        for b in range(n):
            m = mean_of(seq, b)
            if m is None:
                continue
            if b < first or b >= n - last:
                out[row, :, b] = math.inf
            else:
                out[row, :, b] = (q[row].double().view(hk, g, d) * m.double()[:, None]).sum(2).amax(1) * scale
    return out, counts
