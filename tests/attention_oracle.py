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
    """(out, lse) in 64 bits, or with ``dout`` (out, lse, dq, dk, dv, sizes):
    ``sizes`` are, for dq, dk and dv, the sums of the absolute terms, where a
    score's gradient counts with what a rounding of out moves it by.  CPU tensors."""
    t, h, d = q.shape
    hk = k.shape[1]
    g = h // hk
    scale = 1 / math.sqrt(d) if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    out, lse = torch.zeros(t, h, d, dtype=torch.float64), torch.full((t, h), -math.inf, dtype=torch.float64)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    sq, sk, sv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
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
                    size = ds.abs() + p * (do * out[r, heads]).abs().sum(1, keepdim=True) * scale
                    sq[r, heads] = size @ k[at, hh].abs()
                    sk[at, hh] += size.T @ q[r, heads].abs()
                    sv[at, hh] += p.T @ do.abs()
    return (out, lse) if dout is None else (out, lse, dq, dk, dv, (sq, sk, sv))


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


def scale_for(most):
    """The smallest power of two, 2^-60 at least, that brings ``most`` to 448 or less."""
    s = 2.0 ** -60
    while most > 448 * s:
        s *= 2
    return s


def append(k, v, k_cache, v_cache, k_scale, v_scale, table, lengths, bs, cu=None, k_mean=None):
    """kv8_append on CPU copies, a page and head at a time; caches as float values of the codes."""
    n = len(lengths)
    for i in range(n):
        a, b = (i, i + 1) if cu is None else (int(cu[i]), int(cu[i + 1]))
        length = int(lengths[i])
        start = length - (b - a)
        for j in range(max(start, 0) // bs, -(-length // bs) if b > a else 0):
            if j >= table.shape[1] or not 0 <= int(table[i, j]) < k_cache.shape[0]:
                continue
            page = int(table[i, j])
            lo, hi = max(0, start - j * bs), min(bs, length - j * bs)
            for x, cache, scale in ((k, k_cache, k_scale), (v, v_cache, v_scale)):
                for c in range(x.shape[1]):
                    new = x[a + j * bs + lo - start:a + j * bs + hi - start, c].double()
                    finite = new[torch.isfinite(new)].abs()
                    s = scale_for(finite.max().item() if finite.numel() else 0.0)
                    old = float(scale[page, c])
                    if lo > 0:
                        s = max(s, old)
                        if s > old:
                            cache[page, c, :lo] = round8(cache[page, c, :lo].double() * old / s)
                    cache[page, c, lo:hi] = round8(new / s)
                    scale[page, c] = s
            if k_mean is not None:
                k_mean[page] = (k_cache[page, :, :hi].double().mean(1) * k_scale[page, :, None].double()).to(k_mean.dtype)


def round8(x):
    """Rounded to nearest even e4m3, values behind 448 to it."""
    return x.clamp(-448, 448).float().to(torch.float8_e4m3fn).float()


def cache_attention(q, k_cache, v_cache, k_scale, v_scale, table, lengths, bs, cu=None, blocks=None, scale=None):
    """(out, lse) of kv8_attention in 64 bits; caches as float values of the codes."""
    t, h, d = q.shape
    hk = k_cache.shape[1]
    g = h // hk
    scale = 1 / math.sqrt(d) if scale is None else scale
    out, lse = torch.zeros(t, h, d, dtype=torch.float64), torch.full((t, h), -math.inf, dtype=torch.float64)
    for i in range(len(lengths)):
        a, b = (i, i + 1) if cu is None else (int(cu[i]), int(cu[i + 1]))
        for r in range(a, b):
            pos = int(lengths[i]) - (b - a) + r - a
            if pos < 0:
                continue
            pos = min(pos, table.shape[1] * bs - 1)
            for c in range(hk):
                seen = range(pos // bs + 1)
                if blocks is not None:
                    seen = sorted({x for x in blocks[r, c].tolist() if 0 <= x <= pos // bs})
                ks, vs = [], []
                for x in seen:
                    page = int(table[i, x])
                    if 0 <= page < k_cache.shape[0]:
                        e = min(bs, pos + 1 - x * bs)
                        ks.append(k_cache[page, c, :e].double() * float(k_scale[page, c]))
                        vs.append(v_cache[page, c, :e].double() * float(v_scale[page, c]))
                if not ks:
                    continue
                heads = slice(c * g, (c + 1) * g)
                s = q[r, heads].double() @ torch.cat(ks).T * scale
                lse[r, heads] = torch.logsumexp(s, 1)
                out[r, heads] = torch.softmax(s, 1) @ torch.cat(vs)
    return out, lse
