"""Plain forms of the serving operators for the tests, from the definitions:
attention in 64 bits a query at a time, pages with Python lists, logits an id at
a time.  CPU tensors."""

import math

import torch


def spans(total, n, cu=None):
    """(first, last) row of every sequence."""
    if cu is None:
        return [(i, i + 1) for i in range(n)]
    cu = [max(0, min(int(c), total)) for c in cu.tolist()]
    return list(zip(cu, cu[1:]))


def chunk_attention(q, k, v, k_cache, v_cache, k_scale, v_scale, table, lengths, bs, cu=None, scale=None):
    """(out, lse, size) in 64 bits; caches as float values of the codes; ``size``: for
    each query and head the largest sum of a score's absolute terms."""
    t, h, d = q.shape
    hk = k.shape[1]
    g = h // hk
    scale = 1 / math.sqrt(d) if scale is None else scale
    out, lse = torch.zeros(t, h, d, dtype=torch.float64), torch.full((t, h), -math.inf, dtype=torch.float64)
    size = torch.zeros(t, h, dtype=torch.float64)
    for i, (a, b) in enumerate(spans(t, len(lengths), cu)):
        context = int(lengths[i]) - (b - a)
        held = max(0, min(context, table.shape[1] * bs))
        for c in range(hk):
            ks, vs = [torch.zeros(0, d, dtype=torch.float64)], [torch.zeros(0, d, dtype=torch.float64)]
            for x in range(-(-held // bs)):
                page = int(table[i, x])
                if 0 <= page < k_cache.shape[0]:
                    e = min(bs, held - x * bs)
                    ks.append(k_cache[page, c, :e].double() * float(k_scale[page, c]))
                    vs.append(v_cache[page, c, :e].double() * float(v_scale[page, c]))
            heads = slice(c * g, (c + 1) * g)
            for r in range(a, b):
                if context + r - a < 0:
                    continue
                first = max(a, a - context)
                kk = torch.cat(ks + [k[first:r + 1, c].double()])
                vv = torch.cat(vs + [v[first:r + 1, c].double()])
                s = q[r, heads].double() @ kk.T * scale
                size[r, heads] = (q[r, heads].double().abs() @ kk.abs().T * scale).amax(1)
                lse[r, heads] = torch.logsumexp(s, 1)
                out[r, heads] = torch.softmax(s, 1) @ vv
    return out, lse, size


class Pages:
    """A block table and its pages with Python lists: block_table, lengths, refs."""

    def __init__(self, table, lengths, refs, bs):
        self.table, self.lengths, self.refs, self.bs = table.tolist(), lengths.tolist(), refs.tolist(), bs
        self.cols = table.shape[1]

    def length(self, i):
        return max(0, min(self.lengths[i], self.cols * self.bs))

    def there(self, page):
        return 0 <= page < len(self.refs)

    def take(self):
        for page, n in enumerate(self.refs):
            if n <= 0:
                self.refs[page] = 1
                return page
        return -1

    def fork(self, parents):
        rows, bs = len(self.table), self.bs
        before = [row[:-(-self.length(i) // bs)] for i, row in enumerate(self.table)]
        had = [self.length(i) for i in range(rows)]
        changed = [i for i in range(rows) if parents[i] != i]
        for i in changed:
            for page in before[i]:
                if self.there(page):
                    self.refs[page] -= 1
        kept = {p for p in range(rows) if parents[p] == p}  # rows whose last page has its holder
        copies, asks = [[-1, -1] for _ in range(rows)], []
        for i in changed:
            p = parents[i]
            if not 0 <= p < rows:
                self.table[i], self.lengths[i] = [-1] * self.cols, 0
                continue
            pages = list(before[p])
            self.lengths[i] = had[p]
            if had[p] % bs:
                if p in kept and self.there(pages[-1]):
                    asks.append((i, pages.pop()))
                else:
                    kept.add(p)
            for page in pages:
                if self.there(page):
                    self.refs[page] += 1
            self.table[i] = pages + [-1] * (self.cols - len(pages))
        for i, source in asks:
            page = self.take()
            copies[i] = [source, page]
            whole = self.lengths[i] // bs
            if page < 0:
                self.lengths[i] = whole * bs
            else:
                self.table[i][whole] = page
        return copies

    def grow(self, grow):
        grown, asked = [0] * len(grow), 0
        free = sum(n <= 0 for n in self.refs)
        for i, n in enumerate(grow):
            n = max(n, 0)
            had, length = -(-self.length(i) // self.bs), self.length(i)
            want = -(-(length + n) // self.bs)
            if want > self.cols:
                continue
            asked += want - had
            if want > had and asked > free:
                continue
            for c in range(had, want):
                self.table[i][c] = self.take()
            if n:
                self.lengths[i] = length + n
            grown[i] = n
        return grown

    def compact(self):
        used = sum(n > 0 for n in self.refs)
        moves = [p for p, n in enumerate(self.refs) if n > 0 and p >= used]
        to = dict(zip(moves, [p for p, n in enumerate(self.refs) if n <= 0 and p < used]))
        for p, t in to.items():
            self.refs[t], self.refs[p] = self.refs[p], 0
        for i, row in enumerate(self.table):
            for c in range(-(-self.length(i) // self.bs)):
                row[c] = to.get(row[c], row[c])
        pairs = [[p, t] for p, t in to.items()]
        return pairs + [[-1, -1]] * (len(self.refs) // 2 - len(pairs))


def penalize(logits, tokens=None, lengths=None, prompts=None, repetition=None, presence=None, frequency=None, bias_ids=None,
             bias=None, mask=None):
    """penalize_logits in 64 bits."""
    y = logits.double().clone()
    rows, vocab = y.shape
    for i in range(rows):
        if tokens is not None:
            n = tokens.shape[1] if lengths is None else max(0, min(int(lengths[i]), tokens.shape[1]))
            prompt = 0 if prompts is None else max(0, min(int(prompts[i]), n))
            r, f, p = (d if x is None else float(x[i]) for x, d in ((repetition, 1.0), (frequency, 0.0), (presence, 0.0)))
            said = {}
            for at, j in enumerate(tokens[i, :n].tolist()):
                if 0 <= j < vocab:
                    said[j] = said.get(j, 0) + (at >= prompt)
            for j, count in said.items():
                x = float(y[i, j])
                x = x / r if x > 0 else x * r
                y[i, j] = x - f * count - p if count else x
        if bias is not None:
            for j, b in dict(zip(bias_ids[i].tolist(), bias[i].tolist())).items():
                if 0 <= j < vocab:
                    y[i, j] += b
        if mask is not None:
            j = torch.arange(vocab)
            y[i, (mask[i].long()[j // 32] >> (j % 32)) % 2 == 0] = -math.inf
    return y
