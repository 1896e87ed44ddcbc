"""What is measured of the operators of a serving loop: a prompt's chunk over the
8-bit paged cache, the pages of that cache, and the rows of logits that
topk_indices ranks.

Kinds of cases, by ``op``:

``chunk``     chunk_attention: new tokens with their keys in 16 bits behind a cache
``fork``      pages_fork and the pages_copy of one layer: a step of beams or samples
``admit``     pages_fork with rows that end, pages_grow with those that take their place
``compact``   pages_compact and the pages_copy of one layer
``penalize``  penalize_logits: repeated tokens, biases, a grammar's mask

Where ``own`` is false ``run`` computes the same with elementary torch
operations, floating-point values in 32 bits.
"""

import math

import torch

own = False

DEV = "cuda:0"
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_F8 = torch.float8_e4m3fn


def listed():
    return [
        # the last piece of a short prompt: latency of one small call
        {"name": "chunk 33 behind 500", "op": "chunk", "dtype": "bf16", "new": "33", "context": "500", "heads": 8, "kv_heads": 2,
         "dim": 64, "block": 16},
        # one chunk of a long prompt
        {"name": "chunk 2048 behind 32000", "op": "chunk", "dtype": "bf16", "new": "2048", "context": "32000", "heads": 64,
         "kv_heads": 8, "dim": 128, "block": 64},
        # a prompt's first chunk: nothing in the cache yet
        {"name": "prompt 8192", "op": "chunk", "dtype": "bf16", "new": "8192", "context": "0", "heads": 32, "kv_heads": 4,
         "dim": 128, "block": 64},
        # chunks of several requests with single decode tokens among them, one request without any
        {"name": "chunks mixed fp16", "op": "chunk", "dtype": "fp16", "new": "512,1,0,77,300", "context": "5000,7001,33,0,6801",
         "heads": 12, "kv_heads": 3, "dim": 64, "block": 32},
        # a question behind a long document: few rows, many keys
        {"name": "chunk 96 behind 100003", "op": "chunk", "dtype": "bf16", "new": "96", "context": "100003", "heads": 32,
         "kv_heads": 2, "dim": 128, "block": 128},
        # a beam step of 16 requests with four beams each
        {"name": "fork 64 beams", "op": "fork", "rows": 64, "low": 500, "high": 3500, "kv_heads": 8, "dim": 128, "block": 64,
         "spare": 200},
        # samples of long requests, small pages: a large table
        {"name": "fork 512 rows", "op": "fork", "rows": 512, "low": 3000, "high": 30000, "kv_heads": 2, "dim": 64, "block": 16,
         "spare": 40000},
        # half of a batch ends and as many prompts take their place
        {"name": "admit 256", "op": "admit", "rows": 256, "low": 100, "high": 30000, "block": 32, "spare": 50000},
        # a cache of which half was freed is brought to its front
        {"name": "compact 20000 pages", "op": "compact", "rows": 160, "low": 1000, "high": 7000, "kv_heads": 8, "dim": 128,
         "block": 64, "pages": 20000},
        # rows of logits of a decode batch: chats with some biases and a grammar
        {"name": "penalize 64x128256", "op": "penalize", "dtype": "bf16", "rows": 64, "vocab": 128256, "low": 300, "high": 8000,
         "bias": 20, "mask": True},
        # one small call of few rows
        {"name": "penalize 3x32000", "op": "penalize", "dtype": "fp32", "rows": 3, "vocab": 32000, "low": 5, "high": 40, "bias": 0,
         "mask": False},
        # rows behind long documents, a large vocabulary of odd size
        {"name": "penalize 32x151937 long", "op": "penalize", "dtype": "fp16", "rows": 32, "vocab": 151937, "low": 50000,
         "high": 100000, "bias": 300, "mask": True},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "fork", "admit", "compact", "penalize", "penalize"])
    if op == "penalize":
        rows, vocab = _log(rng, 1, 200), _log(rng, 1000, 200000)
        rows = max(1, min(rows, 8000000 // vocab))
        high = _log(rng, 2, 60000)
        return {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "rows": rows, "vocab": vocab, "low": max(1, high // rng.choice([1, 3, 20])),
                "high": high, "bias": rng.choice([0, 1, 17, 300]), "mask": rng.random() < 0.5}
    block = rng.choice([16, 32, 64, 128])
    if op == "chunk":
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 5, 8])
        n = rng.choice([1, 1, 2, 3, 6])
        new = [_log(rng, 1, 3000 // n) for _ in range(n)]
        context = [rng.choice([0, 1, 1, 1]) * _log(rng, 1, 30000 // n) for _ in range(n)]
        return {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "new": ",".join(map(str, new)), "context": ",".join(map(str, context)),
                "heads": heads, "kv_heads": kv, "dim": rng.choice([64, 128]), "block": block}
    rows = _log(rng, 2, 300)
    high = _log(rng, 20, 20000)
    case = {"op": op, "rows": rows, "low": max(1, high // rng.choice([1, 4, 30])), "high": high, "block": block}
    total = rows * (high // block + 1)
    if op != "admit":
        case |= {"kv_heads": rng.choice([1, 2, 3, 8]), "dim": rng.choice([64, 128])}
        while total * block * case["kv_heads"] * case["dim"] > 4.0e8 and case["rows"] > 2:
            case["rows"] //= 2
            total = case["rows"] * (high // block + 1)
    if op == "compact":
        case["pages"] = total + _log(rng, 1, 2 * total + 10)
    else:
        case["spare"] = case["rows"] + total + rng.choice([0, 7, 1000])
    return case


def _ints(text):
    return [int(x) for x in text.split(",")]


def _lengths(case):
    """The rows' lengths: spread over [low, high] in a fixed shuffled order."""
    n, lo, hi = case["rows"], case["low"], case["high"]
    return [hi] if n == 1 else [lo + (hi - lo) * ((i * 37) % n) // (n - 1) for i in range(n)]


def _codes(g, *shape):
    # normal values about a quarter of e4m3's range wide
    return (100 * torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)).clamp_(-448, 448).to(_F8)


def _prepare_chunk(case, g):
    new, context = _ints(case["new"]), _ints(case["context"])
    n, h, hk, d, bs, dt = len(new), case["heads"], case["kv_heads"], case["dim"], case["block"], _TYPES[case["dtype"]]
    t, lens = sum(new), [a + b for a, b in zip(new, context)]
    need = [-(-x // bs) for x in lens]
    pages, wide = sum(need) + 3, max(1, max(need))
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(wide, device=DEV)
    needed = torch.tensor(need, device=DEV)[:, None]
    at = torch.cumsum(needed, 0) - needed + col
    table = torch.where(col < needed, order[at.clamp_max(pages - 1)], 0).to(torch.int32)
    count = torch.tensor(new, device=DEV)
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), count)
    row = torch.arange(t, device=DEV) - (torch.cumsum(count, 0) - count)[seq]
    pos = row + torch.tensor(context, device=DEV)[seq]
    cu = torch.nn.functional.pad(torch.cumsum(count, 0), (1, 0)).to(torch.int32)
    scales = lambda: torch.exp2(torch.randint(-8, -5, (pages, hk), generator=g, device=DEV).float())  # noqa: E731
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return {"case": case, "q": (2.5 * rand(t, h, d)).to(dt), "k": (0.8 * rand(t, hk, d)).to(dt), "v": (0.8 * rand(t, hk, d)).to(dt),
            "k_cache": _codes(g, pages, hk, bs, d), "v_cache": _codes(g, pages, hk, bs, d), "k_scale": scales(),
            "v_scale": scales(), "table": table, "lengths": torch.tensor(lens, dtype=torch.int32, device=DEV), "cu": cu,
            "high": max(lens), "most": max(1, max(new)), "seq": seq, "row": row, "pos": pos}


def _prepare_pages(case, g):
    lens, bs = _lengths(case), case["block"]
    rows = len(lens)
    need = [-(-x // bs) for x in lens]
    held = sum(need)
    pages = case["pages"] if case["op"] == "compact" else held + case["spare"]
    wide = -(-case["high"] // bs)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(wide, device=DEV)
    needed = torch.tensor(need, device=DEV)[:, None]
    at = torch.cumsum(needed, 0) - needed + col
    table = torch.where(col < needed, order[at.clamp_max(pages - 1)], -1).to(torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs[order[:held].long()] = 1
    s = {"case": case, "table": table, "refs": refs, "lengths": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    row = torch.arange(rows, device=DEV)
    if case["op"] == "admit":
        # rows end at random; the new prompts are as long as those that were there
        out = torch.rand(rows, generator=g, device=DEV) < 0.5
        s["parents"] = torch.where(out, -1, row).to(torch.int32)
        length = torch.tensor(lens, device=DEV)[torch.randperm(rows, generator=g, device=DEV)]
        s["grow"] = torch.where(out, length, 0).to(torch.int32)
        return s
    hk, d = case["kv_heads"], case["dim"]
    scales = lambda: torch.exp2(torch.randint(-8, -5, (pages, hk), generator=g, device=DEV).float())  # noqa: E731
    s |= {"k_cache": _codes(g, pages, hk, bs, d), "v_cache": _codes(g, pages, hk, bs, d), "k_scale": scales(), "v_scale": scales(),
          "mean": 0.3 * torch.randn(pages, hk, d, generator=g, device=DEV)}
    if case["op"] == "fork":
        # of each four neighbours some go on, the others are replaced by forks of one that does
        best = (row // 4 * 4 + (torch.rand(rows, generator=g, device=DEV) * 4).long()[row // 4 * 4]).clamp_max(rows - 1)
        stays = torch.rand(rows, generator=g, device=DEV) < 0.4
        s["parents"] = torch.where(stays, row, best).to(torch.int32)
        s["parents"][best] = best.to(torch.int32)
    else:
        s["before"] = tuple(s[n].clone() for n in ("table", "refs"))
    return s


def _prepare_penalize(case, g):
    rows, vocab, dt = case["rows"], case["vocab"], _TYPES[case["dtype"]]
    lens = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)
    # a text's tokens: a few ids are frequent, most are rare
    ids = (vocab ** torch.rand(rows, case["high"], generator=g, device=DEV)).long().clamp_max(vocab - 1)
    tokens = torch.randperm(vocab, generator=g, device=DEV)[ids].to(torch.int32)
    some = lambda lo, hi: lo + (hi - lo) * torch.rand(rows, generator=g, device=DEV)  # noqa: E731
    s = {"case": case, "logits": (4 * torch.randn(rows, vocab, generator=g, device=DEV)).to(dt), "tokens": tokens, "lengths": lens,
         "prompt": (lens * some(0.1, 0.9)).to(torch.int32), "repetition": some(1.0, 1.3), "frequency": some(0.0, 0.7),
         "presence": some(0.0, 0.7), "bias_ids": None, "bias": None, "mask": None}
    if case["bias"]:
        pick = torch.rand(rows, vocab, generator=g, device=DEV).topk(case["bias"], dim=1)[1]
        s["bias_ids"], s["bias"] = pick.to(torch.int32), 5 * torch.randn(rows, case["bias"], generator=g, device=DEV)
    if case["mask"]:
        words = torch.randint(-2 ** 31, 2 ** 31, (rows, -(-vocab // 32)), generator=g, device=DEV).to(torch.int32)
        # every other row is within a grammar's rule that allows little, the others nearly everything
        s["mask"] = torch.where(torch.arange(rows, device=DEV)[:, None] % 2 == 0, words & (words >> 3), words | (words << 7) | 1)
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    if case["op"] == "chunk":
        return _prepare_chunk(case, g)
    return _prepare_penalize(case, g) if case["op"] == "penalize" else _prepare_pages(case, g)


def run(state):
    op = state["case"]["op"]
    if op == "compact":  # the cache as it was, where a pass before this one has brought it to the front
        for name, was in zip(("table", "refs"), state["before"]):
            state[name].copy_(was)
    if own:
        return _run_own(state)
    if op == "chunk":
        return _plain_chunk(state)
    if op == "penalize":
        return _plain_penalize(state)
    return _plain_pages(state)


def _run_own(s):
    import row_wise_top_topk_amd as mt
    op, bs = s["case"]["op"], s["case"].get("block")
    if op == "chunk":
        out, lse = mt.chunk_attention(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                      s["lengths"], cu_seqlens=s["cu"], max_length=s["high"])
        return {"out": out, "lse": lse}
    if op == "penalize":
        return mt.penalize_logits(s["logits"], s["tokens"], s["lengths"], s["prompt"], repetition=s["repetition"],
                                  presence=s["presence"], frequency=s["frequency"], bias_ids=s["bias_ids"], bias=s["bias"],
                                  mask=s["mask"])
    if op == "compact":
        copies = mt.pages_compact(s["table"], s["lengths"], s["refs"], bs)
    else:
        copies = mt.pages_fork(s["table"], s["lengths"], s["refs"], s["parents"], bs)
    out = {"copies": copies}
    if op == "admit":
        out["grown"] = mt.pages_grow(s["table"], s["lengths"], s["refs"], s["grow"], bs)
    else:
        mt.pages_copy(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], copies, k_mean=s["mean"])
    return out | {n: s[n] for n in ("table", "lengths", "refs", "k_cache", "v_cache", "k_scale", "v_scale", "mean") if n in s}


# The plain forms.


def _plain_chunk(s):
    case, q = s["case"], s["q"]
    t, h, d = q.shape
    hk, n, most = case["kv_heads"], s["table"].shape[0], s["most"]
    g, seq, table = h // hk, s["seq"], s["table"].long()

    def keys(cache, scale, new):
        x = (cache[table].float() * scale[table][..., None, None]).transpose(1, 2).reshape(n, hk, -1, d)
        x[seq, :, s["pos"]] = new.float()
        return x

    # rows padded to the longest chunk
    a = torch.zeros(n, most, h, d, device=DEV)
    a[seq, s["row"]] = q.float()
    a = a.view(n, most, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, g * most, d)
    k = keys(s["k_cache"], s["k_scale"], s["k"])
    p = torch.matmul(a, k.transpose(2, 3).contiguous()).mul_(1 / math.sqrt(d)).view(n, hk, g, most, -1)
    at = torch.full((n, most), -1, device=DEV)
    at[seq, s["row"]] = s["pos"]
    p.masked_fill_((torch.arange(k.shape[2], device=DEV) > at[:, :, None])[:, None, None], -math.inf)
    top = p.amax(4, keepdim=True).clamp_min(-3e38)
    p = p.sub_(top).exp_()
    total = p.sum(4, keepdim=True)
    p = p.view(n, hk, g * most, -1)
    v = keys(s["v_cache"], s["v_scale"], s["v"])
    out = torch.matmul(p, v).view(n, hk, g, most, d) / total.clamp_min(1e-38)
    lse = (top + total.log())[..., 0]
    out = out.permute(0, 3, 1, 2, 4).reshape(n, most, h, d)[seq, s["row"]]
    return {"out": out.to(q.dtype), "lse": lse.permute(0, 3, 1, 2).reshape(n, most, h)[seq, s["row"]]}


def _lowest_free(refs, rank):
    """The page that is free and has ``rank`` free ones before it; -1 where there are not so many."""
    free = torch.cat([torch.nonzero(refs <= 0)[:, 0], torch.full((1,), -1, device=DEV)])
    return free[rank.clamp(0, free.shape[0] - 1)]


def _count(refs, pages, by):
    """refs[pages] += by, for the pages that are there."""
    at = pages[(pages >= 0) & (pages < refs.shape[0])].long()
    refs.index_add_(0, at, torch.full_like(at, by, dtype=torch.int32))


def _plain_fork(s):
    table, lengths, refs, bs = s["table"], s["lengths"], s["refs"], s["case"]["block"]
    rows, cols = table.shape
    row, col = torch.arange(rows, device=DEV), torch.arange(cols, device=DEV)
    parents = s["parents"].long()
    ends = (parents < 0) | (parents >= rows)
    at = torch.where(ends, row, parents)
    stays = parents == row
    length = torch.where(ends, 0, lengths[at])
    whole, part = length // bs, (length % bs > 0)
    # who has the parent's last page, where that is not full: the parent itself, or its first fork
    claim = torch.where(stays, -1, row)
    first = torch.full((rows,), rows, device=DEV).scatter_reduce_(0, at, torch.where(ends, rows, claim), "amin")
    holds = ~ends & (first[at] == claim)
    held = col < ((lengths + bs - 1) // bs)[:, None]
    share = col < (whole + (holds & part))[:, None]
    new = table[at]
    _count(refs, torch.where(held & ~stays[:, None], table, -1), -1)
    _count(refs, torch.where(share & ~stays[:, None], new, -1), 1)
    asks = ~ends & part & ~holds
    page = torch.where(asks, _lowest_free(refs, torch.cumsum(asks.long(), 0) - 1), -1).to(torch.int32)
    _count(refs, page, 1)
    source = new.gather(1, whole.clamp_max(cols - 1).long()[:, None])[:, 0]
    copies = torch.stack([torch.where(asks, source, -1), page], 1)
    length = torch.where(asks & (page < 0), whole * bs, length)
    new = torch.where(share, new, torch.where(asks[:, None] & (col == whole[:, None]), page[:, None], -1))
    table.copy_(torch.where(stays[:, None], table, new))
    lengths.copy_(torch.where(stays, lengths, length))
    return copies


def _plain_grow(s):
    table, lengths, refs, bs = s["table"], s["lengths"], s["refs"], s["case"]["block"]
    cols = table.shape[1]
    col = torch.arange(cols, device=DEV)
    grow = s["grow"].clamp_min(0).long()
    length = lengths.clamp_min(0).long()
    has, want = (length + bs - 1) // bs, (length + grow + bs - 1) // bs
    fits = want <= cols
    asks = torch.where(fits, want - has, 0)
    before = torch.cumsum(asks, 0) - asks
    fits &= (asks == 0) | (before + asks <= (refs <= 0).sum())
    new = fits[:, None] & (col >= has[:, None]) & (col < want[:, None])
    page = _lowest_free(refs, torch.where(new, before[:, None] + col - has[:, None], 0))
    page = torch.where(new, page, -1)
    _count(refs, page, 1)
    table.copy_(torch.where(new, page, table))
    grown = torch.where(fits, grow, 0).to(torch.int32)
    lengths.copy_((length + grown).to(torch.int32))
    return grown


def _plain_compact(s):
    table, lengths, refs, bs = s["table"], s["lengths"], s["refs"], s["case"]["block"]
    pages = refs.shape[0]
    page = torch.arange(pages, device=DEV)
    live = refs > 0
    cut = live.sum()
    moves = live & (page >= cut)
    rank = torch.cumsum(moves.long(), 0) - 1
    to = torch.where(moves, _lowest_free(refs, rank), page)
    slot = torch.where(moves, rank, pages // 2)
    copies = torch.full((pages // 2 + 1, 2), -1, dtype=torch.int32, device=DEV)
    copies[slot] = torch.where(moves[:, None], torch.stack([page, to], 1), -1).to(torch.int32)
    held = torch.arange(table.shape[1], device=DEV) < ((lengths + bs - 1) // bs)[:, None]
    held &= (table >= 0) & (table < pages)
    table.copy_(torch.where(held, to[torch.where(held, table, 0).long()].to(torch.int32), table))
    refs.copy_(torch.zeros_like(refs).index_add_(0, to, refs))
    return copies[:pages // 2].contiguous()


def _plain_copy(s, copies):
    src, dst = copies[(copies >= 0).all(1)].long().T
    for name in ("k_cache", "v_cache"):
        codes = s[name].view(torch.uint8)
        codes[dst] = codes[src]
    for name in ("k_scale", "v_scale", "mean"):
        s[name][dst] = s[name][src]


def _plain_pages(s):
    op = s["case"]["op"]
    copies = _plain_compact(s) if op == "compact" else _plain_fork(s)
    out = {"copies": copies}
    if op == "admit":
        out["grown"] = _plain_grow(s)
    else:
        _plain_copy(s, copies)
    return out | {n: s[n] for n in ("table", "lengths", "refs", "k_cache", "v_cache", "k_scale", "v_scale", "mean") if n in s}


def _plain_penalize(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    at = torch.arange(s["tokens"].shape[1], device=DEV)
    written = at < s["lengths"][:, None]
    said = written & (at >= s["prompt"][:, None])
    ids = s["tokens"].long()
    count = torch.zeros_like(x).scatter_add_(1, ids, said.float())
    seen = torch.zeros_like(x).scatter_add_(1, ids, written.float()) > 0
    r = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if s["bias"] is not None:
        x = x.scatter_add(1, s["bias_ids"].long(), s["bias"])
    if s["mask"] is not None:
        bit = torch.arange(32, device=DEV, dtype=torch.int32)
        allowed = ((s["mask"][:, :, None] >> bit) & 1).view(rows, -1)[:, :vocab] > 0
        x = x.masked_fill(~allowed, -math.inf)
    return x


# From the definitions, in 64 bits.


def _exact_chunk(case, s):
    t, h, d = s["q"].shape
    hk, bs = case["kv_heads"], case["block"]
    out = torch.zeros(t, h, d, dtype=torch.float64, device=DEV)
    lse = torch.full((t, h), -math.inf, dtype=torch.float64, device=DEV)
    first = 0
    for i, (n, c) in enumerate(zip(_ints(case["new"]), _ints(case["context"]))):
        if n == 0:
            continue
        mine = s["table"][i, :-(-c // bs)].long()
        for j in range(hk):
            k, v = (torch.cat([(s[name + "_cache"][mine, j].double() * s[name + "_scale"][mine, j].double()[:, None, None]).reshape(-1, d)[:c],
                               s[name][first:first + n, j].double()]) for name in ("k", "v"))
            for head in range(j * (h // hk), (j + 1) * (h // hk)):
                score = s["q"][first:first + n, head].double() @ k.T / math.sqrt(d)
                score = torch.where(torch.ones_like(score, dtype=torch.bool).tril(c), score, -math.inf)
                lse[first:first + n, head] = torch.logsumexp(score, 1)
                out[first:first + n, head] = torch.softmax(score, 1) @ v
        first += n
    return {"out": out, "lse": lse}


def _exact_penalize(s):
    y = s["logits"].double()
    vocab = y.shape[1]
    number = torch.arange(vocab, device=DEV)
    for i, (n, prompt) in enumerate(zip(s["lengths"].tolist(), s["prompt"].tolist())):
        mine = s["tokens"][i].long()
        r, f, p = (s[name][i].double() for name in ("repetition", "frequency", "presence"))
        old, mentioned = torch.bincount(mine[:prompt], minlength=vocab), torch.bincount(mine[prompt:n], minlength=vocab).double()
        seen = (old > 0) | (mentioned > 0)
        y[i] = torch.where(seen & (y[i] > 0), y[i] / r, torch.where(seen, y[i] * r, y[i])) - f * mentioned - p * mentioned.clamp_max(1)
        if s["bias"] is not None:
            y[i, s["bias_ids"][i].long()] += s["bias"][i].double()
        if s["mask"] is not None:
            y[i, (s["mask"][i].long()[number // 32] >> (number % 32)) % 2 == 0] = -math.inf
    return y


def exact(case, seed):
    if case["op"] in ("fork", "admit", "compact"):
        return None  # whole numbers, and values that are moved as they are
    s = prepare(case, seed)
    return _exact_chunk(case, s) if case["op"] == "chunk" else _exact_penalize(s)


def _pairs(case):
    return sum(n * c + n * (n + 1) // 2 for n, c in zip(_ints(case["new"]), _ints(case["context"])))


def work(case):
    op = case["op"]
    if op == "chunk":
        new, context = sum(_ints(case["new"])), sum(_ints(case["context"]))
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        return {"bytes": new * h * (4 * d + 4) + new * hk * d * 4 + context * hk * (2 * d + 8 / case["block"]), "flops": 4 * d * h * _pairs(case)}
    if op == "penalize":
        rows, vocab = case["rows"], case["vocab"]
        size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        return {"bytes": rows * vocab * (size + 4 + (0.125 if case["mask"] else 0)) + 4 * sum(_lengths(case)) + 8 * rows * case["bias"],
                "flops": 2 * rows * vocab}
    lens, bs = _lengths(case), case["block"]
    held = sum(-(-n // bs) for n in lens)
    if op == "admit":  # half of the rows give their entries up and get others; a count of each page
        return {"bytes": 12 * held / 2 + 4 * (held + case["spare"]), "flops": held}
    page = case["kv_heads"] * (bs * case["dim"] * 2 + 8 + 4 * case["dim"])
    if op == "fork":  # 0.45 of the rows are replaced: entries given up, read and written, a page copied where the last is not full
        return {"bytes": 0.45 * (12 * held + 2 * page * len(lens)) + 4 * (held + case["spare"]), "flops": held}
    moved = held * max(0, case["pages"] - held) / case["pages"]  # live pages behind the first `held`, where they lie at random
    return {"bytes": 2 * page * moved + 8 * held + 8 * case["pages"], "flops": held}
