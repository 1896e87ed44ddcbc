"""What is measured of the operators around block selection: scores of blocks,
attention over the selected blocks with its gradient, and the 8-bit paged cache
with the attention that reads it.

Five kinds of cases, by ``op``:

``score``   block_means + block_scores over a packed prompt (the step before
            topk_indices while a prompt is read or a model is trained)
``rank``    block_scores over the cached block means of a decode batch
``prompt``  block_attention, forward only
``train``   block_attention and its gradient
``append``  kv8_append: new keys and values into the 8-bit paged cache
``decode``  kv8_attention over that cache, whole or at selected blocks

Where ``own`` is false ``run`` computes the same with elementary torch
operations in 32 bits.
"""

import math

import torch

own = False

DEV = "cuda:0"
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # scoring step of an 8K prompt: 4 key heads, 8 query heads each
        {"name": "score prompt 8192", "op": "score", "dtype": "bf16", "q_lens": "8192", "k_lens": "8192", "heads": 32,
         "kv_heads": 4, "dim": 128, "block": 64, "select": 16},
        # scoring step of a decode batch: 64 requests of up to 60000 tokens
        {"name": "rank decode 64", "op": "rank", "dtype": "bf16", "seqs": 64, "new": 1, "low": 937, "high": 60000,
         "heads": 64, "kv_heads": 8, "dim": 128, "block": 64},
        # a short chat turn: latency of one small call
        {"name": "prompt 517", "op": "prompt", "dtype": "bf16", "q_lens": "517", "k_lens": "517", "heads": 16, "kv_heads": 2,
         "dim": 128, "block": 64, "select": 8},
        # several ragged prompts packed into one call, small heads and blocks, one sequence empty
        {"name": "prompt packed fp16", "op": "prompt", "dtype": "fp16", "q_lens": "1777,1,0,640,3001,129",
         "k_lens": "1777,1,0,640,3001,129", "heads": 12, "kv_heads": 3, "dim": 64, "block": 32, "select": 24},
        # one chunk of a long prompt: the last 2048 of 65536 tokens ask
        {"name": "prompt chunk 2048/65536", "op": "prompt", "dtype": "bf16", "q_lens": "2048", "k_lens": "65536", "heads": 64,
         "kv_heads": 4, "dim": 128, "block": 64, "select": 32},
        # a training step's attention on one 8K sequence
        {"name": "train 8192", "op": "train", "dtype": "bf16", "q_lens": "8192", "k_lens": "8192", "heads": 32, "kv_heads": 2,
         "dim": 128, "block": 64, "select": 16},
        # a training step's attention on packed documents of odd lengths
        {"name": "train packed", "op": "train", "dtype": "bf16", "q_lens": "1031,2,517,1999", "k_lens": "1031,2,517,1999",
         "heads": 8, "kv_heads": 2, "dim": 64, "block": 32, "select": 12},
        # one decode step's new tokens of 64 requests into the cache
        {"name": "append decode 64", "op": "append", "dtype": "bf16", "seqs": 64, "new": 1, "low": 100, "high": 4000,
         "kv_heads": 8, "dim": 128, "block": 64},
        # prompts of two requests into the cache, behind what it holds of them
        {"name": "append prompt 2x8191", "op": "append", "dtype": "bf16", "seqs": 2, "new": 8191, "low": 9001, "high": 12002,
         "kv_heads": 8, "dim": 128, "block": 64},
        # a decode batch over its whole cache
        {"name": "decode 64 whole", "op": "decode", "dtype": "bf16", "seqs": 64, "new": 1, "low": 500, "high": 32000,
         "heads": 64, "kv_heads": 8, "dim": 128, "block": 64, "select": 0},
        # few requests, three new tokens each (a draft being checked), odd heads
        {"name": "decode 3x3 whole fp16", "op": "decode", "dtype": "fp16", "seqs": 3, "new": 3, "low": 7000, "high": 20011,
         "heads": 10, "kv_heads": 2, "dim": 64, "block": 16, "select": 0},
        # long requests at their selected blocks
        {"name": "decode 8x900000 selected", "op": "decode", "dtype": "bf16", "seqs": 8, "new": 1, "low": 800000, "high": 900000,
         "heads": 32, "kv_heads": 2, "dim": 128, "block": 64, "select": 32},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["score", "rank", "prompt", "prompt", "train", "append", "decode", "decode"])
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 5, 8, 16])
    while heads > 64:
        heads //= 2
    heads = max(kv, heads - heads % kv)
    case = {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "heads": heads, "kv_heads": kv, "dim": rng.choice([64, 128]),
            "block": rng.choice([16, 32, 64, 128])}
    if op in ("score", "prompt", "train"):
        lens = [_log(rng, 33, 3000) for _ in range(rng.choice([1, 1, 2, 4, 7]))]
        lens = lens[: 1 + next((i for i in range(len(lens)) if sum(lens[: i + 1]) > 4000), len(lens) - 1)]
        case["q_lens"] = case["k_lens"] = ",".join(str(n) for n in lens)
        if op == "prompt" and rng.random() < 0.3:
            case["k_lens"] = ",".join(str(n + _log(rng, 1, 9000)) for n in lens)
        case["select"] = rng.choice([1, 4, 8, 13, 16, 24, 32])
        return case
    case["seqs"] = _log(rng, 1, 80)
    case["new"] = rng.choice([1, 1, 1, 2, 4])
    if op == "append" and rng.random() < 0.5:
        case["seqs"], case["new"] = rng.choice([1, 2, 3]), _log(rng, 5, 5000)
    top = max(case["new"] + 40, int(min(30000, 3.0e6 / case["seqs"] / kv)))
    case["high"] = max(case["new"], _log(rng, case["new"] + 30, top))
    case["low"] = max(case["new"], case["high"] // rng.choice([1, 2, 9]))
    case["select"] = rng.choice([0, 0, 5, 16, 32]) if op == "decode" else 0
    return case


def _ints(text):
    return [int(x) for x in text.split(",")]


def _lengths(case):
    """The requests' lengths: spread over [low, high] in a fixed shuffled order."""
    n, lo, hi = case["seqs"], case["low"], case["high"]
    return [hi] if n == 1 else [lo + (hi - lo) * ((i * 37) % n) // (n - 1) for i in range(n)]


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def _places(lens, starts):
    """(sequence, position) of every packed token; ``starts``: position of each sequence's first one."""
    n = torch.tensor(lens, device=DEV)
    seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), n)
    first = torch.cumsum(n, 0) - n
    return seq, torch.arange(int(sum(lens)), device=DEV) - first[seq] + torch.tensor(starts, device=DEV)[seq]


def _prepare_packed(case, g):
    ql, kl = _ints(case["q_lens"]), _ints(case["k_lens"])
    h, hk, d, bs = case["heads"], case["kv_heads"], case["dim"], case["block"]
    t, tk, dt = sum(ql), sum(kl), _TYPES[case["dtype"]]
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    # Keys of 64 neighbouring tokens share a subject; queries of 32 neighbouring
    # tokens ask for one subject of the text before them.
    subject = rand(tk // 64 + 2, hk, d)
    at = torch.arange(tk, device=DEV)
    k = (0.8 * subject[at // 64] + 0.6 * rand(tk, hk, d)).to(dt)
    v = (rand(tk, hk, d) + 0.3 * subject[at // 64]).to(dt)
    seq, pos = _places(ql, [b - a for a, b in zip(ql, kl)])
    kseq, kpos = _places(kl, [0] * len(kl))
    cu, cuk = _offsets(ql), _offsets(kl)
    asks = torch.rand(t // 32 + 1, generator=g, device=DEV)[torch.arange(t, device=DEV) // 32]
    asked = (cuk[seq] + (asks * pos).long()) // 64
    q = (0.5 * subject[asked].repeat_interleave(h // hk, 1) + 1.5 * rand(t, h, d)).to(dt)
    s = {"case": case, "q": q, "k": k, "v": v, "cu": cu, "cuk": cuk, "seq": seq, "pos": pos, "kseq": kseq, "kpos": kpos,
         "blocks_most": max(1, -(-max(kl) // bs)), "seqs": len(ql), "plain_rows": tk // bs + len(kl)}
    if case["op"] == "score":
        return s
    # The selection: the blocks of the largest mean score, the first and the own block always among them.
    nb, sel = s["blocks_most"], case["select"]
    row = cuk[kseq] // bs + kseq + kpos // bs
    total = torch.zeros(s["plain_rows"], hk, d, device=DEV).index_add_(0, row, k.float())
    mean = total / torch.bincount(row, minlength=s["plain_rows"]).clamp_min(1)[:, None, None]
    qs = q.float().view(t, hk, h // hk, d).sum(2)
    score = torch.matmul(qs.transpose(0, 1), mean.permute(1, 2, 0).contiguous()).transpose(0, 1)
    block = torch.arange(nb, device=DEV)
    score = score.gather(2, (cuk[seq] // bs + seq)[:, None, None].expand(t, hk, 1) + block.clamp_max(s["plain_rows"] - 1 - (cuk[seq] // bs + seq)[:, None])[:, None])
    last = (pos // bs)[:, None, None]
    score = score.masked_fill((block == 0) | (block == last), math.inf).masked_fill(block > last, -math.inf)
    best, picked = torch.topk(score, min(sel, nb), dim=2)
    picked = torch.where(best == -math.inf, nb, picked).sort(2)[0]
    picked = torch.where(picked == nb, -1, picked).to(torch.int32)
    s["blocks"] = torch.nn.functional.pad(picked, (0, sel - picked.shape[2]), value=-1).contiguous()
    if case["op"] == "train":
        s["dout"] = rand(t, h, d).to(dt)
    return s


def _prepare_cache(case, g):
    lens, new = _lengths(case), case["new"]
    n, hk, d, bs = case["seqs"], case["kv_heads"], case["dim"], case["block"]
    dt = _TYPES[case["dtype"]]
    need = [-(-x // bs) for x in lens]
    pages, wide = sum(need) + 3, max(need)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(n, wide, dtype=torch.int32, device=DEV)
    at = 0
    for i, c in enumerate(need):
        table[i, :c] = order[at:at + c]
        at += c
    s = {"case": case, "table": table, "lengths": torch.tensor(lens, dtype=torch.int32, device=DEV), "wide": wide,
         "cu": _offsets([new] * n), "high": max(lens)}
    s["seq"], s["pos"] = _places([new] * n, [x - new for x in lens])
    if case["op"] != "append":
        s["q"] = (2.5 * torch.randn(n * new, case["heads"], d, generator=g, device=DEV)).to(dt)
    if case["op"] == "rank":
        s["mean"] = 0.3 * torch.randn(pages, hk, d, generator=g, device=DEV)
        return s

    def codes():
        # bfloat16 normal values about a quarter of e4m3's range wide
        return (100 * torch.randn(pages, hk, bs, d, generator=g, device=DEV, dtype=torch.bfloat16)).clamp_(-448, 448).to(torch.float8_e4m3fn)

    def scales():
        return torch.exp2(torch.randint(-8, -5, (pages, hk), generator=g, device=DEV).float())

    s |= {"k_cache": codes(), "v_cache": codes(), "k_scale": scales(), "v_scale": scales()}
    if case["op"] == "append":
        s["mean"] = torch.zeros(pages, hk, d, device=DEV)
        # most new tokens are of the size of what is there, some are larger and raise a page's scale
        big = 1 + 3 * (torch.rand(n * new, hk, 1, generator=g, device=DEV) < 0.02).float()
        s["k"] = (big * torch.randn(n * new, hk, d, generator=g, device=DEV)).to(dt)
        s["v"] = (big * torch.randn(n * new, hk, d, generator=g, device=DEV)).to(dt)
    elif case["select"]:
        # for each query and key head: the first and the last block, and others at random
        last = (s["pos"] // bs)[:, None, None]
        r = torch.rand(n * new, hk, wide, generator=g, device=DEV)
        block = torch.arange(wide, device=DEV)
        r = r.masked_fill((block == 0) | (block == last), 2.0).masked_fill(block > last, -1.0)
        best, picked = torch.topk(r, min(case["select"], wide), dim=2)
        picked = torch.where(best < 0, wide, picked).sort(2)[0]
        picked = torch.where(picked == wide, -1, picked).to(torch.int32)
        s["blocks"] = torch.nn.functional.pad(picked, (0, case["select"] - picked.shape[2]), value=-1).contiguous()
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    return _prepare_packed(case, g) if case["op"] in ("score", "prompt", "train") else _prepare_cache(case, g)


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "score":
        return _plain_score(state)
    if op == "rank":
        return _plain_rank(state)
    if op == "prompt":
        return _plain_attention(state)
    if op == "train":
        return _plain_train(state)
    if op == "append":
        return _plain_append(state)
    return _plain_decode(state)


def _run_own(s):
    import row_wise_top_topk_amd as mt
    case = s["case"]
    op, bs = case["op"], case["block"]
    if op == "score":
        means = mt.block_means(s["k"], bs, cu_seqlens=s["cuk"])
        scores, counts = mt.block_scores(s["q"], means, bs, s["blocks_most"], cu_seqlens=s["cu"], cu_seqlens_k=s["cuk"])
        return {"scores": scores, "counts": counts}
    if op == "rank":
        scores, counts = mt.block_scores(s["q"], s["mean"], bs, s["wide"], cu_seqlens=s["cu"], lengths=s["lengths"],
                                         block_table=s["table"])
        return {"scores": scores, "counts": counts}
    if op == "prompt":
        out, lse = mt.block_attention(s["q"], s["k"], s["v"], s["blocks"], bs, cu_seqlens=s["cu"], cu_seqlens_k=s["cuk"])
        return {"out": out, "lse": lse}
    if op == "train":
        q, k, v = (s[n].detach().requires_grad_() for n in ("q", "k", "v"))
        out, lse = mt.block_attention(q, k, v, s["blocks"], bs, cu_seqlens=s["cu"], cu_seqlens_k=s["cuk"])
        dq, dk, dv = torch.autograd.grad(out, (q, k, v), s["dout"])
        return {"out": out.detach(), "dq": dq, "dk": dk, "dv": dv}
    if op == "append":
        mt.kv8_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lengths"],
                      cu_seqlens=s["cu"], k_mean=s["mean"])
        return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale", "mean")}
    out, lse = mt.kv8_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lengths"],
                                cu_seqlens=s["cu"], blocks=s.get("blocks"), max_length=s["high"])
    return {"out": out, "lse": lse}


# The plain forms.


def _marked(scores, block, pos, bs):
    """Scores with +inf at the first block and at the query's own, -inf behind it, and how many are visible."""
    last = (pos // bs)[:, None, None]
    scores = scores.masked_fill((block == 0) | (block == last), math.inf).masked_fill(block > last, -math.inf)
    counts = (pos // bs + 1).to(torch.int32)[:, None].expand(scores.shape[:2]).contiguous()
    return {"scores": scores, "counts": counts}


def _plain_score(s):
    case, q, k = s["case"], s["q"], s["k"]
    t, h, d = q.shape
    hk, bs, nb, rows = case["kv_heads"], case["block"], s["blocks_most"], s["plain_rows"]
    base = s["cuk"][s["kseq"]] // bs + s["kseq"]
    row = base + s["kpos"] // bs
    total = torch.zeros(rows, hk, d, device=DEV, dtype=torch.float64).index_add_(0, row, k.double())
    mean = (total / torch.bincount(row, minlength=rows).clamp_min(1)[:, None, None]).float()
    g = h // hk
    a = q.float().view(t, hk, g, d).permute(1, 0, 2, 3).reshape(hk, t * g, d)
    best = torch.matmul(a, mean.permute(1, 2, 0).contiguous()).view(hk, t, g, rows).amax(2) * (1 / math.sqrt(d))
    block = torch.arange(nb, device=DEV)
    at = ((s["cuk"][s["seq"]] // bs + s["seq"])[:, None] + block).clamp_max(rows - 1)
    scores = best.gather(2, at.expand(hk, t, nb)).permute(1, 0, 2)
    return _marked(scores, block, s["pos"], bs)


def _plain_rank(s):
    case, q = s["case"], s["q"]
    t, h, d = q.shape
    hk, bs, n, new = case["kv_heads"], case["block"], case["seqs"], case["new"]
    mean = s["mean"][s["table"].long()].permute(0, 2, 3, 1).contiguous()  # [seqs, kv_heads, dim, blocks]
    a = q.float().view(n, new, hk, h // hk, d).permute(0, 2, 1, 3, 4).reshape(n, hk, new * (h // hk), d)
    best = torch.matmul(a, mean).view(n, hk, new, h // hk, -1).amax(3) * (1 / math.sqrt(d))
    scores = best.permute(0, 2, 1, 3).reshape(t, hk, -1)
    return _marked(scores, torch.arange(s["wide"], device=DEV), s["pos"], bs)


def _allowed(s):
    """[kv_heads, queries, keys]: whether the query sees the key."""
    nb, hk, t = s["blocks_most"], s["case"]["kv_heads"], s["q"].shape[0]
    picked = s["blocks"].permute(1, 0, 2).long()
    chosen = torch.zeros(hk, t, nb + 1, dtype=torch.bool, device=DEV)
    chosen.scatter_(2, torch.where(picked < 0, nb, picked), True)
    seen = chosen[:, :, s["kpos"] // s["case"]["block"]]
    return seen & (s["seq"][:, None] == s["kseq"]) & (s["kpos"] <= s["pos"][:, None])


def _heads_first(x, hk):
    t, h, d = x.shape
    return x.float().view(t, hk, h // hk, d).permute(1, 2, 0, 3).reshape(hk, (h // hk) * t, d)


def _tokens_first(x, t):
    hk, gt, d = x.shape
    return x.view(hk, gt // t, t, d).permute(2, 0, 1, 3).reshape(t, hk * (gt // t), d)


def _softmax(s, q, kt):
    """Probabilities and log-sums of the masked scores; a row without keys has zeros and -inf."""
    hk, t = s["case"]["kv_heads"], s["q"].shape[0]
    p = torch.matmul(q, kt).mul_(1 / math.sqrt(q.shape[2]))
    p = p.view(hk, -1, t, kt.shape[2]).masked_fill_(~_allowed(s)[:, None], -math.inf)
    most = p.amax(3, keepdim=True).clamp_min(-3e38)
    p = p.sub_(most).exp_()
    total = p.sum(3, keepdim=True)
    p = p.div_(total.clamp_min(1e-38)).view(hk, -1, kt.shape[2])
    lse = (most + total.log()).view(hk, -1, 1)
    return p, _tokens_first(lse, t)[:, :, 0]


def _plain_attention(s):
    q, v = _heads_first(s["q"], s["case"]["kv_heads"]), s["v"].float().transpose(0, 1).contiguous()
    p, lse = _softmax(s, q, s["k"].float().permute(1, 2, 0).contiguous())
    return {"out": _tokens_first(torch.matmul(p, v), s["q"].shape[0]).to(s["q"].dtype), "lse": lse}


def _plain_train(s):
    t, dt = s["q"].shape[0], s["q"].dtype
    q, do = (_heads_first(s[n], s["case"]["kv_heads"]) for n in ("q", "dout"))
    k, v = (s[n].float().transpose(0, 1).contiguous() for n in ("k", "v"))
    p, _ = _softmax(s, q, k.transpose(1, 2).contiguous())
    out = torch.matmul(p, v)
    dv = torch.matmul(p.transpose(1, 2), do)
    dp = torch.matmul(do, v.transpose(1, 2))
    ds = dp.sub_((out * do).sum(2, keepdim=True)).mul_(p).mul_(1 / math.sqrt(q.shape[2]))
    dq, dk = torch.matmul(ds, k), torch.matmul(ds.transpose(1, 2), q)
    return {"out": _tokens_first(out, t).to(dt), "dq": _tokens_first(dq, t).to(dt),
            "dk": dk.transpose(0, 1).to(dt), "dv": dv.transpose(0, 1).to(dt)}


def _scale_for(most):
    """The smallest power of two that brings ``most`` to 448 or less, 2^-60 at least."""
    f, x = torch.frexp(most)  # most = f * 2^x, f in [0.5, 1); 448 = 0.875 * 2^9
    return torch.ldexp(torch.ones_like(f), (x - 9 + (f > 0.875)).clamp_min(-60))


def _plain_append(s):
    case, bs, hk = s["case"], s["case"]["block"], s["case"]["kv_heads"]
    pages, n = s["k_cache"].shape[0], case["seqs"]
    start = s["lengths"].long() - case["new"]
    page = s["table"][s["seq"], s["pos"] // bs].long()
    # the touched pages, one row each: [seqs, blocks that new tokens may reach]
    reach = (case["new"] + bs - 2) // bs + 1
    block = (start // bs)[:, None] + torch.arange(reach, device=DEV)
    live = block * bs < s["lengths"][:, None]
    touched = s["table"].gather(1, block.clamp_max(s["wide"] - 1)).long()[live]
    first = (block * bs)[live]
    held = (start[:, None].expand_as(block)[live] - first).clamp(0, bs)  # tokens that the page held before
    there = (s["lengths"][:, None].expand_as(block)[live] - first).clamp(0, bs)
    slot = torch.arange(bs, device=DEV)

    def one(x, cache, scale):
        most = torch.zeros(pages, hk, device=DEV)
        most.scatter_reduce_(0, page[:, None].expand(-1, hk), x.float().abs().amax(2), "amax")
        now = _scale_for(most)[touched]
        now = torch.where((held > 0)[:, None], torch.maximum(now, scale[touched]), now)
        rows = cache[touched].float() * scale[touched][:, :, None, None]
        stay = (slot < held[:, None])[:, None, :, None]
        wide = (rows / now[:, :, None, None]).clamp(-448, 448)
        codes = torch.where(stay, wide, cache[touched].float()).to(torch.float8_e4m3fn)
        cache[touched] = codes
        scale[touched] = now
        cache[page, :, s["pos"] % bs] = (x.float() / scale[page][:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)

    one(s["k"], s["k_cache"], s["k_scale"])
    one(s["v"], s["v_cache"], s["v_scale"])
    rows = s["k_cache"][touched].float() * (slot < there[:, None])[:, None, :, None]
    s["mean"][touched] = rows.sum(2) * s["k_scale"][touched][:, :, None] / there[:, None, None]
    return {x: s[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale", "mean")}


def _plain_decode(s):
    case, q = s["case"], s["q"]
    t, h, d = q.shape
    hk, bs, n, new = case["kv_heads"], case["block"], case["seqs"], case["new"]
    if case["select"]:
        blocks = s["blocks"].long()
        page = s["table"][s["seq"][:, None, None], blocks.clamp_min(0)].long()
        head = torch.arange(hk, device=DEV)[None, :, None]
        k = s["k_cache"][page, head].float() * s["k_scale"][page, head][..., None, None]
        v = s["v_cache"][page, head].float() * s["v_scale"][page, head][..., None, None]
        at = blocks[..., None] * bs + torch.arange(bs, device=DEV)
        seen = ((blocks >= 0)[..., None] & (at <= s["pos"][:, None, None, None])).view(t, hk, 1, -1)
        a = q.float().view(t, hk, h // hk, d)
        k, v = k.view(t, hk, -1, d), v.view(t, hk, -1, d)
    else:
        table = s["table"].long()
        k = (s["k_cache"][table].float() * s["k_scale"][table][..., None, None]).transpose(1, 2).reshape(n, hk, -1, d)
        v = (s["v_cache"][table].float() * s["v_scale"][table][..., None, None]).transpose(1, 2).reshape(n, hk, -1, d)
        at = torch.arange(k.shape[2], device=DEV)
        seen = (at <= s["pos"].view(n, 1, new, 1, 1)).expand(n, hk, new, h // hk, -1).reshape(n, hk, -1, k.shape[2])
        a = q.float().view(n, new, hk, h // hk, d).permute(0, 2, 1, 3, 4).reshape(n, hk, -1, d)
    p = torch.matmul(a, k.transpose(2, 3).contiguous()).mul_(1 / math.sqrt(d)).masked_fill_(~seen, -math.inf)
    most = p.amax(3, keepdim=True).clamp_min(-3e38)
    p = p.sub_(most).exp_()
    total = p.sum(3, keepdim=True)
    out, lse = torch.matmul(p, v) / total.clamp_min(1e-38), (most + total.log())[..., 0]
    if not case["select"]:
        out = out.view(n, hk, new, h // hk, d).permute(0, 2, 1, 3, 4)
        lse = lse.view(n, hk, new, h // hk).permute(0, 2, 1, 3)
    return {"out": out.reshape(t, h, d).to(q.dtype), "lse": lse.reshape(t, h)}


# The definitions in 64 bits, a sequence, a head or a request at a time.


def _exact_score(s):
    case, bs, hk = s["case"], s["case"]["block"], s["case"]["kv_heads"]
    ql, kl = _ints(case["q_lens"]), _ints(case["k_lens"])
    t, h, d = s["q"].shape
    scores = torch.full((t, hk, s["blocks_most"]), -math.inf, dtype=torch.float64, device=DEV)
    counts = torch.zeros(t, hk, dtype=torch.int32, device=DEV)
    a = b = 0
    for n, m in zip(ql, kl):
        k, q = s["k"][b:b + m].double(), s["q"][a:a + n].double().view(n, hk, h // hk, d)
        pos = torch.arange(m - n, m, device=DEV)
        for j in range(-(-m // bs) if n else 0):
            mean = k[j * bs:(j + 1) * bs].mean(0)
            x = (q * mean[None, :, None]).sum(3).amax(2) / math.sqrt(d)
            own_block = (pos // bs == j) | (j == 0)
            x[own_block] = math.inf
            x[pos < j * bs] = -math.inf
            scores[a:a + n, :, j] = x
        counts[a:a + n] = (pos // bs + 1).to(torch.int32)[:, None]
        a, b = a + n, b + m
    return {"scores": scores, "counts": counts}


def _exact_rank(s):
    case, bs, hk, new = s["case"], s["case"]["block"], s["case"]["kv_heads"], s["case"]["new"]
    t, h, d = s["q"].shape
    scores = torch.full((t, hk, s["wide"]), -math.inf, dtype=torch.float64, device=DEV)
    counts = torch.zeros(t, hk, dtype=torch.int32, device=DEV)
    for i, n in enumerate(_lengths(case)):
        for r in range(new):
            row, last = i * new + r, (n - new + r) // bs
            mean = s["mean"][s["table"][i, :last + 1].long()].double()
            x = (s["q"][row].double().view(1, hk, h // hk, d) * mean[:, :, None]).sum(3).amax(2) / math.sqrt(d)
            scores[row, :, :last + 1] = x.T
            scores[row, :, 0] = scores[row, :, last] = math.inf
            counts[row] = last + 1
    return {"scores": scores, "counts": counts}


def _exact_attention(s, gradient):
    case, bs, hk = s["case"], s["case"]["block"], s["case"]["kv_heads"]
    ql, kl = _ints(case["q_lens"]), _ints(case["k_lens"])
    t, h, d = s["q"].shape
    g, scale = h // hk, 1 / math.sqrt(d)
    zeros = lambda like: torch.zeros(like.shape, dtype=torch.float64, device=DEV)  # noqa: E731
    out, dq, dk, dv = zeros(s["q"]), zeros(s["q"]), zeros(s["k"]), zeros(s["v"])
    lse = torch.full((t, h), -math.inf, dtype=torch.float64, device=DEV)
    a = b = 0
    for n, m in zip(ql, kl):
        step = max(1, min(n, 40_000_000 // max(m, 1)))
        for c in range(hk):
            k, v = s["k"][b:b + m, c].double(), s["v"][b:b + m, c].double()
            for x in range(0, n, step):
                y = min(n, x + step)
                rows = slice(a + x, a + y)
                pos = torch.arange(m - n + x, m - n + y, device=DEV)[:, None]
                own_blocks = s["blocks"][rows, c].long()
                seen = torch.zeros(y - x, -(-m // bs) + 1, dtype=torch.bool, device=DEV)
                seen.scatter_(1, own_blocks.masked_fill(own_blocks < 0, seen.shape[1] - 1), True)
                key = torch.arange(m, device=DEV)
                seen = seen[:, key // bs] & (key <= pos)
                for i in range(c * g, (c + 1) * g):
                    q = s["q"][rows, i].double()
                    z = (q @ k.T * scale).masked_fill(~seen, -math.inf)
                    lse[rows, i] = torch.logsumexp(z, 1)
                    p = torch.exp(z - lse[rows, i].clamp_min(-1e300)[:, None])
                    out[rows, i] = p @ v
                    if gradient:
                        do = s["dout"][rows, i].double()
                        dv[b:b + m, c] += p.T @ do
                        ds = p * (do @ v.T - (do * out[rows, i]).sum(1, keepdim=True)) * scale
                        dq[rows, i] = ds @ k
                        dk[b:b + m, c] += ds.T @ q
        a, b = a + n, b + m
    return {"out": out, "dq": dq, "dk": dk, "dv": dv} if gradient else {"out": out, "lse": lse}


def _exact_append(s):
    """Only the means are sums; the codes and scales have no value between their steps."""
    case, bs = s["case"], s["case"]["block"]
    mean = s["mean"].double()
    kept = _plain_append(s)  # the codes as they are held afterwards
    for i, n in enumerate(_lengths(case)):
        for b in range((n - case["new"]) // bs, (n - 1) // bs + 1):
            page = s["table"][i, b].long()
            rows = kept["k_cache"][page][:, :min(bs, n - b * bs)].double()
            mean[page] = rows.mean(1) * kept["k_scale"][page].double()[:, None]
    return {"k_cache": None, "v_cache": None, "k_scale": None, "v_scale": None, "mean": mean}


def _exact_decode(s):
    case, bs, hk, new = s["case"], s["case"]["block"], s["case"]["kv_heads"], s["case"]["new"]
    t, h, d = s["q"].shape
    out = torch.zeros(t, h, d, dtype=torch.float64, device=DEV)
    lse = torch.full((t, h), -math.inf, dtype=torch.float64, device=DEV)
    for i, n in enumerate(_lengths(case)):
        for c in range(hk):
            heads = slice(c * (h // hk), (c + 1) * (h // hk))
            whole = torch.arange(-(-n // bs), device=DEV)
            for r in range(new):
                row = i * new + r
                block = s["blocks"][row, c].long() if case["select"] else whole
                block = block[block >= 0]
                page = s["table"][i, block].long()
                k = (s["k_cache"][page, c].double() * s["k_scale"][page, c].double()[:, None, None]).reshape(-1, d)
                v = (s["v_cache"][page, c].double() * s["v_scale"][page, c].double()[:, None, None]).reshape(-1, d)
                at = (block[:, None] * bs + torch.arange(bs, device=DEV)).reshape(-1)
                z = (s["q"][row, heads].double() @ k.T / math.sqrt(d)).masked_fill(at > n - new + r, -math.inf)
                lse[row, heads] = torch.logsumexp(z, 1)
                out[row, heads] = torch.softmax(z, 1) @ v
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "score":
        return _exact_score(s)
    if op == "rank":
        return _exact_rank(s)
    if op in ("prompt", "train"):
        return _exact_attention(s, op == "train")
    return _exact_append(s) if op == "append" else _exact_decode(s)


def _visible(case):
    """Keys seen by all queries of one head: whole selected blocks and the own one up to the query."""
    total = 0
    for n, m in zip(_ints(case["q_lens"]), _ints(case["k_lens"])):
        bs = case["block"]
        for p in range(m - n, m):
            total += min(p // bs, max(1, case["select"]) - 1) * bs + p % bs + 1
    return total


def work(case):
    op, hk, d, bs = case["op"], case["kv_heads"], case["dim"], case["block"]
    h = case.get("heads", hk)
    if op in ("score", "prompt", "train"):
        ql, kl = _ints(case["q_lens"]), _ints(case["k_lens"])
        t, tk = sum(ql), sum(kl)
        if op == "score":
            nb = max(1, -(-max(kl) // bs))
            pairs = sum(p // bs + 1 for n, m in zip(ql, kl) for p in range(m - n, m))
            return {"bytes": 2 * (t * h + tk * hk) * d + 4 * t * hk * (nb + 1), "flops": 2 * pairs * h * d + tk * hk * d}
        seen = _visible(case) * h
        io = 2 * (2 * t * h + 2 * tk * hk) * d + 4 * t * hk * case["select"]
        if op == "prompt":
            return {"bytes": io + 4 * t * h, "flops": 4 * seen * d}
        return {"bytes": 2 * io, "flops": 14 * seen * d}
    lens, new = _lengths(case), case["new"]
    t = case["seqs"] * new
    if op == "rank":
        nb = sum(-(-n // bs) for n in lens)
        wide = max(-(-n // bs) for n in lens)
        return {"bytes": 2 * t * h * d + 4 * nb * hk * d + 4 * t * hk * (wide + 1) + 4 * nb, "flops": 2 * nb * new * h * d}
    if op == "append":
        held = sum((n - new) % bs for n in lens)
        touched = sum((n - 1) // bs - (n - new) // bs + 1 for n in lens)
        # new rows in and out, the keys that the first pages hold, scales and means
        return {"bytes": 2 * t * hk * d * 3 + held * hk * d + touched * hk * (16 + 4 * d), "flops": 4 * t * hk * d}
    seen = sum(min(n, case["select"] * bs) if case["select"] else n for n in lens)
    rows = seen * (new if case["select"] else 1)
    return {"bytes": 2 * rows * hk * d + 4 * t * h * d + 4 * t * h + (8 * hk + 4) * rows // bs, "flops": 4 * seen * new * h * d}
