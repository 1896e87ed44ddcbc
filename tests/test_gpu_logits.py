"""GPU: penalties, biases and masks on rows of logits, against a plain 64-bit form.

Four roundings to 32 bits at most (the quotient or product, two differences, the
sum with the bias; a product that is fused with a difference has none), each half
a step of an intermediate that is at most the sum of the terms' sizes: 4 2^-24 of
that sum.
"""

import math

import pytest
import torch

import row_wise_top_topk_amd as mt
import serving_oracle as oracle

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def build(seed, rows, vocab, cols, dtype, bias=0, mask=False):
    g = torch.Generator().manual_seed(seed)
    x = {"logits": (4 * torch.randn(rows, vocab, generator=g)).to(dtype),
         "tokens": torch.randint(-1, vocab + 2, (rows, cols), generator=g).to(torch.int32),
         "lengths": torch.randint(-1, cols + 3, (rows,), generator=g).to(torch.int32),
         "prompt_lengths": torch.randint(-1, cols + 3, (rows,), generator=g).to(torch.int32),
         "repetition": 0.7 + torch.rand(rows, generator=g), "presence": torch.rand(rows, generator=g) - 0.3,
         "frequency": torch.rand(rows, generator=g) - 0.3}
    if cols:  # ids that come often
        x["tokens"][:, ::3] = torch.randint(0, min(vocab, 5), (rows, -(-cols // 3)), generator=g).to(torch.int32)
    if bias:
        x["bias_ids"] = torch.randint(-2, vocab + 3, (rows, bias), generator=g).to(torch.int32)
        x["bias"] = 5 * torch.randn(rows, bias, generator=g)
    if mask:
        x["mask"] = torch.randint(-2 ** 31, 2 ** 31, (rows, -(-vocab // 32)), generator=g).to(torch.int32)
    return x


def put(x):
    return {n: t.to(DEV) for n, t in x.items()}


def expect(x):
    names = {"lengths": "lengths", "prompt_lengths": "prompts"}
    return oracle.penalize(**{names.get(n, n): t for n, t in x.items()})


def check(x, got):
    want = expect(x)
    got = got.cpu()
    assert got.dtype == torch.float32 and got.shape == want.shape
    size = x["logits"].double().abs() * 4
    if "tokens" in x:
        big = max((float(x[n].abs().max()) if n in x and x[n].numel() else 0.0) for n in ("presence", "frequency"))
        size = size + big * (x["tokens"].shape[1] + 1)
    if "bias" in x and x["bias"].numel():
        size = size + float(x["bias"].abs().max())
    same = (got.double() == want) | (torch.isnan(got) & torch.isnan(want))
    assert torch.all(same | ((got.double() - want).abs() <= 4 * 2 ** -24 * size))
    if not any(n in x for n in ("tokens", "bias")):
        assert torch.all(same)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab,cols,bias,mask", [
    (1, 1, 1, 0, False), (3, 5, 4, 2, True), (2, 31, 0, 0, True), (4, 64, 9, 0, False), (3, 257, 40, 7, True), (2, 8191, 300, 0, True),
    (2, 8192, 1000, 33, False), (3, 8193, 100, 1, True), (2, 32003, 700, 1023, True), (1, 151937, 5000, 20, True), (40, 1000, 17, 3, True),
])
def test_rows(dtype, rows, vocab, cols, bias, mask):
    x = build(vocab, rows, vocab, cols, dtype, bias, mask)
    check(x, mt.penalize_logits(**put(x)))


@pytest.mark.parametrize("dtype", TYPES)
def test_each_part_alone(dtype):
    x = build(1, 3, 777, 50, dtype, 9, True)
    for names in ((), ("tokens",), ("tokens", "repetition"), ("tokens", "presence"), ("tokens", "frequency", "lengths"),
                  ("tokens", "prompt_lengths", "frequency", "repetition"), ("bias_ids", "bias"), ("mask",), ("mask", "bias_ids", "bias")):
        part = {n: x[n] for n in ("logits",) + names}
        check(part, mt.penalize_logits(**put(part)))


def test_rows_of_no_use_are_left_alone():
    x = build(2, 5, 100, 8, torch.float32, 4, True)
    for n in ("tokens", "bias_ids", "bias"):
        x[n] = x[n][:, :0]
    check(x, mt.penalize_logits(**put(x)))
    for rows, vocab in ((0, 10), (3, 0)):
        y = mt.penalize_logits(torch.zeros(rows, vocab, device=DEV), mask=torch.zeros(rows, -(-vocab // 32), dtype=torch.int32, device=DEV))
        assert y.shape == (rows, vocab)


def test_special_values():
    vocab = 64
    x = {"logits": torch.zeros(2, vocab), "tokens": torch.arange(vocab, dtype=torch.int32).repeat(2, 1), "repetition": torch.tensor([2.0, 0.5]),
         "frequency": torch.tensor([0.5, 0.25]), "mask": torch.tensor([[-1, 1], [0, 0]], dtype=torch.int32)}
    x["logits"][:, :6] = torch.tensor([math.inf, -math.inf, math.nan, torch.finfo(torch.float32).min, -0.0, 1e-45])
    got = mt.penalize_logits(**put(x)).cpu()
    assert got[0, 0] == math.inf and got[0, 1] == -math.inf and torch.isnan(got[0, 2]) and got[0, 3] == -math.inf
    assert torch.isneginf(got[1]).all()                   # a mask that allows nothing
    assert torch.isneginf(got[0, 33:]).all() and torch.isfinite(got[0, 6:33]).all()


def test_repetitions_at_the_ends_of_their_range():
    # the product of 1 / r, rounded, and x is within 2^-23 of the quotient, and below the
    # least normal number each rounding is within 2^-150
    values = torch.tensor([1.0, 1e-5, 3e38, 3e-39, 1e-45, 0.0, -1.0, -1e-5, -3e38, -3e-39, math.inf, -math.inf])
    factors = torch.tensor([1e-39, 1e-45, 2e-38, 1.0, 1.5e38, 3e38, 0.0, math.inf])
    x = {"logits": values.repeat(len(factors), 1), "tokens": torch.arange(len(values), dtype=torch.int32).repeat(len(factors), 1),
         "repetition": factors}
    got = mt.penalize_logits(**put(x)).cpu().double()
    y, r = x["logits"].double(), factors.double()[:, None]
    want = torch.where(y > 0, y / r, y * r)
    large = want.abs() > torch.finfo(torch.float32).max * (1 + 2 ** -25)
    want = torch.where(large, want.sign() * math.inf, want)
    same = (got == want) | (got.isnan() & want.isnan())
    off = (got - want).abs() <= want.abs() * 2 ** -22 + 2 ** -149
    assert (same | (off & torch.isfinite(want))).all(), (got, want)


def test_the_last_bias_of_an_id_counts():
    x = {"logits": torch.zeros(1, 10), "bias_ids": torch.tensor([[3, 3, 4, 3, 4]], dtype=torch.int32),
         "bias": torch.tensor([[1.0, 2.0, 3.0, 4.0, 5.0]])}
    got = mt.penalize_logits(**put(x)).cpu()
    assert got[0].tolist() == [0, 0, 0, 4, 5, 0, 0, 0, 0, 0]


def test_counts_up_to_the_limit():
    # one id, 2^21 - 1 times
    n = (1 << 21) - 1
    tokens = torch.full((1, n), 7, dtype=torch.int32, device=DEV)
    got = mt.penalize_logits(torch.zeros(1, 16, device=DEV), tokens, frequency=torch.ones(1, device=DEV), bias=torch.ones(1, 1, device=DEV),
                             bias_ids=torch.full((1, 1), 7, dtype=torch.int32, device=DEV))
    assert got[0].tolist() == [0] * 7 + [1 - n] + [0] * 8
    with pytest.raises(ValueError, match="columns"):
        mt.penalize_logits(torch.zeros(1, 16, device=DEV), torch.cat([tokens, tokens[:, :1]], 1))


@pytest.mark.parametrize("dtype", TYPES)
def test_strides(dtype):
    x = build(4, 5, 1001, 33, dtype, 6, True)
    dev = put(x)
    for n in ("logits", "tokens", "bias_ids", "bias", "mask"):   # rows 3 entries apart from each other, from an odd address
        t = dev[n]
        wide = torch.zeros(t.shape[0], t.shape[1] + 3, dtype=t.dtype, device=DEV)
        wide[:, 1:-2] = t
        dev[n] = wide[:, 1:-2]
    out = torch.full((5, 1010), 7.5, device=DEV)
    got = mt.penalize_logits(**dev, out=out[:, 2:1003])
    assert got.data_ptr() == out[:, 2:].data_ptr() and (out[:, :2] == 7.5).all() and (out[:, 1003:] == 7.5).all()
    check(x, got)
    x["tokens"] = x["tokens"][:1].expand(5, 33)      # one list for all rows
    check(x, mt.penalize_logits(**(put(x) | {"tokens": x["tokens"][:1].to(DEV).expand(5, 33)})))


def test_in_place():
    x = build(5, 4, 3333, 60, torch.float32, 5, True)
    dev = put(x)
    got = mt.penalize_logits(**dev, out=dev["logits"])
    assert got is dev["logits"]
    check(x, got)


def test_rows_past_32_bits():
    # rows 2^30 elements apart
    rows, vocab, apart = 4, 100, 1 << 30
    buf = torch.zeros(rows * apart, dtype=torch.bfloat16, device=DEV)
    x = build(6, rows, vocab, 12, torch.bfloat16)
    dev = put(x)
    dev["logits"] = buf.view(rows, apart)[:, :vocab]
    dev["logits"].copy_(x["logits"])
    check(x, mt.penalize_logits(**dev))


def test_ranked_by_value():
    # the rows as topk_indices takes them: candidates of a sampler
    x = build(7, 6, 5000, 200, torch.bfloat16, 10, True)
    rows = mt.penalize_logits(**put(x))
    best = mt.topk_indices(rows, torch.full((6,), 5000, dtype=torch.int32, device=DEV), 20, order="value").cpu().long()
    want = expect(x)
    picked = want.gather(1, best)
    assert torch.allclose(picked, want.topk(20)[0], atol=1e-4) and torch.isfinite(picked).all()


def test_refusals():
    x = put(build(8, 3, 100, 7, torch.float32, 2, True))
    one = torch.ones(1, device=DEV)
    for bad in (dict(logits=x["logits"][0]), dict(logits=x["logits"].t()), dict(logits=x["logits"].double()), dict(tokens=x["tokens"].long()),
                dict(tokens=x["tokens"][:2]), dict(tokens=x["tokens"].cpu()), dict(lengths=x["lengths"][:2]), dict(lengths=x["lengths"].long()),
                dict(prompt_lengths=x["lengths"][:1]), dict(repetition=one), dict(presence=x["presence"].double()), dict(frequency=one),
                dict(bias=None), dict(bias_ids=None), dict(bias=x["bias"][:, :1]), dict(bias_ids=x["bias_ids"].long()), dict(mask=x["mask"][:, :3]),
                dict(mask=x["mask"].long()), dict(out=torch.empty(3, 99, device=DEV)), dict(out=torch.empty(3, 100, device=DEV).half()),
                dict(out=torch.empty(1, 100, device=DEV).expand(3, 100)), dict(tokens=None), dict(tokens=None, lengths=None, prompt_lengths=None)):
        with pytest.raises(ValueError):
            mt.penalize_logits(**(x | bad))
