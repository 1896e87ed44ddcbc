"""What the attention operators decide on the host: no GPU needed."""

import ctypes
import sys
import threading

import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import row_wise_top_topk_amd as mt
from row_wise_top_topk_amd import attention as binding


def test_forward_mode_derivatives_are_refused():
    """A tangent would be dropped without a word."""
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    blocks = torch.zeros(4, 2, 1, dtype=torch.int32)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        calls = [lambda: mt.block_means(dual, 16), lambda: mt.block_scores(dual, x.float(), 16, 1),
                 lambda: mt.block_attention(dual, x, x, blocks, 16),
                 lambda: mt.block_attention_backward(x, dual, x, x, x, None, blocks, 16),
                 lambda: mt.kv8_append(dual, x, *[None] * 6), lambda: mt.kv8_attention(dual, *[None] * 6)]
        for call in calls:
            with pytest.raises(ValueError, match="forward-mode"):
                call()
        # the operands themselves are looked at: a primal of a level has no tangent
        with pytest.raises(ValueError, match="GPU"):
            mt.block_means(forward_ad.unpack_dual(dual).primal, 16)


def test_the_node_that_sums_a_leafs_gradients():
    """It keeps the stream of the first living graph, also when that graph goes before the others."""
    x, y = torch.zeros(4), torch.zeros(4)
    first = binding._summed([x], 1)
    second = binding._summed([y, x], 2)
    assert second[1] is first[0] and [n.stream for n in second] == [2, 1]
    del first
    third = binding._summed([x], 2)
    assert third[0].stream == 1
    with pytest.raises(RuntimeError, match="captured"):
        binding._check_capture(third, 2)
    binding._check_capture(third, 1)
    del second, third
    assert len(binding._summing) == 0
    assert [n.stream for n in binding._summed([x], 2)] == [2]
    assert len(binding._summing) == 0
    other = binding._summed([x], 3)
    binding._summing[id(y)] = other[0]                    # what a reused id would look like
    assert [n.stream for n in binding._summed([y], 4)] == [4]


def test_threads_of_graphs():
    """Graphs that come and go in several threads while others look them up."""
    leaves = [torch.zeros(1) for _ in range(3)]
    errors, interval = [], sys.getswitchinterval()

    def work(stream):
        try:
            kept = []
            for i in range(4000):
                kept.append(binding._summed(leaves if stream else leaves[:1], stream))
                binding._check_capture(kept[-1][:1], kept[-1][0].stream)
                if i % 50 == stream:
                    kept.clear()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=work, args=(s,)) for s in range(4)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    assert not errors and len(binding._summing) == 0


def decode(total_q, columns, max_length=None, heads=64, kv_heads=8, dim=128, block_size=64, num_seqs=1, select=0):
    a = binding._DecodeArgs()
    for name in ("q", "k_cache", "v_cache", "k_scale", "v_scale", "block_table", "lengths", "cu", "out", "lse"):
        setattr(a, name, 1 << 20)
    a.blocks, a.select = (1 << 20, select) if select else (0, 0)
    a.q_stride_t, a.q_stride_h, a.total_q, a.num_pages = heads * dim, dim, total_q, 1 << 20
    a.block_table_cols = a.block_table_stride = columns
    a.max_length = columns * block_size if max_length is None else max_length
    a.dtype, a.num_seqs, a.heads, a.kv_heads, a.dim, a.block_size, a.scale = 0, num_seqs, heads, kv_heads, dim, block_size, 0.1
    return mt.load_library().kv8_attention_workspace(ctypes.byref(a))


def test_the_largest_bound_of_the_lengths():
    """A bound past what the table can hold is the table's."""
    want = decode(4, 1000)
    assert want > 0
    for n in (64000, 64001, 1 << 32, (1 << 63) - 64, (1 << 63) - 1):
        assert decode(4, 1000, max_length=n) == want


def test_the_workspace_of_many_tokens_is_bounded():
    """Many new tokens fill the card by themselves: their chunks are longer, so that the partial results stay below a
    fixed size whatever the table can hold (2^19 rows of dim + 2 floats), and a large call needs none.  Where sequences
    have few tokens there may be 32 results for each row."""
    bound = (1 << 19) * (128 + 2) * 4
    for columns in (1, 100, 2048, 14063, (1 << 24) - 1):        # pages of 64: up to 2^30 tokens
        for total_q in (1, 7, 64, 500, 2048, 4095, 8192, 32768, 1 << 20):
            for heads, kv in ((64, 8), (8, 8), (128, 1), (32, 2), (30, 3)):
                for seqs in (1, 3, 64, 1024):
                    for select in (0, 32):
                        if seqs <= total_q:
                            got = decode(total_q, columns, heads=heads, kv_heads=kv, num_seqs=seqs, select=select)
                            rows = total_q * heads + 2 * 128 * kv * seqs if total_q < 64 * seqs else 0
                            assert got <= max(bound, 32 * rows * 130 * 4), (columns, total_q, heads, kv, seqs, select, got)
    for total_q in (8192, 32768):
        for columns in (2048, 14063):
            assert decode(total_q, columns) <= 2 * total_q * 64 * 128
    for heads, seqs in ((8, 0), (64, 0), (64, 3), (1024, 2)):
        assert decode(0, 2048, heads=heads, num_seqs=seqs) <= bound
    # a decode batch keeps its chunks
    assert decode(64, 500, num_seqs=64) == (64 // 2 + 64 + 1) * 8 * 8 * 16 * 130 * 4
