"""Block scores, block sparse attention and the 8-bit paged cache: what produces
the rows that ``topk_indices`` selects from, and what reads the blocks that it
selects.

Argument marshalling only, as in the package's other functions: every step
runs in the library's HIP kernels on the current stream of the tensors'
device.  Outputs and scratch memory come from PyTorch's allocator, so a call
can be captured into a graph, and two graphs share nothing.

    means = block_means(k, 64)
    scores, counts = block_scores(q, means, 64, max_blocks)
    blocks = topk_indices(scores.flatten(0, 1), counts.flatten(), 16)
    out, lse = block_attention(q, k, v, blocks.view(tokens, kv_heads, 16), 64)

Packed sequences: ``cu_seqlens`` (int32, one entry more than sequences, first
0, not decreasing, on the device) gives each sequence's queries,
``cu_seqlens_k`` its keys (default: the same).  Query r of a sequence with n
queries and m keys stands at position ``m - n + r``.
"""

from __future__ import annotations

import ctypes
import math
import threading
import weakref

import torch
import torch.autograd.forward_ad as _forward_ad

__all__ = ["block_means", "block_scores", "block_attention", "block_attention_backward", "kv8_append", "kv8_attention"]

BLOCK_SIZES = (16, 32, 64, 128)
HEAD_DIMS = (64, 128)
MAX_SELECT = 1024
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_STATUS = {1: "invalid argument", 2: "workspace too small", 3: "kernel launch failed"}

_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class _ScoreArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("q", "means", "cu_q", "cu_k", "lengths", "block_table", "scores", "counts")]
                + [(n, _i64) for n in ("q_stride_t", "q_stride_h", "total_q", "total_k", "mean_rows", "block_table_stride")]
                + [(n, _i32) for n in ("dtype", "num_seqs", "heads", "kv_heads", "dim", "block_size", "max_blocks",
                                       "first", "last")]
                + [("scale", _f32)])


class _AttentionArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("q", "k", "v", "blocks", "cu_q", "cu_k", "out", "rest", "lse", "dout", "dq", "dk",
                                    "dv", "workspace")]
                + [("workspace_bytes", ctypes.c_uint64)]
                + [(n, _i64) for n in ("q_stride_t", "q_stride_h", "k_stride_t", "k_stride_h", "v_stride_t", "v_stride_h",
                                       "dout_stride_t", "dout_stride_h", "total_q", "total_k")]
                + [(n, _i32) for n in ("dtype", "num_seqs", "heads", "kv_heads", "dim", "block_size", "select", "causal")]
                + [("scale", _f32)])


class _AppendArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("k", "v", "k_cache", "v_cache", "k_scale", "v_scale", "k_mean", "block_table", "lengths",
                                    "cu")]
                + [(n, _i64) for n in ("k_stride_t", "k_stride_h", "v_stride_t", "v_stride_h", "total", "num_pages",
                                       "block_table_stride")]
                + [(n, _i32) for n in ("block_table_cols", "dtype", "num_seqs", "kv_heads", "dim", "block_size")])


class _DecodeArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("q", "k_cache", "v_cache", "k_scale", "v_scale", "block_table", "lengths", "cu", "blocks",
                                    "out", "lse", "workspace")]
                + [("workspace_bytes", ctypes.c_uint64)]
                + [(n, _i64) for n in ("q_stride_t", "q_stride_h", "total_q", "num_pages", "block_table_stride", "max_length")]
                + [(n, _i32) for n in ("block_table_cols", "dtype", "num_seqs", "heads", "kv_heads", "dim", "block_size",
                                       "select")]
                + [("scale", _f32)])


def declare(lib: ctypes.CDLL) -> None:
    """Argument and result types of the exported functions of this module."""
    lib.block_means.argtypes = [_i32, _vp, _i64, _i64, _i64, _i32, _i32, _i32, _vp, _i32, _vp, _vp]
    lib.block_means.restype = ctypes.c_int
    lib.block_scores.argtypes = [ctypes.POINTER(_ScoreArgs), _vp]
    lib.block_scores.restype = ctypes.c_int
    lib.block_attention.argtypes = [ctypes.POINTER(_AttentionArgs), _vp]
    lib.block_attention.restype = ctypes.c_int
    lib.block_attention_workspace.argtypes = [ctypes.POINTER(_AttentionArgs)]
    lib.block_attention_workspace.restype = ctypes.c_uint64
    lib.block_attention_backward.argtypes = [ctypes.POINTER(_AttentionArgs), _vp]
    lib.block_attention_backward.restype = ctypes.c_int
    lib.kv8_append.argtypes = [ctypes.POINTER(_AppendArgs), _vp]
    lib.kv8_append.restype = ctypes.c_int
    lib.kv8_attention.argtypes = [ctypes.POINTER(_DecodeArgs), _vp]
    lib.kv8_attention.restype = ctypes.c_int
    lib.kv8_attention_workspace.argtypes = [ctypes.POINTER(_DecodeArgs)]
    lib.kv8_attention_workspace.restype = ctypes.c_uint64


_loaded = None
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _lib():
    global _loaded
    if _loaded is None:
        from . import load_library
        _loaded = load_library()
    return _loaded


def _run(device, what: str, fn, *args) -> None:
    """``fn(*args, stream)`` on ``device`` and its current stream."""
    index = device.index
    if index == torch.cuda.current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(index))
    if status != 0:
        raise RuntimeError(f"{what} failed: {_STATUS.get(status, 'unknown status')} (status {status})")


def _no_tangent(t, what: str) -> None:
    """Refuses an operand with a forward-mode derivative, which the result would not have."""
    if getattr(_forward_ad, "_current_level", 0) >= 0 and _forward_ad.unpack_dual(t).tangent is not None:
        raise ValueError(f"{what} has a tangent: there is no forward-mode derivative")


def _heads(t, what: str, device=None, dtype=None, dim=None):
    """Checks a [tokens, heads, dim] operand; returns its shape and (token, head) strides, 0 for an axis of one entry."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES or t.dim() != 3:
        raise ValueError(f"{what} must be a 3-D bfloat16 or float16 tensor [tokens, heads, dim]")
    _no_tangent(t, what)
    if not t.is_cuda:
        raise ValueError(f"{what} must be on a GPU")
    if (device is not None and t.device != device) or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{what} must have the others' type and device")
    tokens, heads, d = t.shape
    if d not in HEAD_DIMS or (dim is not None and d != dim):
        raise ValueError(f"{what} must have a head dimension in {HEAD_DIMS}, the same for all")
    if heads < 1:
        raise ValueError(f"{what} must have at least one head")
    st, sh, sd = t.stride()
    if tokens <= 1:
        st = 0
    if heads <= 1:
        sh = 0
    if tokens and (sd != 1 or st % 8 or sh % 8 or st < 0 or sh < 0 or t.data_ptr() % 16):
        raise ValueError(f"{what} must have unit stride along its last axis, 16-byte-aligned data and other strides "
                         "that are multiples of 8 elements")
    return tokens, heads, d, st, sh


def _ints(t, what: str, device, dims: int, shape=None) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.dim() != dims or t.device != device:
        raise ValueError(f"{what} must be a {dims}-D int32 tensor on the others' device")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what} must have the shape {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def _sequences(cu_q, cu_k, device, total_q: int, total_k: int):
    """(cu_q, cu_k, sequences) with the defaults filled in."""
    if cu_q is None and cu_k is None:
        return None, None, 1
    if cu_q is None:
        raise ValueError("cu_seqlens_k needs cu_seqlens")
    if cu_k is None:
        if total_q != total_k:
            raise ValueError("cu_seqlens_k is needed where queries and keys differ in number")
        cu_k = cu_q
    for t, what in ((cu_q, "cu_seqlens"), (cu_k, "cu_seqlens_k")):
        _ints(t, what, device, 1)
        if t.shape[0] < 1 or t.shape[0] != cu_q.shape[0]:
            raise ValueError(f"{what} must have one entry more than there are sequences")
    return cu_q, cu_k, int(cu_q.shape[0]) - 1


def _table(t, device):
    """(sequences, columns, stride) of a block table."""
    if isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.dim() == 2 and t.device == device:
        (n, cols), (rows_at, cols_at) = t.shape, t.stride()
        if (cols <= 1 or cols_at == 1) and (n <= 1 or rows_at >= cols):
            return n, cols, rows_at if n > 1 else cols
    raise ValueError("block_table must be a 2-D int32 tensor on the others' device with unit stride along its last axis")


def _block_size(block_size) -> int:
    if block_size not in BLOCK_SIZES:
        raise ValueError(f"block_size must be one of {BLOCK_SIZES}")
    return int(block_size)


def _scale(scale, dim: int) -> float:
    scale = 1.0 / math.sqrt(dim) if scale is None else float(scale)
    if not 0.0 < scale < math.inf:
        raise ValueError("scale must be positive and finite")
    return scale


def _groups(heads: int, kv_heads: int) -> None:
    if heads % kv_heads or heads // kv_heads > 128:
        raise ValueError("the query heads must be a multiple of the key heads, 128 times as many at most")


def _output(out, shape, dtype, device, what: str):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if (not isinstance(out, torch.Tensor) or out.dtype != dtype or tuple(out.shape) != tuple(shape)
            or not out.is_contiguous() or out.device != device):
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on the others' device")
    return out


def _like(t):
    """A contiguous tensor of t's shape and type (the quickest way to one)."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _ptr(t):
    return None if t is None else t.data_ptr()


def block_means(k: torch.Tensor, block_size: int, cu_seqlens: torch.Tensor = None,
                out: torch.Tensor = None) -> torch.Tensor:
    """Mean of the keys of each block of ``block_size`` tokens.

    ``k``: bfloat16 or float16 ``[tokens, kv_heads, dim]``.  Returns float32
    ``[tokens // block_size + sequences, kv_heads, dim]``: block b of sequence
    i is row ``cu_seqlens[i] // block_size + i + b``; rows that are no block
    are 0.  No gradient goes back through the means."""
    bs = _block_size(block_size)
    total, hk, dim, st, sh = _heads(k, "k")
    device = k.device
    cu, _, n = _sequences(cu_seqlens, None, device, total, total)
    out = _output(out, (total // bs + n, hk, dim), torch.float32, device, "out")
    _run(device, "block_means", _lib().block_means, _DTYPES[k.dtype], k.data_ptr(), st, sh, total, hk, dim, bs, _ptr(cu), n,
         out.data_ptr())
    return out


def block_scores(q: torch.Tensor, means: torch.Tensor, block_size: int, max_blocks: int,
                 cu_seqlens: torch.Tensor = None, cu_seqlens_k: torch.Tensor = None,
                 lengths: torch.Tensor = None, block_table: torch.Tensor = None,
                 first: int = 1, last: int = 1, scale: float = None):
    """Scores of key blocks for each query and key head, as the rows that
    ``topk_indices`` selects from.

    Returns ``(scores, counts)``: float32 ``[tokens, kv_heads, max_blocks]``
    and int32 ``[tokens, kv_heads]``.  A block's score is the largest
    ``scale * q . mean`` of the group's query heads; the first ``first`` and
    the last ``last`` of the ``counts`` blocks that the query can see have
    +inf, so a selection always takes them, and the blocks behind have -inf.
    The last visible block is the query's own: its mean covers tokens behind
    the query, which ``last >= 1`` keeps out of the selection.

    Packed form: ``means`` of ``block_means`` (over ``cu_seqlens_k``, default
    ``cu_seqlens``; without both, one sequence with as many keys as queries).
    Paged form: ``block_table`` (int32 ``[sequences,
    >= max_blocks]``), ``lengths`` (int32 ``[sequences]``, keys with the
    queries' own) and ``means`` float32 ``[pages, kv_heads, dim]``; without
    ``cu_seqlens`` each sequence has one query.  An entry of the table outside
    the pages gives its block -inf.  Rows behind the last sequence are -inf
    with count 0.  No gradient goes back through the scores: what is selected
    is constant to ``block_attention``."""
    bs = _block_size(block_size)
    a = _ScoreArgs()
    total, heads, dim, a.q_stride_t, a.q_stride_h = _heads(q, "q")
    device = q.device
    if (not isinstance(means, torch.Tensor) or means.dtype != torch.float32 or means.dim() != 3 or means.device != device
            or not means.is_contiguous() or means.shape[2] != dim or means.shape[1] < 1):
        raise ValueError("means must be a contiguous float32 tensor [rows, kv_heads, dim] on q's device")
    _no_tangent(means, "means")
    if means.numel() and means.data_ptr() % 16:
        raise ValueError("means must be 16-byte aligned")
    hk = int(means.shape[1])
    _groups(heads, hk)
    max_blocks, first, last = int(max_blocks), int(first), int(last)
    if max_blocks < 1 or max_blocks >= 1 << 22 or first < 0 or last < 0:
        raise ValueError("max_blocks must be in [1, 2^22), first and last not negative")
    if block_table is not None:
        if lengths is None or cu_seqlens_k is not None:
            raise ValueError("the paged form takes block_table and lengths, without cu_seqlens_k")
        n, cols, a.block_table_stride = _table(block_table, device)
        if cols < max_blocks:
            raise ValueError("block_table must have max_blocks columns at least")
        _ints(lengths, "lengths", device, 1, (n,))
        if cu_seqlens is not None:
            _ints(cu_seqlens, "cu_seqlens", device, 1, (n + 1,))
        elif total != n:
            raise ValueError("without cu_seqlens there must be one query for each sequence")
        cu_q, cu_k = cu_seqlens, None
        if n == 0:  # all rows lie behind the last sequence, as in the packed form
            cu_k, block_table, lengths = cu_seqlens, None, None
    else:
        if lengths is not None:
            raise ValueError("lengths goes with block_table")
        cu_q, cu_k, n = _sequences(cu_seqlens, cu_seqlens if cu_seqlens_k is None else cu_seqlens_k, device, total, total)
        if cu_q is None and means.shape[0] < total // bs + 1:
            raise ValueError("means must have a row for every block, as block_means gives them")
    scores = means.new_empty((total, hk, max_blocks))
    counts = means.new_empty((total, hk), dtype=torch.int32)
    scale = _scale(scale, dim)
    if total == 0:
        return scores, counts
    a.q, a.means, a.cu_q, a.cu_k = q.data_ptr(), means.data_ptr(), _ptr(cu_q), _ptr(cu_k)
    a.lengths, a.block_table, a.scores, a.counts = _ptr(lengths), _ptr(block_table), scores.data_ptr(), counts.data_ptr()
    a.total_q, a.total_k, a.mean_rows = total, total, int(means.shape[0])
    a.dtype, a.num_seqs, a.heads, a.kv_heads, a.dim, a.block_size = _DTYPES[q.dtype], n, heads, hk, dim, bs
    a.max_blocks, a.first, a.last, a.scale = max_blocks, min(first, max_blocks), min(last, max_blocks), scale
    _run(device, "block_scores", _lib().block_scores, ctypes.byref(a))
    return scores, counts


def _attention_args(q, k, v, blocks, block_size, cu_seqlens, cu_seqlens_k, scale, causal):
    bs = _block_size(block_size)
    a = _AttentionArgs()
    total, heads, dim, a.q_stride_t, a.q_stride_h = _heads(q, "q")
    device = q.device
    total_k, hk, _, a.k_stride_t, a.k_stride_h = _heads(k, "k", device, q.dtype, dim)
    _, _, _, a.v_stride_t, a.v_stride_h = _heads(v, "v", device, q.dtype, dim)
    if k.shape != v.shape:
        raise ValueError("k and v must have the same shape")
    if a.k_stride_t >= 1 << 23 or a.v_stride_t >= 1 << 23:
        raise ValueError("k and v must have token strides below 2^23 elements")
    _groups(heads, hk)
    if not isinstance(blocks, torch.Tensor) or blocks.dim() != 3 or not 1 <= blocks.shape[2] <= MAX_SELECT:
        raise ValueError(f"blocks must be an int32 tensor [tokens, kv_heads, selected], selected in [1, {MAX_SELECT}]")
    _ints(blocks, "blocks", device, 3, (total, hk, blocks.shape[2]))
    cu_q, cu_k, n = _sequences(cu_seqlens, cu_seqlens_k, device, total, total_k)
    a.q, a.k, a.v, a.blocks = q.data_ptr(), k.data_ptr(), v.data_ptr(), blocks.data_ptr()
    a.cu_q, a.cu_k = _ptr(cu_q), _ptr(cu_k)
    a.total_q, a.total_k = total, total_k
    a.dtype, a.num_seqs, a.heads, a.kv_heads, a.dim, a.block_size = _DTYPES[q.dtype], n, heads, hk, dim, bs
    a.select, a.causal, a.scale = int(blocks.shape[2]), int(bool(causal)), _scale(scale, dim)
    return a


def block_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, blocks: torch.Tensor, block_size: int,
                    cu_seqlens: torch.Tensor = None, cu_seqlens_k: torch.Tensor = None, scale: float = None,
                    causal: bool = True, out: torch.Tensor = None, rest: torch.Tensor = None):
    """Attention of each query over the key blocks that it selects.

    ``q`` ``[tokens, heads, dim]``, ``k`` and ``v`` ``[keys, kv_heads, dim]``
    (bfloat16 or float16, dim 64 or 128, any strides that are multiples of 8
    elements with unit stride along dim); ``blocks`` int32 ``[tokens, kv_heads,
    selected]``, block numbers within the query's sequence in any order, where
    an entry that is negative or names no block selects nothing and a repeated
    one counts once.  ``causal`` hides the keys behind the query's position.

    Returns ``(out, lse)``: ``[tokens, heads, dim]`` of q's type, and the
    log-sum of the scaled scores' exponentials, float32 ``[tokens, heads]``.  A
    query that sees no key, and a row behind the last sequence, has 0 and -inf.

    Differentiable once in q, k and v through autograd (``lse`` is not; ``out=``
    and ``rest=`` are refused then; forward-mode derivatives are refused always).
    A graph can capture the call with its backward, but not while an eager
    gradient graph of the same leaves is alive: any operation's such graph would
    end the capture, this one sees its own and refuses the call, also where only
    the forward would be captured (capture that under ``torch.no_grad``).  A
    caller of ``block_attention_backward`` gives ``rest`` (like ``out``), which
    receives what the rounding of ``out`` leaves out."""
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in (q, k, v)):
        if out is not None or rest is not None:
            raise ValueError("out and rest cannot be given where a gradient is asked for")
        return _BlockAttention.apply(q, k, v, blocks, block_size, cu_seqlens, cu_seqlens_k, scale, causal)
    a = _attention_args(q, k, v, blocks, block_size, cu_seqlens, cu_seqlens_k, scale, causal)
    out = _like(q) if out is None else _output(out, q.shape, q.dtype, q.device, "out")
    lse = q.new_empty((a.total_q, a.heads), dtype=torch.float32)
    if rest is not None:
        _output(rest, q.shape, q.dtype, q.device, "rest")
    a.out, a.rest, a.lse = out.data_ptr(), _ptr(rest), lse.data_ptr()
    _run(q.device, "block_attention", _lib().block_attention, ctypes.byref(a))
    return out, lse


def block_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                             lse: torch.Tensor, blocks: torch.Tensor, block_size: int, cu_seqlens: torch.Tensor = None,
                             cu_seqlens_k: torch.Tensor = None, scale: float = None, causal: bool = True,
                             rest: torch.Tensor = None):
    """Gradients ``(dq, dk, dv)`` of ``block_attention`` for the gradient ``dout``
    of its ``out``; ``out`` and ``lse`` as it returned them, the rest as it was
    called; ``rest`` as ``block_attention`` filled it in (without it dq loses
    precision).  The result is the same from run to run.  With float16 the
    probabilities and the scores' gradients are held in float16: below about 6e-8
    they are lost (to dv; to dq and dk, unless the loss is scaled).  The gradients
    are constants: nothing goes back through them."""
    a = _attention_args(q, k, v, blocks, block_size, cu_seqlens, cu_seqlens_k, scale, causal)
    _, _, _, a.dout_stride_t, a.dout_stride_h = _heads(dout, "dout", q.device, q.dtype, q.shape[2])
    if dout.shape != q.shape:
        raise ValueError("dout must have q's shape")
    _output(out, q.shape, q.dtype, q.device, "out")
    _output(lse, q.shape[:2], torch.float32, q.device, "lse")
    if rest is not None:
        _output(rest, q.shape, q.dtype, q.device, "rest")
    dq, dk, dv = _like(q), _like(k), _like(v)
    a.out, a.rest, a.lse, a.dout, a.dq, a.dk, a.dv = (_ptr(t) for t in (out, rest, lse, dout, dq, dk, dv))
    lib = _lib()
    a.workspace_bytes = lib.block_attention_workspace(ctypes.byref(a))
    workspace = torch.empty(a.workspace_bytes, dtype=torch.uint8, device=q.device)
    a.workspace = workspace.data_ptr()
    _run(q.device, "block_attention_backward", lib.block_attention_backward, ctypes.byref(a))
    return dq, dk, dv


class _Summing:
    """Stands for the node that sums a leaf's gradients: made by the first gradient
    graph of the leaf and kept by all that follow while any of them lives."""

    def __init__(self, leaf, stream: int):
        self.leaf, self.stream = weakref.ref(leaf), stream


_summing = weakref.WeakValueDictionary()  # by the leaf's id: held by the calls' gradient graphs
_summing_lock = threading.RLock()  # a finalizer may call in between


def _summed(leaves, stream: int) -> list:
    """The leaves' nodes, for a call on ``stream``."""
    nodes = []
    with _summing_lock:
        for leaf in leaves:
            node = _summing.get(id(leaf))
            if node is None or node.leaf() is not leaf:
                node = _summing[id(leaf)] = _Summing(leaf, stream)
            nodes.append(node)
    return nodes


def _check_capture(nodes, stream: int) -> None:
    """Refuses a call under capture whose leaves' gradients are summed on another
    stream, that of the first living gradient graph: the backward would pull that
    stream into the capture, which ends the process."""
    if any(node.stream != stream for node in nodes):
        raise RuntimeError("block_attention cannot be captured while a gradient graph of the same leaves, first made on another "
                           "stream, is alive: drop the results of all such graphs first, or capture without gradients "
                           "(torch.no_grad)")


class _BlockAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, blocks, block_size, cu_seqlens, cu_seqlens_k, scale, causal):
        leaves = [t for t in (q, k, v) if t.requires_grad and t.is_leaf]
        if leaves and q.is_cuda:
            stream = _raw_stream(q.device.index)
            ctx.nodes = _summed(leaves, stream)
            if torch.cuda.is_current_stream_capturing():
                _check_capture(ctx.nodes, stream)
        rest = _like(q)
        out, lse = block_attention(q, k, v, blocks, block_size, cu_seqlens, cu_seqlens_k, scale, causal, rest=rest)
        ctx.save_for_backward(q, k, v, out, rest, lse, blocks, cu_seqlens, cu_seqlens_k)
        ctx.rest = (block_size, scale, causal)
        ctx.mark_non_differentiable(lse)
        ctx.set_materialize_grads(False)
        return out, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, _):
        if dout is None:
            return (None,) * 9
        q, k, v, out, rest, lse, blocks, cu_q, cu_k = ctx.saved_tensors
        block_size, scale, causal = ctx.rest
        if dout.stride(2) != 1 or dout.data_ptr() % 16 or any(dout.stride(i) % 8 for i in (0, 1)):
            dout = dout.clone(memory_format=torch.contiguous_format)
        dq, dk, dv = block_attention_backward(dout, q, k, v, out, lse, blocks, block_size, cu_q, cu_k, scale, causal, rest)
        need = ctx.needs_input_grad
        return dq if need[0] else None, dk if need[1] else None, dv if need[2] else None, *(None,) * 6


_F8 = torch.float8_e4m3fn


def _cache(k_cache, v_cache, k_scale, v_scale, device, hk=None, dim=None):
    """Pages of the 8-bit cache; returns (pages, kv_heads, block_size, dim)."""
    for t, what in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if (not isinstance(t, torch.Tensor) or t.dtype is not _F8 or t.dim() != 4 or t.device != device
                or not t.is_contiguous() or t.data_ptr() % 16):
            raise ValueError(f"{what} must be a contiguous float8_e4m3fn tensor [pages, kv_heads, block_size, dim] on the "
                             "others' device, 16-byte aligned, k_cache and v_cache of one shape")
    pages, heads, bs, d = shape = k_cache.shape
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must have one shape")
    _block_size(bs)
    if d not in HEAD_DIMS or heads < 1 or (hk is not None and heads != hk) or (dim is not None and d != dim):
        raise ValueError(f"the cache must have the others' heads and head dimension, one of {HEAD_DIMS}")
    shape = shape[:2]
    for t, what in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if (not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.shape != shape or not t.is_contiguous()
                or t.device != device):
            raise ValueError(f"{what} must be a contiguous float32 tensor [pages, kv_heads] on the others' device")
    return pages, heads, bs, d


def _cache_sequences(cu, lengths, n: int, total: int, device):
    _ints(lengths, "lengths", device, 1, (n,))
    if cu is not None:
        _ints(cu, "cu_seqlens", device, 1, (n + 1,))
    elif total != n:
        raise ValueError("without cu_seqlens there must be one token for each sequence")


def kv8_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
               v_scale: torch.Tensor, block_table: torch.Tensor, lengths: torch.Tensor, cu_seqlens: torch.Tensor = None,
               k_mean: torch.Tensor = None) -> None:
    """Stores new tokens' keys and values in the 8-bit paged cache, in place.

    ``k``, ``v`` ``[tokens, kv_heads, dim]``: each sequence's last tokens, those
    of sequence i at ``cu_seqlens[i]:cu_seqlens[i + 1]`` (default: one each);
    ``lengths`` int32 ``[sequences]`` counts them already.  ``k_cache``,
    ``v_cache`` float8_e4m3fn ``[pages, kv_heads, block_size, dim]``, ``k_scale``,
    ``v_scale`` float32 ``[pages, kv_heads]``; block b of sequence i is page
    ``block_table[i, b]``.

    A page's scale is the smallest power of two that brings what it holds to
    448 or less; it grows when a token needs it (the codes that are there are
    rounded again) and starts anew in a page whose first token is stored.
    Pages outside the cache store nothing; a call may store into a page through
    one entry of one sequence's row only.  ``k_mean`` (float32 ``[pages, kv_heads, dim]``) receives the mean of
    the keys of each page that got tokens: the ``means`` of ``block_scores``."""
    a = _AppendArgs()
    total, hk, dim, a.k_stride_t, a.k_stride_h = _heads(k, "k")
    device = k.device
    _, _, _, a.v_stride_t, a.v_stride_h = _heads(v, "v", device, k.dtype, dim)
    if k.shape != v.shape:
        raise ValueError("k and v must have the same shape")
    pages, _, bs, _ = _cache(k_cache, v_cache, k_scale, v_scale, device, hk, dim)
    n, a.block_table_cols, a.block_table_stride = _table(block_table, device)
    _cache_sequences(cu_seqlens, lengths, n, total, device)
    if k_mean is not None:
        _output(k_mean, (pages, hk, dim), torch.float32, device, "k_mean")
    a.k, a.v, a.k_cache, a.v_cache = k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
    a.k_scale, a.v_scale, a.k_mean = k_scale.data_ptr(), v_scale.data_ptr(), _ptr(k_mean)
    a.block_table, a.lengths, a.cu = block_table.data_ptr(), lengths.data_ptr(), _ptr(cu_seqlens)
    a.total, a.num_pages, a.num_seqs = total, pages, n
    a.dtype, a.kv_heads, a.dim, a.block_size = _DTYPES[k.dtype], hk, dim, bs
    _run(device, "kv8_append", _lib().kv8_append, ctypes.byref(a))


def kv8_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                  v_scale: torch.Tensor, block_table: torch.Tensor, lengths: torch.Tensor,
                  cu_seqlens: torch.Tensor = None, blocks: torch.Tensor = None, max_length: int = None,
                  scale: float = None, out: torch.Tensor = None):
    """Causal attention of each sequence's last tokens over the 8-bit paged cache
    (``kv8_append`` gives the layout), over all of it or at selected blocks.

    ``q`` ``[tokens, heads, dim]``; those of sequence i are its last ones
    (``cu_seqlens``; default one each) and ``lengths`` counts them.  ``blocks``
    (int32 ``[tokens, kv_heads, selected]``) names the blocks that each query
    reads, as for ``block_attention``.  ``max_length`` bounds the lengths where
    the caller knows them (default: what the table can hold); it only decides
    how the work is split.

    Returns ``(out, lse)`` as ``block_attention`` does, without its gradient:
    neither is differentiable, whatever ``q`` asks for."""
    a = _DecodeArgs()
    total, heads, dim, a.q_stride_t, a.q_stride_h = _heads(q, "q")
    device = q.device
    pages, hk, bs, _ = _cache(k_cache, v_cache, k_scale, v_scale, device, None, dim)
    _groups(heads, hk)
    n, a.block_table_cols, a.block_table_stride = _table(block_table, device)
    _cache_sequences(cu_seqlens, lengths, n, total, device)
    if a.block_table_cols * bs >= 1 << 30:
        raise ValueError("a sequence can hold less than 2^30 tokens")
    if blocks is not None:
        if not isinstance(blocks, torch.Tensor) or blocks.dim() != 3 or not 1 <= blocks.shape[2] <= MAX_SELECT:
            raise ValueError(f"blocks must be an int32 tensor [tokens, kv_heads, selected], selected in [1, {MAX_SELECT}]")
        _ints(blocks, "blocks", device, 3, (total, hk, blocks.shape[2]))
    if max_length is not None and max_length < 0:
        raise ValueError("max_length must not be negative")
    most = a.block_table_cols * bs
    max_length = most if max_length is None else min(int(max_length), most)
    out = _like(q) if out is None else _output(out, q.shape, q.dtype, device, "out")
    lse = q.new_empty((total, heads), dtype=torch.float32)
    a.q, a.k_cache, a.v_cache = q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
    a.k_scale, a.v_scale, a.block_table = k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr()
    a.lengths, a.cu, a.blocks, a.out, a.lse = lengths.data_ptr(), _ptr(cu_seqlens), _ptr(blocks), out.data_ptr(), lse.data_ptr()
    a.total_q, a.num_pages, a.max_length, a.num_seqs = total, pages, max_length, n
    a.dtype, a.heads, a.kv_heads, a.dim, a.block_size = _DTYPES[q.dtype], heads, hk, dim, bs
    a.select, a.scale = 0 if blocks is None else int(blocks.shape[2]), _scale(scale, dim)
    lib = _lib()
    a.workspace_bytes = lib.kv8_attention_workspace(ctypes.byref(a))
    if a.workspace_bytes:
        workspace = torch.empty(a.workspace_bytes, dtype=torch.uint8, device=device)
        a.workspace = workspace.data_ptr()
    _run(device, "kv8_attention", lib.kv8_attention, ctypes.byref(a))
    return out, lse
