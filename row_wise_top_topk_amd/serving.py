"""What a serving loop does around the selection and the 8-bit paged cache: a
prompt's chunk behind the cache, the pages of the cache, and the rows of logits
that ``topk_indices`` ranks.

Argument marshalling only, as in the package's other functions: every step
runs in the library's HIP kernels on the current stream of the tensors'
device.  Outputs and scratch memory come from PyTorch's allocator, so a call
can be captured into a graph, and two graphs share nothing.

    pages_grow(block_table, lengths, refs, new, 64)          # room for the new tokens
    out, lse = chunk_attention(q, k, v, k_cache, v_cache, k_scale, v_scale, block_table, lengths, cu_seqlens=cu, max_length=longest)
    kv8_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, lengths, cu_seqlens=cu)
    ...
    rows = penalize_logits(logits, tokens, lengths, repetition=r, mask=grammar)
    best = topk_indices(rows, ids, 40, order="value")        # ids: the vocabulary's size, a row each
    copies = pages_fork(block_table, lengths, refs, parents, 64)
    pages_copy(k_cache, v_cache, k_scale, v_scale, copies)   # in each layer's cache

One ``block_table`` (with ``lengths`` and ``refs``) serves all layers of a model.
``refs`` int32 ``[pages]`` counts the table's entries that name each page; a page
with 0 is free.  Full pages may be named by several rows, a row's last page, while
it is not full, by that row alone, since ``kv8_append`` writes into it.  A caller
may count holders of its own besides.  Nothing here has a gradient.
"""

from __future__ import annotations

import ctypes

import torch

from .attention import (_DTYPES, _block_size, _cache, _cache_sequences, _dual_level, _f32, _groups, _heads, _i32, _i64, _ints,
                        _lib, _like, _no_tangent, _no_tangents, _output, _ptr, _run, _scale, _table, _vp)

__all__ = ["chunk_attention", "pages_fork", "pages_grow", "pages_compact", "pages_copy", "penalize_logits"]

MAX_TOKENS = (1 << 21) - 1
MAX_BIAS = 1023
_FORK, _GROW, _COMPACT = 0, 1, 2
_LOGITS = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class _ChunkArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("q", "k", "v", "k_cache", "v_cache", "k_scale", "v_scale", "block_table", "lengths", "cu",
                                    "out", "lse", "workspace")]
                + [("workspace_bytes", ctypes.c_uint64)]
                + [(n, _i64) for n in ("q_stride_t", "q_stride_h", "k_stride_t", "k_stride_h", "v_stride_t", "v_stride_h", "total",
                                       "num_pages", "block_table_stride", "max_length")]
                + [(n, _i32) for n in ("block_table_cols", "dtype", "num_seqs", "heads", "kv_heads", "dim", "block_size")]
                + [("scale", _f32)])


class _PagesArgs(ctypes.Structure):
    _fields_ = ([("block_table", _vp), ("lengths", _vp), ("refs", _vp), ("given", _vp), ("out", _vp), ("workspace", _vp),
                 ("workspace_bytes", ctypes.c_uint64), ("num_pages", _i64), ("block_table_stride", _i64)]
                + [(n, _i32) for n in ("rows", "block_table_cols", "block_size", "op")])


class _CopyArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("k_cache", "v_cache", "k_scale", "v_scale", "k_mean", "copies")]
                + [("num", _i64), ("num_pages", _i64)] + [(n, _i32) for n in ("kv_heads", "dim", "block_size")])


class _PenalizeArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("logits", "out", "tokens", "lengths", "prompt_lengths", "repetition", "frequency", "presence",
                                    "bias_ids", "bias", "mask")]
                + [(n, _i64) for n in ("rows", "vocab", "logits_stride", "out_stride", "tokens_stride", "bias_stride", "mask_stride")]
                + [(n, _i32) for n in ("token_cols", "bias_cols", "dtype")])


def declare(lib: ctypes.CDLL) -> None:
    """Argument and result types of the exported functions of this module."""
    for name, cls in (("chunk_attention", _ChunkArgs), ("pages_update", _PagesArgs), ("pages_copy", _CopyArgs),
                      ("logits_penalize", _PenalizeArgs)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = [ctypes.POINTER(cls), _vp], ctypes.c_int
    for name, cls in (("chunk_attention_workspace", _ChunkArgs), ("pages_workspace", _PagesArgs)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = [ctypes.POINTER(cls)], ctypes.c_uint64


def chunk_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    k_scale: torch.Tensor, v_scale: torch.Tensor, block_table: torch.Tensor, lengths: torch.Tensor,
                    cu_seqlens: torch.Tensor = None, max_length: int = None, scale: float = None, out: torch.Tensor = None):
    """Causal attention of a chunk of new tokens: over what stands before them in
    the 8-bit paged cache, and over their own keys and values in 16 bits.

    ``q`` ``[tokens, heads, dim]``, ``k`` and ``v`` ``[tokens, kv_heads, dim]``
    (bfloat16 or float16, dim 64 or 128): the last tokens of each sequence, those
    of sequence i at ``cu_seqlens[i]:cu_seqlens[i + 1]`` (default: one each);
    ``lengths`` int32 ``[sequences]`` counts them.  The cache's arguments are
    those of ``kv8_append``; it holds each sequence's tokens before the chunk, and
    is read there only: the chunk may be appended before, after or never.  A
    prompt's first chunk has nothing in the cache.  ``max_length`` bounds the
    lengths where the caller knows them (default: what the table can hold, and
    the chunk); it only decides how the work is split.  A few tokens behind a long
    context need it: a bound far above the lengths, as that of a wide table, can
    cost them several times the time.

    Pages and table columns that are not there give no keys.  Returns ``(out,
    lse)`` as ``kv8_attention`` does: ``[tokens, heads, dim]`` of q's type, and
    float32 ``[tokens, heads]``; a query that sees no key, and a row behind the
    last sequence, has 0 and -inf.  Neither is differentiable."""
    total, heads, dim, q_t, q_h = _heads(q, "q")
    device = q.device
    total_k, hk, _, k_t, k_h = _heads(k, "k", device, q.dtype, dim)
    _, _, _, v_t, v_h = _heads(v, "v", device, q.dtype, dim)
    if k.shape != v.shape or total_k != total:
        raise ValueError("k and v must have the same shape, with a row for each of q's")
    if k_t >= 1 << 23 or v_t >= 1 << 23:
        raise ValueError("k and v must have token strides below 2^23 elements")
    _groups(heads, hk)
    pages, _, bs, _ = _cache(k_cache, v_cache, k_scale, v_scale, device, hk, dim)
    n, cols, table_at = _table(block_table, device)
    _cache_sequences(cu_seqlens, lengths, n, total, device)
    most = cols * bs
    if most >= 1 << 30:
        raise ValueError("a sequence can hold less than 2^30 tokens")
    if max_length is not None and max_length < 0:
        raise ValueError("max_length must not be negative")
    most += total
    out = _like(q) if out is None else _output(out, q.shape, q.dtype, device, "out")
    lse = q.new_empty((total, heads), dtype=torch.float32)
    a = _ChunkArgs(q.data_ptr(), k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                   v_scale.data_ptr(), block_table.data_ptr(), lengths.data_ptr(), None if cu_seqlens is None else cu_seqlens.data_ptr(),
                   out.data_ptr(), lse.data_ptr(), None, 0, q_t, q_h, k_t, k_h, v_t, v_h, total, pages, table_at,
                   min(most if max_length is None else int(max_length), most, (1 << 31) - 1), cols, _DTYPES[q.dtype], n, heads, hk, dim,
                   bs, _scale(scale, dim))
    lib = _lib()
    a.workspace_bytes = lib.chunk_attention_workspace(ctypes.byref(a))
    if a.workspace_bytes:
        workspace = torch.empty(a.workspace_bytes, dtype=torch.uint8, device=device)
        a.workspace = workspace.data_ptr()
    _run(device, "chunk_attention", lib.chunk_attention, ctypes.byref(a))
    return out, lse


def _pages(op: int, what: str, block_table, lengths, refs, given, given_what, out_shape, block_size):
    bs = _block_size(block_size)
    if not isinstance(block_table, torch.Tensor) or not block_table.is_cuda:
        raise ValueError("block_table must be on a GPU")
    device = block_table.device
    rows, cols, table_at = _table(block_table, device)
    if cols * bs >= 1 << 30:
        raise ValueError("a sequence can hold less than 2^30 tokens")
    _ints(lengths, "lengths", device, 1, (rows,))
    _ints(refs, "refs", device, 1)
    if given is not None or given_what:
        _ints(given, given_what, device, 1, (rows,))
    pages = refs.shape[0]
    out = block_table.new_empty(out_shape(rows, pages))
    a = _PagesArgs(block_table.data_ptr(), lengths.data_ptr(), refs.data_ptr(), _ptr(given), out.data_ptr(), None, 0, pages, table_at, rows,
                   cols, bs, op)
    lib = _lib()
    a.workspace_bytes = lib.pages_workspace(ctypes.byref(a))
    if a.workspace_bytes:
        workspace = torch.empty(a.workspace_bytes, dtype=torch.uint8, device=device)
        a.workspace = workspace.data_ptr()
    _run(device, what, lib.pages_update, ctypes.byref(a))
    return out


def pages_fork(block_table: torch.Tensor, lengths: torch.Tensor, refs: torch.Tensor, parents: torch.Tensor,
               block_size: int) -> torch.Tensor:
    """Forks, reorders and ends rows of a paged cache, in place: row i of
    ``block_table`` (int32 ``[rows, columns]``) and ``lengths`` (int32 ``[rows]``)
    becomes a fork of what row ``parents[i]`` (int32) was before the call, for all
    rows at once.

    ``parents[i] == i`` leaves the row as it is; a parent outside ``[0, rows)`` ends
    it: length 0, pages given up.  A fork shares its parent's full pages (``refs``
    counts them).  The parent's last page, where it is not full, stays with the
    parent's own row if that goes on, else with its first fork; every other fork
    gets a free page, lowest pages first, lower rows first.

    Returns int32 ``[rows, 2]``, the copies that ``pages_copy`` then makes in each
    layer's cache: (page, page to copy it to), or (-1, -1).  A fork for which no
    page is free has (page, -1) and the tokens of its full pages only.  Entries
    behind the last page of a row that changed are -1."""
    return _pages(_FORK, "pages_fork", block_table, lengths, refs, parents, "parents", lambda rows, _: (rows, 2), block_size)


def pages_grow(block_table: torch.Tensor, lengths: torch.Tensor, refs: torch.Tensor, grow: torch.Tensor,
               block_size: int) -> torch.Tensor:
    """Makes room for ``grow[i]`` (int32 ``[rows]``; none if negative) more tokens in
    row i, in place: ``lengths[i]`` grows by that, and the row gets the pages that it
    lacks, lowest free pages first, lower rows first.  ``kv8_append`` and the
    attention functions then take ``lengths`` as it is.

    Returns int32 ``[rows]``, by how many tokens each row grew: ``grow[i]``, or 0
    for a row whose table has not the columns, or for which, with what the rows
    before it ask for, not enough pages are free; such a row stays as it is."""
    return _pages(_GROW, "pages_grow", block_table, lengths, refs, grow, "grow", lambda rows, _: (rows,), block_size)


def pages_compact(block_table: torch.Tensor, lengths: torch.Tensor, refs: torch.Tensor, block_size: int) -> torch.Tensor:
    """Brings the pages in use to the front of the cache, in place: with n in use,
    those from page n on move to the free ones below it, the lowest to the lowest;
    the rows' entries and ``refs`` follow.

    Returns int32 ``[pages // 2, 2]``, the copies that ``pages_copy`` then makes in
    each layer's cache: (page, page to copy it to), (-1, -1) behind the last one.  A
    caller that holds pages of its own (counted in ``refs``) finds them there."""
    return _pages(_COMPACT, "pages_compact", block_table, lengths, refs, None, "", lambda _, pages: (pages // 2, 2), block_size)


def pages_copy(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, copies: torch.Tensor,
               k_mean: torch.Tensor = None) -> None:
    """Copies pages within one layer's 8-bit cache, in place: codes, scales and,
    where given, ``k_mean`` (float32 ``[pages, kv_heads, dim]``).

    ``copies``: int32 ``[n, 2]`` of ``pages_fork`` or ``pages_compact``; a pair with
    an entry outside the pages copies nothing.  In pairs of a caller's own no page
    may be copied to twice, nor be copied both from and to."""
    if not isinstance(k_cache, torch.Tensor) or not k_cache.is_cuda:
        raise ValueError("k_cache must be on a GPU")
    device = k_cache.device
    pages, hk, bs, dim = _cache(k_cache, v_cache, k_scale, v_scale, device)
    _ints(copies, "copies", device, 2)
    if copies.shape[1] != 2:
        raise ValueError("copies must have the shape [n, 2]")
    if k_mean is not None:
        _output(k_mean, (pages, hk, dim), torch.float32, device, "k_mean")
        _no_tangent(k_mean, "k_mean")
    a = _CopyArgs(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), _ptr(k_mean), copies.data_ptr(),
                  copies.shape[0], pages, hk, dim, bs)
    _run(device, "pages_copy", _lib().pages_copy, ctypes.byref(a))


def _matrix(t, what: str, dtype, device, rows: int):
    """(columns, row stride) of a 2-D operand with unit stride along its last axis."""
    shape = t.shape if isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device else ()
    if len(shape) != 2 or shape[0] != rows:
        raise ValueError(f"{what} must be a 2-D {dtype} tensor with a row for each of the logits, on their device")
    cols = shape[1]
    at, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{what} must have unit stride along its last axis")
    return cols, at if rows > 1 else 0


def _row(t, what: str, dtype, device, rows: int):
    """Address of a 1-D operand with an entry for each row, None where it is not given."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.shape == (rows,) and t.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous 1-D {dtype} tensor with an entry for each row, on the logits' device")
    return t.data_ptr()


def penalize_logits(logits: torch.Tensor, tokens: torch.Tensor = None, lengths: torch.Tensor = None,
                    prompt_lengths: torch.Tensor = None, repetition: torch.Tensor = None, presence: torch.Tensor = None,
                    frequency: torch.Tensor = None, bias_ids: torch.Tensor = None, bias: torch.Tensor = None,
                    mask: torch.Tensor = None, out: torch.Tensor = None) -> torch.Tensor:
    """Rows of logits with penalties for repeated tokens, biases and a grammar's
    mask: the rows that ``topk_indices`` ranks for a sampler or a beam search.

    ``logits`` ``[rows, vocab]``, bfloat16, float16 or float32, any row stride.
    For id j of row i, in 32 bits:

    - where j is among ``tokens[i, :lengths[i]]``: x > 0 ? x / r : x * r, with
      r = ``repetition[i]``;
    - minus ``frequency[i]`` * n, and minus ``presence[i]`` where n > 0: n is the
      number of times that j is among the generated tokens, ``tokens[i,
      prompt_lengths[i]:lengths[i]]``;
    - plus ``bias[i, e]`` where ``bias_ids[i, e] == j`` (the last such e);
    - -inf where bit j % 32 of ``mask[i, j // 32]`` is 0.

    ``tokens`` int32 ``[rows, columns]`` (up to 2^21 - 1), ``lengths`` and
    ``prompt_lengths`` int32 ``[rows]`` (default: all columns, and 0);
    ``repetition``, ``presence`` and ``frequency`` float32 ``[rows]``; ``bias_ids``
    int32 and ``bias`` float32 ``[rows, columns]`` (up to 1023); ``mask`` int32
    ``[rows, (vocab + 31) // 32]``.  What is not given changes nothing; ids outside
    the vocabulary (-1 for padding) count nowhere.  Returns float32 ``[rows,
    vocab]``; ``out`` may be ``logits`` itself where that is float32, and shares no
    memory with it otherwise.  It has no gradient, whatever the operands ask for;
    operands with a forward-mode derivative are refused."""
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _LOGITS or logits.dim() != 2:
        raise ValueError("logits must be a 2-D bfloat16, float16 or float32 tensor [rows, vocab]")
    if _dual_level():
        _no_tangents(((logits, "logits"), (repetition, "repetition"), (presence, "presence"), (frequency, "frequency"), (bias, "bias")))
    if not logits.is_cuda:
        raise ValueError("logits must be on a GPU")
    device = logits.device
    rows = logits.shape[0]
    vocab, logits_at = _matrix(logits, "logits", logits.dtype, device, rows)
    if out is None:
        out = torch.empty_like(logits, dtype=torch.float32, memory_format=torch.contiguous_format)
        out_at = vocab
    else:
        cols, out_at = _matrix(out, "out", torch.float32, device, rows)
        if cols != vocab or (rows > 1 and out_at < vocab):
            raise ValueError("out must have the logits' shape, and rows that do not overlap")
        if out.data_ptr() == logits.data_ptr() and rows > 1 and vocab and (out.dtype != logits.dtype or out_at != logits_at):
            raise ValueError("out may be the logits themselves only where both have one type and stride")
    said = said_at = ids = ids_at = words_at = 0
    if tokens is not None:
        said, said_at = _matrix(tokens, "tokens", torch.int32, device, rows)
        if said > MAX_TOKENS:
            raise ValueError(f"tokens must have {MAX_TOKENS} columns at most")
    elif not (lengths is None and prompt_lengths is None and repetition is None and presence is None and frequency is None):
        raise ValueError("lengths, prompt_lengths, repetition, presence and frequency go with tokens")
    if (bias is None) != (bias_ids is None):
        raise ValueError("bias and bias_ids go together")
    if bias is not None:
        ids, ids_at = _matrix(bias_ids, "bias_ids", torch.int32, device, rows)
        if ids > MAX_BIAS or _matrix(bias, "bias", torch.float32, device, rows) != (ids, ids_at):
            raise ValueError(f"bias and bias_ids must have one shape and strides, with {MAX_BIAS} columns at most")
    if mask is not None:
        words, words_at = _matrix(mask, "mask", torch.int32, device, rows)
        if words != (vocab + 31) // 32:
            raise ValueError("mask must have (vocab + 31) // 32 columns")
    a = _PenalizeArgs(logits.data_ptr(), out.data_ptr(), _ptr(tokens), _row(lengths, "lengths", torch.int32, device, rows),
                      _row(prompt_lengths, "prompt_lengths", torch.int32, device, rows),
                      _row(repetition, "repetition", torch.float32, device, rows),
                      _row(frequency, "frequency", torch.float32, device, rows),
                      _row(presence, "presence", torch.float32, device, rows), _ptr(bias_ids), _ptr(bias), _ptr(mask), rows, vocab,
                      logits_at, out_at, said_at, ids_at, words_at, said, ids, _LOGITS[logits.dtype])
    _run(device, "penalize_logits", _lib().logits_penalize, ctypes.byref(a))
    return out
