"""The serving headers against the library and the binding, every refusal of the C
entries that is decided on the host, and what the binding refuses without a GPU.

No GPU needed: only calls that return before they touch a device are made; the
pointers are numbers that nothing reads.
"""

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import row_wise_top_topk_amd as mt
from row_wise_top_topk_amd import serving as binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = [os.path.join(ROOT, "include", h) for h in ("attention/mi_chunk.h", "serving/mi_pages.h", "serving/mi_logits.h")]
STRUCTS = {"mi_chunk_attention_args": binding._ChunkArgs, "mi_pages_args": binding._PagesArgs, "mi_pages_copy_args": binding._CopyArgs,
           "mi_penalize_args": binding._PenalizeArgs}
OK, EINVAL, EWORKSPACE = 0, 1, 2
A = 1 << 20          # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    return mt.load_library()


def test_every_declared_function_is_exported(lib):
    names = []
    for h in HEADERS:
        text = re.sub(r"/\*.*?\*/", "", open(h).read(), flags=re.S)
        names += re.findall(r"^(?:int|uint64_t) ([a-z0-9_]+)\(", text, flags=re.M)
    assert sorted(names) == sorted(["chunk_attention", "chunk_attention_workspace", "pages_update", "pages_workspace", "pages_copy",
                                    "logits_penalize"])
    out = subprocess.run(["nm", "-D", "--defined-only", mt.library_path()], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert {e for e in exported if e.startswith(("chunk_", "pages_", "logits_"))} == set(names)
    for n in names:
        assert getattr(lib, n).argtypes


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host compiler")
def test_the_binding_mirrors_the_structs(tmp_path):
    lines = []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu %zu\\n", offsetof({name}, {f[0]}), sizeof((({name}*)0)->{f[0]}));' for f in cls._fields_]
    src = tmp_path / "sizes.cpp"
    src.write_text("#include <cstdio>\n#include <cstddef>\n" + "".join(f'#include "{h}"\n' for h in HEADERS)
                   + "int main() {\n" + "\n".join(lines) + "\n}\n")
    exe = tmp_path / "sizes"
    subprocess.run(["g++", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    at = iter(subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n"))
    for name, cls in STRUCTS.items():
        assert int(next(at)) == ctypes.sizeof(cls), name
        for f in cls._fields_:
            d = getattr(cls, f[0])
            assert next(at) == f"{d.offset} {d.size}", (name, f[0])


def make(cls, base, kw):
    a = cls()
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


def chunk(**kw):
    return make(binding._ChunkArgs, dict(
        q=A, k=A, v=A, k_cache=A, v_cache=A, k_scale=A, v_scale=A, block_table=A, lengths=A, cu=A, out=A, lse=A, q_stride_t=256,
        q_stride_h=64, k_stride_t=128, k_stride_h=64, v_stride_t=128, v_stride_h=64, total=10, num_pages=8, block_table_stride=4,
        max_length=64, block_table_cols=4, dtype=0, num_seqs=3, heads=4, kv_heads=2, dim=64, block_size=16, scale=0.125), kw)


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(dtype=-1), dict(dim=96), dict(block_size=8), dict(block_size=48), dict(kv_heads=0), dict(heads=3), dict(heads=0),
    dict(heads=258), dict(total=-1), dict(total=1 << 31), dict(num_pages=-1), dict(num_pages=1 << 31), dict(num_seqs=-1), dict(cu=0),
    dict(block_table_cols=-1), dict(block_table_stride=3), dict(block_table_cols=1 << 26, block_table_stride=1 << 26), dict(max_length=-1),
    dict(max_length=1 << 31), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q_stride_t=-8),
    dict(q_stride_h=4), dict(k_stride_t=12), dict(v_stride_h=-64), dict(k_stride_t=1 << 23), dict(v_stride_t=1 << 23), dict(q=0), dict(k=0),
    dict(v=0), dict(out=0), dict(lse=0), dict(lengths=0), dict(block_table=0), dict(k_cache=0), dict(v_cache=0), dict(k_scale=0),
    dict(v_scale=0), dict(q=A + 8), dict(k=A + 2), dict(v=A + 4), dict(out=A + 8), dict(k_cache=A + 8), dict(v_cache=A + 4),
    dict(k_scale=A + 2), dict(v_scale=A + 1), dict(lse=A + 2), dict(lengths=A + 2), dict(block_table=A + 1), dict(cu=A + 2),
    dict(workspace=A + 8), dict(num_seqs=(1 << 31) - 1), dict(total=(1 << 31) - 1, max_length=100000)], ids=str)
def test_chunk_attention_refuses(lib, bad):
    assert lib.chunk_attention(ctypes.byref(chunk(**bad)), None) == EINVAL


def test_chunk_attention_workspace(lib):
    assert lib.chunk_attention(None, None) == EINVAL and lib.chunk_attention_workspace(None) == 0
    assert lib.chunk_attention_workspace(ctypes.byref(chunk(dim=96))) == 0
    assert lib.chunk_attention(ctypes.byref(chunk(total=0, q=0, k=0, v=0, out=0, lse=0)), None) == OK
    long = dict(block_table_cols=1 << 12, block_table_stride=1 << 12, max_length=1 << 16)
    need = lib.chunk_attention_workspace(ctypes.byref(chunk(**long)))
    assert need > 0
    for ws, n in ((0, need), (A, need - 1)):
        assert lib.chunk_attention(ctypes.byref(chunk(**long, workspace=ws, workspace_bytes=n)), None) == EWORKSPACE


def test_chunk_attention_workspace_is_bounded(lib):
    # partial results of 1024 workgroups of 128 rows at most, whatever the call
    for total in (1, 17, 100, 1000, 10000, 1 << 20, (1 << 31) - 1):
        for seqs in (1, 7, 300):
            for cols in (1, 100, 1 << 20):
                a = chunk(total=total, num_seqs=seqs, heads=64, kv_heads=8, dim=128, block_table_cols=cols, block_table_stride=cols,
                          max_length=(1 << 31) - 1)
                assert lib.chunk_attention_workspace(ctypes.byref(a)) <= 1024 * 128 * 130 * 4


def pages(**kw):
    return make(binding._PagesArgs, dict(block_table=A, lengths=A, refs=A, given=A, out=A, workspace=A, workspace_bytes=1 << 30,
                                         num_pages=100, block_table_stride=4, rows=3, block_table_cols=4, block_size=16, op=0), kw)


@pytest.mark.parametrize("bad", [
    dict(op=-1), dict(op=3), dict(rows=-1), dict(block_table_cols=-1), dict(block_table_stride=3), dict(num_pages=-1),
    dict(num_pages=1 << 31), dict(block_size=8), dict(block_size=24), dict(block_table_cols=1 << 26, block_table_stride=1 << 26),
    dict(block_table=0), dict(lengths=0), dict(refs=0), dict(given=0), dict(out=0), dict(given=0, op=1), dict(out=0, op=1),
    dict(out=0, op=2), dict(block_table=A + 2), dict(lengths=A + 1), dict(refs=A + 2), dict(given=A + 2), dict(out=A + 2),
    dict(workspace=A + 8), dict(rows=1 << 24, workspace_bytes=1 << 50), dict(rows=1 << 24, op=1, workspace_bytes=1 << 50),
    dict(rows=1 << 24, op=2, workspace_bytes=1 << 50)], ids=str)
def test_pages_update_refuses(lib, bad):
    assert lib.pages_update(ctypes.byref(pages(**bad)), None) == EINVAL


@pytest.mark.parametrize("op", [0, 1, 2])
def test_pages_workspace(lib, op):
    assert lib.pages_update(None, None) == EINVAL and lib.pages_workspace(None) == 0
    assert lib.pages_workspace(ctypes.byref(pages(op=op))) == 0   # one workgroup's work
    for more in (dict(num_pages=(1 << 13) + 1), dict(rows=1025), dict(block_table_cols=1 << 12, block_table_stride=1 << 12)):
        need = lib.pages_workspace(ctypes.byref(pages(op=op, **more)))
        assert need > 0
        for ws, n in ((0, need), (A, need - 1)):
            assert lib.pages_update(ctypes.byref(pages(op=op, workspace=ws, workspace_bytes=n, **more)), None) == EWORKSPACE
    nothing = dict(op=op, rows=0, num_pages=0, block_table=0, lengths=0, refs=0, given=0, out=0, workspace=0, workspace_bytes=0)
    assert lib.pages_update(ctypes.byref(pages(**nothing)), None) == OK


def copy(**kw):
    return make(binding._CopyArgs, dict(k_cache=A, v_cache=A, k_scale=A, v_scale=A, k_mean=A, copies=A, num=3, num_pages=8, kv_heads=2,
                                        dim=64, block_size=16), kw)


@pytest.mark.parametrize("bad", [
    dict(num=-1), dict(num=1 << 31), dict(num_pages=-1), dict(num_pages=1 << 31), dict(kv_heads=0), dict(dim=96), dict(block_size=8),
    dict(kv_heads=1 << 21), dict(copies=0), dict(k_cache=0), dict(v_cache=0), dict(k_scale=0), dict(v_scale=0), dict(k_cache=A + 8),
    dict(v_cache=A + 4), dict(k_scale=A + 2), dict(v_scale=A + 1), dict(k_mean=A + 2), dict(copies=A + 2)], ids=str)
def test_pages_copy_refuses(lib, bad):
    assert lib.pages_copy(ctypes.byref(copy(**bad)), None) == EINVAL
    assert lib.pages_copy(None, None) == EINVAL
    assert lib.pages_copy(ctypes.byref(copy(num=0, copies=0)), None) == OK


def penalize(**kw):
    return make(binding._PenalizeArgs, dict(
        logits=A, out=2 * A, tokens=A, lengths=A, prompt_lengths=A, repetition=A, frequency=A, presence=A, bias_ids=A, bias=A, mask=A, rows=3,
        vocab=100, logits_stride=100, out_stride=100, tokens_stride=8, bias_stride=4, mask_stride=4, token_cols=8, bias_cols=4, dtype=2), kw)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(rows=1 << 31), dict(vocab=-1), dict(vocab=1 << 31), dict(token_cols=-1),
    dict(token_cols=1 << 21), dict(bias_cols=-1), dict(bias_cols=1024), dict(logits_stride=-1), dict(out_stride=99), dict(tokens_stride=-1),
    dict(bias_stride=-1), dict(mask_stride=-1), dict(logits=0), dict(out=0), dict(tokens=0), dict(bias_ids=0), dict(bias=0),
    dict(logits=A + 2), dict(logits=A + 1, dtype=0), dict(out=A + 2), dict(tokens=A + 2), dict(lengths=A + 1), dict(prompt_lengths=A + 2),
    dict(repetition=A + 2), dict(frequency=A + 2), dict(presence=A + 2), dict(bias_ids=A + 2), dict(bias=A + 2), dict(mask=A + 2),
    dict(out=A, logits_stride=128), dict(out=A, dtype=1), dict(rows=1 << 23), dict(rows=1 << 16, vocab=1 << 21, logits_stride=1 << 21,
                                                                                   out_stride=1 << 21)], ids=str)
def test_logits_penalize_refuses(lib, bad):
    assert lib.logits_penalize(ctypes.byref(penalize(**bad)), None) == EINVAL
    assert lib.logits_penalize(None, None) == EINVAL
    assert lib.logits_penalize(ctypes.byref(penalize(rows=0, logits=0, out=0)), None) == OK


def test_python_refuses_tensors_of_the_host():
    q, ints = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        mt.chunk_attention(q, q, q, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="3-D"):
        mt.chunk_attention(q[0], q, q, None, None, None, None, None, None)
    for call in (lambda: mt.pages_fork(ints.view(4, 1), ints, ints, ints, 16), lambda: mt.pages_grow(ints.view(4, 1), ints, ints, ints, 16),
                 lambda: mt.pages_compact(ints.view(4, 1), ints, ints, 16), lambda: mt.pages_copy(q, q, q, q, ints.view(2, 2)),
                 lambda: mt.penalize_logits(torch.zeros(2, 5))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="block_size"):
        mt.pages_fork(ints.view(4, 1), ints, ints, ints, 20)
    with pytest.raises(ValueError, match="2-D"):
        mt.penalize_logits(torch.zeros(2, 5, dtype=torch.float64))
