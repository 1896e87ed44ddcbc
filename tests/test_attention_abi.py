"""The attention headers against the library and the binding, and every refusal
of the C entries that is decided on the host.

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
from row_wise_top_topk_amd import attention as binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = [os.path.join(ROOT, "include", "attention", h) for h in ("mi_block_attention.h", "mi_kv8.h")]
STRUCTS = {"mi_block_scores_args": binding._ScoreArgs, "mi_block_attention_args": binding._AttentionArgs,
           "mi_kv8_append_args": binding._AppendArgs, "mi_kv8_attention_args": binding._DecodeArgs}
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
    assert sorted(names) == sorted(["block_means", "block_scores", "block_attention", "block_attention_workspace",
                                    "block_attention_backward", "kv8_append", "kv8_attention", "kv8_attention_workspace"])
    out = subprocess.run(["nm", "-D", "--defined-only", mt.library_path()], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert set(names) <= exported
    assert {e for e in exported if e.startswith(("block_", "kv8_"))} == set(names)
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
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    at = iter(got)
    for name, cls in STRUCTS.items():
        assert int(next(at)) == ctypes.sizeof(cls), name
        for f in cls._fields_:
            d = getattr(cls, f[0])
            assert next(at) == f"{d.offset} {d.size}", (name, f[0])


def make(cls, **kw):
    a = cls()
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attention(**kw):
    base = dict(q=A, k=A, v=A, blocks=A, out=A, lse=A, dout=A, dq=A, dk=A, dv=A, q_stride_t=256, q_stride_h=64, k_stride_t=128,
                k_stride_h=64, v_stride_t=128, v_stride_h=64, dout_stride_t=256, dout_stride_h=64, total_q=10, total_k=10, dtype=0,
                num_seqs=1, heads=4, kv_heads=2, dim=64, block_size=16, select=2, causal=1, scale=0.125)
    return make(binding._AttentionArgs, **{**base, **kw})


BAD_ATTENTION = [
    dict(total_q=-1), dict(total_q=1 << 31), dict(total_k=-1), dict(total_k=1 << 31), dict(num_seqs=-1), dict(num_seqs=2), dict(num_seqs=0),
    dict(cu_q=A), dict(cu_k=A), dict(dtype=2), dict(dtype=-1), dict(dim=32), dict(dim=96), dict(dim=256), dict(block_size=0),
    dict(block_size=8), dict(block_size=48), dict(block_size=256), dict(kv_heads=0), dict(heads=3), dict(heads=1), dict(heads=258),
    dict(select=0), dict(select=1025), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
    dict(q_stride_t=-8), dict(q_stride_h=4), dict(k_stride_t=12), dict(v_stride_h=-64), dict(k_stride_t=1 << 23), dict(v_stride_t=1 << 23),
    dict(q=0), dict(k=0), dict(v=0), dict(blocks=0), dict(out=0), dict(lse=0), dict(q=A + 8), dict(k=A + 2), dict(v=A + 4),
    dict(out=A + 8), dict(rest=A + 8), dict(blocks=A + 2), dict(lse=A + 1), dict(cu_q=A + 2, cu_k=A), dict(cu_q=A, cu_k=A + 2),
]


@pytest.mark.parametrize("bad", BAD_ATTENTION, ids=str)
def test_block_attention_refuses(lib, bad):
    a = attention(**bad)
    assert lib.block_attention(ctypes.byref(a), None) == EINVAL
    assert lib.block_attention_backward(ctypes.byref(a), None) == EINVAL


@pytest.mark.parametrize("bad", [dict(dout=0), dict(dq=0), dict(dk=0), dict(dv=0), dict(dout=A + 8), dict(dq=A + 4), dict(dk=A + 8),
                                 dict(dv=A + 2), dict(workspace=A + 8), dict(dout_stride_t=-8), dict(dout_stride_h=4)], ids=str)
def test_backward_refuses(lib, bad):
    assert lib.block_attention_backward(ctypes.byref(attention(**bad)), None) == EINVAL


def test_nothing_to_do_and_small_workspaces(lib):
    assert lib.block_attention(None, None) == EINVAL
    assert lib.block_attention_backward(None, None) == EINVAL
    empty = attention(total_q=0, total_k=0, q=0, k=0, v=0, blocks=0, out=0, lse=0, dout=0, dq=0, dk=0, dv=0)
    assert lib.block_attention(ctypes.byref(empty), None) == OK
    assert lib.block_attention_backward(ctypes.byref(empty), None) == OK
    a = attention()
    need = lib.block_attention_workspace(ctypes.byref(a))
    assert need > 0
    for ws, n in ((0, need), (A, need - 1), (A, 0)):
        assert lib.block_attention_backward(ctypes.byref(attention(workspace=ws, workspace_bytes=n)), None) == EWORKSPACE
    assert lib.block_attention_workspace(ctypes.byref(attention(dim=96))) == 0
    assert lib.block_attention_workspace(None) == 0


def test_workspace_grows_with_what_it_holds(lib):
    sizes = [lib.block_attention_workspace(ctypes.byref(attention(total_q=n, total_k=n, select=16))) for n in (1, 100, 4096, 65536)]
    assert sizes == sorted(sizes) and sizes[-1] > 4 * 65536


def scores(**kw):
    base = dict(q=A, means=A, scores=A, counts=A, q_stride_t=256, q_stride_h=64, total_q=10, total_k=10, mean_rows=4, dtype=0,
                num_seqs=1, heads=4, kv_heads=2, dim=64, block_size=16, max_blocks=4, first=1, last=1, scale=0.125)
    return make(binding._ScoreArgs, **{**base, **kw})


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(dim=65), dict(block_size=24), dict(kv_heads=0), dict(heads=5), dict(heads=0), dict(heads=258), dict(total_q=-1),
    dict(total_q=1 << 31), dict(total_k=-1), dict(num_seqs=-1), dict(num_seqs=2), dict(max_blocks=0), dict(first=-1), dict(last=-1),
    dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q_stride_t=-8), dict(q_stride_h=12), dict(mean_rows=-1),
    dict(mean_rows=0), dict(total_k=64), dict(q=0), dict(q=A + 8), dict(means=0), dict(means=A + 4), dict(scores=0), dict(counts=0),
    dict(scores=A + 2), dict(cu_q=A), dict(cu_k=A), dict(block_table=A), dict(block_table=A, lengths=A, block_table_stride=3),
    dict(block_table=A, lengths=A, block_table_stride=4, num_seqs=3), dict(block_table=A + 1, lengths=A, block_table_stride=4, num_seqs=10),
], ids=str)
def test_block_scores_refuses(lib, bad):
    assert lib.block_scores(ctypes.byref(scores(**bad)), None) == EINVAL
    assert lib.block_scores(None, None) == EINVAL
    assert lib.block_scores(ctypes.byref(scores(total_q=0, q=0)), None) == OK


def test_block_means_refuses(lib):
    good = [0, A, 128, 64, 100, 2, 64, 16, None, 1, A, None]
    for at, value in ((0, 2), (1, 0), (1, A + 8), (2, -8), (2, 12), (3, 4), (4, -1), (4, 1 << 31), (5, 0), (6, 96), (7, 40), (8, A + 2),
                      (9, 2), (9, -1), (9, 0), (10, 0), (10, A + 4)):
        args = list(good)
        args[at] = value
        assert lib.block_means(*args) == EINVAL, (at, value)
    assert lib.block_means(0, 0, 0, 0, 0, 2, 64, 16, A, 0, 0, None) == OK


def cache(cls, **kw):
    base = dict(k_cache=A, v_cache=A, k_scale=A, v_scale=A, block_table=A, lengths=A, num_pages=8, block_table_stride=4,
                block_table_cols=4, dtype=0, num_seqs=3, kv_heads=2, dim=64, block_size=16)
    return make(cls, **{**base, **kw})


def append(**kw):
    return cache(binding._AppendArgs, **{**dict(k=A, v=A, k_stride_t=128, k_stride_h=64, v_stride_t=128, v_stride_h=64, total=3), **kw})


def decode(**kw):
    return cache(binding._DecodeArgs, **{**dict(q=A, out=A, lse=A, q_stride_t=256, q_stride_h=64, total_q=3, heads=4, max_length=64,
                                                scale=0.125), **kw})


BAD_CACHE = [dict(dtype=2), dict(dim=96), dict(block_size=20), dict(kv_heads=0), dict(num_pages=-1), dict(num_pages=1 << 31),
             dict(num_seqs=-1), dict(num_seqs=2), dict(block_table_cols=-1), dict(block_table_stride=3), dict(lengths=0),
             dict(block_table=0), dict(lengths=A + 2), dict(block_table=A + 1), dict(k_cache=0), dict(v_cache=0), dict(k_scale=0),
             dict(v_scale=0), dict(k_cache=A + 8), dict(v_cache=A + 4), dict(k_scale=A + 2), dict(cu=A + 2)]


@pytest.mark.parametrize("bad", BAD_CACHE + [dict(k=0), dict(v=0), dict(k=A + 2), dict(k_stride_t=4), dict(v_stride_h=-8), dict(total=-1),
                                             dict(total=1 << 31), dict(k_mean=A + 2)], ids=str)
def test_append_refuses(lib, bad):
    assert lib.kv8_append(ctypes.byref(append(**bad)), None) == EINVAL
    assert lib.kv8_append(None, None) == EINVAL
    assert lib.kv8_append(ctypes.byref(append(total=0, num_seqs=0, k=0, v=0)), None) == OK


@pytest.mark.parametrize("bad", BAD_CACHE + [
    dict(q=0), dict(out=0), dict(lse=0), dict(q=A + 8), dict(out=A + 8), dict(heads=3), dict(heads=0), dict(heads=258), dict(total_q=-1),
    dict(total_q=1 << 31), dict(max_length=-1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q_stride_t=4),
    dict(q_stride_h=-8), dict(blocks=A, select=0), dict(blocks=A, select=1025), dict(blocks=A + 2, select=4),
    dict(block_table_cols=1 << 26, block_table_stride=1 << 26), dict(workspace=A + 8)], ids=str)
def test_decode_refuses(lib, bad):
    assert lib.kv8_attention(ctypes.byref(decode(**bad)), None) == EINVAL


def test_decode_workspace(lib):
    assert lib.kv8_attention(None, None) == EINVAL and lib.kv8_attention_workspace(None) == 0
    assert lib.kv8_attention(ctypes.byref(decode(total_q=0, num_seqs=0, q=0, out=0, lse=0)), None) == OK
    long = dict(block_table_cols=1 << 12, block_table_stride=1 << 12, max_length=1 << 16)
    need = lib.kv8_attention_workspace(ctypes.byref(decode(**long)))
    assert need > 0
    for ws, n in ((0, need), (A, need - 1)):
        assert lib.kv8_attention(ctypes.byref(decode(**long, workspace=ws, workspace_bytes=n)), None) == EWORKSPACE


def test_python_refuses_tensors_of_the_host():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    blocks = torch.zeros(4, 2, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        mt.block_means(q, 16)
    with pytest.raises(ValueError, match="GPU"):
        mt.block_attention(q, q, q, blocks, 16)
    with pytest.raises(ValueError, match="GPU"):
        mt.block_attention(q.requires_grad_(), q, q, blocks, 16)
    with pytest.raises(ValueError, match="3-D"):
        mt.block_means(q.detach().float(), 16)
    with pytest.raises(ValueError, match="3-D"):
        mt.kv8_append(q[0], q, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="block_size"):
        mt.block_means(q, 20)
