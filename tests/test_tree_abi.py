"""The tree-verification entry points without a GPU: the argument structs'
layout, the host checks of the C ABI, and the binding's refusals.  No call
here reaches a launch."""

import ctypes
import os
import shutil
import struct
import subprocess

import pytest
import torch

import layer_gram_embedding_gb300 as ple
from layer_gram_embedding_gb300 import build, tree

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000  # a device address that no call below reaches

FIELDS = {
    "ple_qk_norm_rope": (tree._NORM_ROPE, """q k v q_token q_head k_token k_head v_token v_head
        positions rope q_weight k_weight q_out q_out_token q_out_head k_out k_out_token k_out_head
        k_cache v_cache page_stride head_stride slot_stride num_pages page_table ctx_lens
        cu_seqlens num_tokens num_requests max_pages page_size dtype q_heads kv_heads head_dim
        rotary_dim interleaved rope_scale eps""".split()),
    "ple_tree_attention": (tree._ATTENTION, """q q_token q_head k_cache v_cache page_stride
        head_stride slot_stride num_pages page_table ctx_lens cu_seqlens tree_mask out lse
        workspace workspace_bytes num_tokens num_requests max_pages page_size dtype q_heads
        kv_heads head_dim mask_words scale""".split()),
    "ple_tree_commit": (tree._COMMIT, """input_ids path accepted cu_seqlens ngram_context
        next_context ctx_lens next_ctx_lens page_table k_cache v_cache layer_stride page_stride
        head_stride slot_stride num_pages num_tokens num_requests path_len id_dtype ctx_len
        num_layers max_pages page_size kv_heads head_dim dtype""".split()),
}
GOOD = {
    "ple_qk_norm_rope": dict(
        q=A, k=A, v=A, q_token=512, q_head=64, k_token=512, k_head=64, v_token=512, v_head=64,
        positions=A, rope=A, q_weight=A, k_weight=A, q_out=A, q_out_token=512, q_out_head=64,
        k_out=0, k_out_token=0, k_out_head=0, k_cache=A, v_cache=A, page_stride=4096,
        head_stride=1024, slot_stride=64, num_pages=9, page_table=A, ctx_lens=A, cu_seqlens=A,
        num_tokens=5, num_requests=2, max_pages=4, page_size=16, dtype=0, q_heads=4, kv_heads=2,
        head_dim=64, rotary_dim=64, interleaved=0, rope_scale=1.0, eps=1e-6),
    "ple_tree_attention": dict(
        q=A, q_token=512, q_head=64, k_cache=A, v_cache=A, page_stride=4096, head_stride=1024,
        slot_stride=64, num_pages=9, page_table=A, ctx_lens=A, cu_seqlens=A, tree_mask=A, out=A,
        lse=A, workspace=A, workspace_bytes=2 ** 40, num_tokens=5, num_requests=2, max_pages=4,
        page_size=16, dtype=0, q_heads=4, kv_heads=2, head_dim=64, mask_words=1, scale=0.125),
    "ple_tree_commit": dict(
        input_ids=A, path=A, accepted=A, cu_seqlens=A, ngram_context=A, next_context=A,
        ctx_lens=A, next_ctx_lens=A, page_table=A, k_cache=A, v_cache=A, layer_stride=65536,
        page_stride=4096, head_stride=1024, slot_stride=64, num_pages=9, num_tokens=5,
        num_requests=2, path_len=3, id_dtype=1, ctx_len=2, num_layers=3, max_pages=4,
        page_size=16, kv_heads=2, head_dim=64, dtype=0),
}
NULL, SIZE, DTYPE, ALIGN, ELEMENT, OK = (ple.PLE_ERR_NULL, ple.PLE_ERR_SIZE, ple.PLE_ERR_DTYPE,
                                         ple.PLE_ERR_ALIGN, ple.PLE_ERR_ELEMENT, ple.PLE_OK)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ple.lib()


def call(lib, name, **kw):
    packer, fields = FIELDS[name]
    values = dict(GOOD[name], **kw)
    assert set(values) == set(fields)
    return getattr(lib, name)(packer.pack(*(values[f] for f in fields)), None)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a C compiler")
def test_packed_fields_are_the_headers(tmp_path):
    lines = []
    for name, (_, fields) in FIELDS.items():
        for f in fields:
            lines.append(f'printf("%zu %zu\\n", offsetof({name}_args, {f}), '
                         f'sizeof((({name}_args*)0)->{f}));')
    src = tmp_path / "offsets.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "ple.h"\nint main(void) {\n'
                   + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "offsets"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    told = iter(subprocess.run([str(exe)], check=True, capture_output=True,
                               text=True).stdout.split())
    for name, (packer, fields) in FIELDS.items():
        codes = packer.format.lstrip("@")
        assert len(codes) == len(fields), name
        for i, f in enumerate(fields):
            at = struct.calcsize("@" + codes[:i] + "0" + codes[i])
            assert (at, struct.calcsize(codes[i])) == (int(next(told)), int(next(told))), f


@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), SIZE), (dict(num_tokens=2 ** 31), SIZE), (dict(q_heads=-1), SIZE),
    (dict(q_heads=0, kv_heads=0), SIZE), (dict(q_heads=65535), SIZE), (dict(head_dim=4), SIZE),
    (dict(head_dim=68), SIZE), (dict(head_dim=264), SIZE), (dict(rotary_dim=63), SIZE),
    (dict(rotary_dim=66), SIZE), (dict(rotary_dim=-2), SIZE), (dict(eps=-1.0), SIZE),
    (dict(eps=float("nan")), SIZE), (dict(rope_scale=float("inf")), SIZE),
    (dict(num_requests=0), SIZE), (dict(num_pages=0), SIZE), (dict(num_pages=2 ** 31), SIZE),
    (dict(page_size=0), SIZE), (dict(max_pages=0), SIZE),
    (dict(max_pages=2 ** 20, page_size=2 ** 11), SIZE), (dict(page_stride=-8), SIZE),
    (dict(page_stride=2 ** 60), SIZE), (dict(q_token=2 ** 60), SIZE), (dict(k_head=-8), SIZE),
    (dict(v_token=2 ** 60), SIZE), (dict(dtype=2), ELEMENT), (dict(dtype=-1), ELEMENT),
    (dict(q=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL), (dict(q_out=0), NULL),
    (dict(positions=0), NULL), (dict(rope=0), NULL), (dict(v_cache=0), NULL),
    (dict(k_cache=0), NULL), (dict(page_table=0), NULL), (dict(ctx_lens=0), NULL),
    (dict(cu_seqlens=0), NULL), (dict(k_cache=0, v_cache=0), NULL),  # then k_out is wanted
    (dict(q=A + 8), ALIGN), (dict(k_cache=A + 2), ALIGN), (dict(q_weight=A + 4), ALIGN),
    (dict(q_token=516), ALIGN), (dict(slot_stride=68), ALIGN), (dict(positions=A + 2), ALIGN),
    (dict(rope=A + 4), ALIGN), (dict(k_cache=0, v_cache=0, k_out=A + 8), ALIGN),
    (dict(num_tokens=0, q=0, k=0, v=0, q_out=0), OK),
    # no rotation: neither positions nor rope are looked at, nor a cache's arguments without one
    (dict(rotary_dim=0, positions=0, rope=0, q_weight=0, k_weight=0, slot_stride=63), ALIGN),
])
def test_qk_norm_rope_host_checks(lib, kw, status):
    assert call(lib, "ple_qk_norm_rope", **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), SIZE), (dict(kv_heads=0), SIZE), (dict(kv_heads=3), SIZE),
    (dict(q_heads=65536 * 2, kv_heads=65536), SIZE), (dict(head_dim=100), SIZE),
    (dict(head_dim=512), SIZE), (dict(mask_words=0), SIZE), (dict(mask_words=9), SIZE),
    (dict(scale=float("nan")), SIZE), (dict(num_requests=0), SIZE), (dict(num_pages=0), SIZE),
    (dict(page_size=0), SIZE), (dict(max_pages=2 ** 30, page_size=2), SIZE),
    (dict(dtype=7), ELEMENT), (dict(q=0), NULL), (dict(k_cache=0), NULL), (dict(v_cache=0), NULL),
    (dict(page_table=0), NULL), (dict(ctx_lens=0), NULL), (dict(cu_seqlens=0), NULL),
    (dict(tree_mask=0), NULL), (dict(out=0), NULL), (dict(workspace=0), NULL),
    (dict(q=A + 2), ALIGN), (dict(v_cache=A + 8), ALIGN), (dict(out=A + 8), ALIGN),
    (dict(lse=A + 2), ALIGN), (dict(tree_mask=A + 4), ALIGN), (dict(workspace=A + 8), ALIGN),
    (dict(q_head=60), ALIGN), (dict(head_stride=1028), ALIGN), (dict(num_tokens=0, q=0), OK),
])
def test_tree_attention_host_checks(lib, kw, status):
    assert call(lib, "ple_tree_attention", **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(num_requests=-1), SIZE), (dict(path_len=0), SIZE), (dict(num_layers=0), SIZE),
    (dict(num_layers=65536), SIZE), (dict(layer_stride=-8), SIZE), (dict(head_dim=12), SIZE),
    (dict(ctx_len=0), SIZE), (dict(ctx_len=16), SIZE), (dict(num_pages=0), SIZE),
    (dict(layer_stride=2 ** 62), SIZE), (dict(kv_heads=0), SIZE), (dict(num_tokens=-1), SIZE),
    (dict(id_dtype=2), DTYPE), (dict(dtype=2), ELEMENT), (dict(path=0), NULL),
    (dict(accepted=0), NULL), (dict(cu_seqlens=0), NULL), (dict(ctx_lens=0), NULL),
    (dict(next_ctx_lens=0), NULL), (dict(page_table=0), NULL), (dict(k_cache=0), NULL),
    (dict(v_cache=0), NULL), (dict(input_ids=0), NULL), (dict(next_context=0), NULL),
    (dict(layer_stride=65540), ALIGN), (dict(k_cache=A + 8), ALIGN), (dict(path=A + 2), ALIGN),
    (dict(ngram_context=A + 4), ALIGN), (dict(id_dtype=0, input_ids=A + 2), ALIGN),
    (dict(num_requests=0, path=0), OK),
])
def test_tree_commit_host_checks(lib, kw, status):
    assert call(lib, "ple_tree_commit", **kw) == status


@pytest.mark.parametrize("args,status", [
    ((A, A, A, 2, -1, 1, A, A), SIZE), ((A, A, A, 2, 2 ** 31, 1, A, A), SIZE),
    ((A, A, A, 0, 5, 1, A, A), SIZE), ((A, A, A, 2, 5, 0, A, A), SIZE),
    ((A, A, A, 2, 5, 9, A, A), SIZE), ((None, A, A, 2, 5, 1, A, A), NULL),
    ((A, None, A, 2, 5, 1, A, A), NULL), ((A, A, None, 2, 5, 1, A, A), NULL),
    ((A, A, A, 2, 5, 1, None, A), NULL), ((A, A, A, 2, 5, 1, A, None), NULL),
    ((A + 2, A, A, 2, 5, 1, A, A), ALIGN), ((A, A, A, 2, 5, 1, A, A + 4), ALIGN),
    ((None, None, None, 0, 0, 1, None, None), OK),
])
def test_build_tree_index_host_checks(lib, args, status):
    assert lib.ple_build_tree_index(*args, None) == status


def tree_row_ids(lib, **kw):
    a = dict(ids=A, dtype=1, T=64, parent=A, cu=A, ctx=A, B=1, C=2, M=A, vocab=A, off=A, H=4, N=3,
             hpn=2, L=1, b=7, out=A, out_dtype=1, heads=None)
    a.update(kw)
    return lib.ple_tree_row_ids(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=1, C=0, H=0), SIZE), (dict(N=17, C=16, H=32), SIZE), (dict(hpn=0, H=0), SIZE),
    (dict(L=0), SIZE), (dict(T=-1), SIZE), (dict(T=2 ** 31), SIZE),
    (dict(T=2 ** 30, L=2 ** 30), SIZE), (dict(C=3), ple.PLE_ERR_GEOMETRY_CTX),
    (dict(H=5), ple.PLE_ERR_GEOMETRY_HEADS), (dict(hpn=200, H=400), SIZE), (dict(B=0), SIZE),
    (dict(ids=None), NULL), (dict(parent=None), NULL), (dict(cu=None), NULL),
    (dict(ctx=None), NULL), (dict(M=None), NULL), (dict(vocab=None), NULL), (dict(off=None), NULL),
    (dict(out=None), NULL), (dict(dtype=2), DTYPE), (dict(out_dtype=2), DTYPE),
    (dict(ids=A + 4), ALIGN), (dict(parent=A + 2), ALIGN), (dict(out=A + 4), ALIGN),
    (dict(heads=A + 8), ALIGN), (dict(vocab=None, off=None, heads=A, ids=None), NULL),
    (dict(T=0, ids=None, parent=None, out=None), OK),
])
def test_tree_row_ids_host_checks(lib, kw, status):
    assert tree_row_ids(lib, **kw) == status


@pytest.mark.parametrize("args,status", [
    ((0, 1e4, 0, 1.0, 0.0, 0.0, 0.0, A), SIZE), ((63, 1e4, 0, 1.0, 0.0, 0.0, 0.0, A), SIZE),
    ((258, 1e4, 0, 1.0, 0.0, 0.0, 0.0, A), SIZE), ((64, 0.5, 0, 1.0, 0.0, 0.0, 0.0, A), SIZE),
    ((64, float("nan"), 0, 1.0, 0.0, 0.0, 0.0, A), SIZE),
    ((64, 1e4, 4, 1.0, 0.0, 0.0, 0.0, A), SIZE), ((64, 1e4, -1, 1.0, 0.0, 0.0, 0.0, A), SIZE),
    ((64, 1e4, 1, 0.5, 0.0, 0.0, 0.0, A), SIZE), ((64, 1e4, 3, 2.0, 0.0, 32.0, 1.0, A), SIZE),
    ((64, 1e4, 3, 2.0, 4096.0, 1.0, 1.0, A), SIZE), ((64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, None), NULL),
    ((64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, A + 4), ALIGN),
])
def test_prepare_rope_host_checks(lib, args, status):
    assert lib.ple_prepare_rope(*args, None) == status


@pytest.mark.parametrize("args", [(-1, 4, 2, 64), (5, 4, 3, 64), (5, 4, 0, 64), (5, 4, 2, 65)])
def test_workspace_of_sizes_out_of_range(lib, args):
    assert lib.ple_tree_attention_workspace(*args) == -1


def test_a_null_struct_is_refused(lib):
    for name in FIELDS:
        assert getattr(lib, name)(ctypes.c_char_p(None), None) == NULL
    assert ple.status_string(ple.PLE_ERR_ELEMENT) != "unknown status"


def test_binding_refuses_cpu_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    t = torch.zeros((3, 1), dtype=torch.int32)
    m = torch.zeros((4, 1), dtype=torch.int64)
    ids = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        ple.ple_build_tree_index(i, i, i[:3], 1)
    with pytest.raises(ValueError, match="CUDA"):
        ple.ple_tree_row_ids(ids, i, i, m, m, m, m, 3, 2, 7)
    with pytest.raises(ValueError, match="CUDA"):
        ple.ple_prepare_rope(64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        ple.ple_qk_norm_rope(x, x, x, i, ids)
    with pytest.raises(ValueError, match="CUDA"):
        ple.ple_tree_attention(x, c, c, t, i[:3], i, m)
    with pytest.raises(ValueError, match="CUDA"):
        ple.ple_tree_commit(ids, t, i[:3], i, None, i[:3], t, c, c)
