"""The entry points for caches in 8 bits and for pages without a GPU: the
argument structs' layout, the host checks of the C ABI, the binding's refusals,
and the plain implementations that the GPU tests compare with.  No call here
reaches a launch."""

import contextlib
import ctypes
import os
import shutil
import struct
import subprocess
import types

import numpy as np
import pytest
import torch

import cache_reference as ref8
import layer_gram_embedding_gb300 as ple
from layer_gram_embedding_gb300 import build, cache
from test_tree_abi import FIELDS as TREE_FIELDS, GOOD as TREE_GOOD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000  # a device address that no call below reaches

SCALES = "k v layer_stride page_stride head_stride block".split()
GOOD_SCALES = {"s.k": A, "s.v": A, "s.layer_stride": 1024, "s.page_stride": 2, "s.head_stride": 1,
               "s.block": 16}


def fields_of(tree):
    return ["base." + f for f in TREE_FIELDS[tree][1]] + ["scales." + f for f in SCALES]


PLAN = """page_table ctx_lens source want next_table next_ctx_lens copies counts workspace
    workspace_bytes num_requests num_rows max_pages page_size num_pages page_limit""".split()
COPY = """copies k_cache v_cache layer_stride page_stride head_stride slot_stride scales.k scales.v
    scales.layer_stride scales.page_stride scales.head_stride scales.block num_pages num_copies
    num_layers kv_heads page_size head_dim element_bytes""".split()
FIELDS = {
    "ple_qk_norm_rope_fp8": (cache._NORM_ROPE8, fields_of("ple_qk_norm_rope")),
    "ple_tree_attention_fp8": (cache._ATTENTION8, fields_of("ple_tree_attention")),
    "ple_tree_commit_fp8": (cache._COMMIT8, fields_of("ple_tree_commit")),
    "ple_plan_pages": (cache._PLAN, PLAN),
    "ple_copy_pages": (cache._COPY, COPY),
}
GOOD = {name + "_fp8": dict(TREE_GOOD[name], **GOOD_SCALES)
        for name in ("ple_qk_norm_rope", "ple_tree_attention", "ple_tree_commit")}
GOOD["ple_plan_pages"] = dict(
    page_table=A, ctx_lens=2 * A, source=3 * A, want=4 * A, next_table=5 * A,
    next_ctx_lens=6 * A, copies=7 * A, counts=8 * A, workspace=9 * A, workspace_bytes=2 ** 40,
    num_requests=2, num_rows=3, max_pages=4, page_size=16, num_pages=9, page_limit=9)
GOOD["ple_copy_pages"] = dict(
    {f: v for f, v in GOOD_SCALES.items()}, copies=A, k_cache=A, v_cache=A, layer_stride=65536,
    page_stride=4096, head_stride=1024, slot_stride=64, num_pages=9, num_copies=2, num_layers=3,
    kv_heads=2, page_size=16, head_dim=64, element_bytes=1)
NULL, SIZE, DTYPE, ALIGN, ELEMENT, OK = (ple.PLE_ERR_NULL, ple.PLE_ERR_SIZE, ple.PLE_ERR_DTYPE,
                                         ple.PLE_ERR_ALIGN, ple.PLE_ERR_ELEMENT, ple.PLE_OK)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ple.lib()


def call(lib, name, **kw):
    packer, fields = FIELDS[name]
    kw = {k.replace("s_", "s.", 1) if k.startswith("s_") else k: v for k, v in kw.items()}
    values = dict(GOOD[name], **kw)
    order = [f.replace("scales.", "s.").replace("base.", "") for f in fields]
    assert set(values) == set(order)
    return getattr(lib, name)(packer.pack(*(values[f] for f in order)), None)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a C compiler")
def test_packed_fields_are_the_headers(tmp_path):
    lines = []
    for name, (_, fields) in FIELDS.items():
        for f in fields:
            lines.append(f'printf("%zu %zu\\n", offsetof({name}_args, {f}), '
                         f'sizeof((({name}_args*)0)->{f}));')
        lines.append(f'printf("%zu 0\\n", sizeof({name}_args));')
    src = tmp_path / "offsets.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "ple.h"\nint main(void) {\n'
                   + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "offsets"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    told = iter(subprocess.run([str(exe)], check=True, capture_output=True,
                               text=True).stdout.split())
    for name, (packer, fields) in FIELDS.items():
        # "0q" aligns a nested struct's end: what follows one begins with 8 bytes
        codes = packer.format.lstrip("@").replace("0q", "")
        assert len(codes) == len(fields), name
        for i, f in enumerate(fields):
            at = struct.calcsize("@" + codes[:i] + "0" + codes[i])
            assert (at, struct.calcsize(codes[i])) == (int(next(told)), int(next(told))), f
        assert packer.size == int(next(told)), name
        next(told)


SCALE_CASES = [
    (dict(s_block=0), SIZE), (dict(s_block=8), SIZE), (dict(s_block=48), SIZE),
    (dict(s_block=32), SIZE),       # half a page
    (dict(s_page_stride=-1), SIZE), (dict(s_head_stride=-1), SIZE),
    (dict(s_page_stride=2 ** 61), SIZE), (dict(s_k=A + 1), ALIGN), (dict(s_v=A + 1), ALIGN),
    (dict(page_stride=4104), ALIGN), (dict(head_stride=1032), ALIGN),
    (dict(slot_stride=72), ALIGN), (dict(k_cache=A + 8), ALIGN), (dict(v_cache=A + 4), ALIGN),
]


@pytest.mark.parametrize("kw,status", SCALE_CASES + [
    (dict(s_k=0), NULL), (dict(s_v=0), NULL),
    (dict(num_tokens=-1), SIZE), (dict(num_tokens=2 ** 31), SIZE), (dict(q_heads=-1), SIZE),
    (dict(kv_heads=0), SIZE), (dict(q_heads=65535), SIZE), (dict(head_dim=8), SIZE),
    (dict(head_dim=72), SIZE), (dict(head_dim=272), SIZE), (dict(rotary_dim=63), SIZE),
    (dict(rotary_dim=66), SIZE), (dict(rotary_dim=-2), SIZE), (dict(eps=-1.0), SIZE),
    (dict(eps=float("nan")), SIZE), (dict(rope_scale=float("inf")), SIZE),
    (dict(num_requests=0), SIZE), (dict(num_pages=0), SIZE), (dict(num_pages=2 ** 31), SIZE),
    (dict(max_pages=0), SIZE), (dict(max_pages=2 ** 20, page_size=2 ** 11), SIZE),
    (dict(page_stride=2 ** 60), SIZE), (dict(q_token=2 ** 60), SIZE), (dict(k_head=-8), SIZE),
    (dict(v_token=2 ** 60), SIZE), (dict(dtype=2), ELEMENT), (dict(q=0), NULL), (dict(k=0), NULL),
    (dict(v=0), NULL), (dict(q_out=0), NULL), (dict(positions=0), NULL), (dict(rope=0), NULL),
    (dict(k_cache=0), NULL), (dict(v_cache=0), NULL), (dict(page_table=0), NULL),
    (dict(ctx_lens=0), NULL), (dict(cu_seqlens=0), NULL), (dict(q=A + 8), ALIGN),
    (dict(q_weight=A + 4), ALIGN), (dict(q_token=516), ALIGN), (dict(positions=A + 2), ALIGN),
    (dict(rope=A + 4), ALIGN), (dict(num_tokens=0, q=0, k=0, v=0, q_out=0), OK),
])
def test_qk_norm_rope_fp8_host_checks(lib, kw, status):
    assert call(lib, "ple_qk_norm_rope_fp8", **kw) == status


@pytest.mark.parametrize("kw,status", SCALE_CASES + [
    (dict(s_k=0), NULL), (dict(s_v=0), NULL),
    (dict(num_tokens=-1), SIZE), (dict(kv_heads=0), SIZE), (dict(kv_heads=3), SIZE),
    (dict(q_heads=65536 * 2, kv_heads=65536), SIZE), (dict(head_dim=8), SIZE),
    (dict(head_dim=72), SIZE), (dict(head_dim=272), SIZE), (dict(mask_words=0), SIZE),
    (dict(mask_words=9), SIZE), (dict(scale=float("nan")), SIZE), (dict(num_requests=0), SIZE),
    (dict(num_pages=0), SIZE), (dict(max_pages=2 ** 27, page_size=16), SIZE),
    (dict(max_pages=2 ** 27 - 1, page_size=16), SIZE),     # a tile of 128 would pass 31 bits
    (dict(page_stride=0), SIZE), (dict(head_stride=0), SIZE), (dict(slot_stride=0), SIZE),
    (dict(slot_stride=2 ** 40), SIZE), (dict(dtype=7), ELEMENT), (dict(q=0), NULL),
    (dict(k_cache=0), NULL), (dict(v_cache=0), NULL), (dict(page_table=0), NULL),
    (dict(ctx_lens=0), NULL), (dict(cu_seqlens=0), NULL), (dict(tree_mask=0), NULL),
    (dict(out=0), NULL), (dict(workspace=0), NULL), (dict(q=A + 2), ALIGN),
    (dict(out=A + 8), ALIGN), (dict(lse=A + 2), ALIGN), (dict(tree_mask=A + 4), ALIGN),
    (dict(workspace=A + 8), ALIGN), (dict(q_head=60), ALIGN), (dict(num_tokens=0, q=0), OK),
])
def test_tree_attention_fp8_host_checks(lib, kw, status):
    assert call(lib, "ple_tree_attention_fp8", **kw) == status


@pytest.mark.parametrize("kw,status", SCALE_CASES + [
    (dict(s_k=0), NULL), (dict(s_v=0), NULL), (dict(s_layer_stride=-1), SIZE),
    (dict(s_layer_stride=2 ** 61), SIZE), (dict(layer_stride=65544), ALIGN),
    (dict(num_requests=-1), SIZE), (dict(path_len=0), SIZE), (dict(num_layers=0), SIZE),
    (dict(num_layers=65536), SIZE), (dict(layer_stride=-16), SIZE), (dict(head_dim=8), SIZE),
    (dict(ctx_len=0), SIZE), (dict(ctx_len=16), SIZE), (dict(layer_stride=2 ** 62), SIZE),
    (dict(kv_heads=0), SIZE), (dict(num_tokens=-1), SIZE), (dict(id_dtype=2), DTYPE),
    (dict(path=0), NULL), (dict(accepted=0), NULL), (dict(cu_seqlens=0), NULL),
    (dict(ctx_lens=0), NULL), (dict(next_ctx_lens=0), NULL), (dict(page_table=0), NULL),
    (dict(k_cache=0), NULL), (dict(v_cache=0), NULL), (dict(input_ids=0), NULL),
    (dict(next_context=0), NULL), (dict(path=A + 2), ALIGN), (dict(ngram_context=A + 4), ALIGN),
    (dict(next_ctx_lens=A), SIZE),      # over ctx_lens
    (dict(num_requests=0, path=0), OK),
])
def test_tree_commit_fp8_host_checks(lib, kw, status):
    good = dict(next_ctx_lens=20 * A, next_context=30 * A)
    assert call(lib, "ple_tree_commit_fp8", **dict(good, **kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(num_requests=-1), SIZE), (dict(num_rows=0), SIZE), (dict(max_pages=0), SIZE),
    (dict(page_size=0), SIZE), (dict(max_pages=2 ** 20, page_size=2 ** 11), SIZE),
    (dict(num_pages=0), SIZE), (dict(page_limit=-1), SIZE), (dict(page_limit=10), SIZE),
    (dict(num_rows=2 ** 29), SIZE), (dict(num_rows=2 ** 15, max_pages=2 ** 16), SIZE),
    (dict(workspace_bytes=0), SIZE),
    (dict(page_table=0), NULL), (dict(ctx_lens=0), NULL), (dict(source=0), NULL),
    (dict(want=0), NULL), (dict(next_table=0), NULL), (dict(next_ctx_lens=0), NULL),
    (dict(copies=0), NULL), (dict(counts=0), NULL), (dict(workspace=0), NULL),
    (dict(page_table=A + 2), ALIGN), (dict(copies=7 * A + 2), ALIGN),
    (dict(workspace=9 * A + 4), ALIGN), (dict(next_table=A + 16), SIZE),
    (dict(next_ctx_lens=2 * A), SIZE), (dict(counts=3 * A + 8), SIZE), (dict(copies=4 * A), SIZE),
    (dict(workspace=5 * A + 32), SIZE), (dict(next_ctx_lens=5 * A), SIZE),
])
def test_plan_pages_host_checks(lib, kw, status):
    assert call(lib, "ple_plan_pages", **kw) == status


@pytest.mark.parametrize("kw,status", [c for c in SCALE_CASES if "v_cache" not in c[0]] + [
    (dict(s_k=0), SIZE), (dict(s_v=0), SIZE), (dict(s_layer_stride=-1), SIZE),
    (dict(num_copies=-1), SIZE), (dict(num_layers=0), SIZE), (dict(num_layers=65536), SIZE),
    (dict(layer_stride=-16), SIZE), (dict(layer_stride=8), ALIGN), (dict(element_bytes=0), SIZE),
    (dict(element_bytes=4), SIZE), (dict(element_bytes=2), SIZE),      # with scales
    (dict(element_bytes=2, s_k=0, s_v=0, head_dim=4), SIZE), (dict(head_dim=0), SIZE),
    (dict(head_dim=72), SIZE), (dict(head_dim=272), SIZE), (dict(kv_heads=0), SIZE),
    (dict(num_pages=0), SIZE), (dict(page_size=0), SIZE),
    (dict(s_k=0, s_v=0, page_size=2 ** 30, slot_stride=64), SIZE),     # more shares than a grid has
    (dict(copies=0), NULL), (dict(k_cache=0), NULL), (dict(v_cache=0), NULL),
    (dict(copies=A + 4), ALIGN), (dict(num_copies=0, copies=0), OK),
    (dict(element_bytes=2, s_k=0, s_v=0, slot_stride=68), ALIGN),
])
def test_copy_pages_host_checks(lib, kw, status):
    assert call(lib, "ple_copy_pages", **kw) == status


@pytest.mark.parametrize("args", [(-1, 4, 2, 64), (5, 4, 3, 64), (5, 4, 0, 64), (5, 4, 2, 72)])
def test_workspace_of_sizes_out_of_range(lib, args):
    assert lib.ple_tree_attention_fp8_workspace(*args) == -1


def test_workspace_of_a_plan(lib):
    assert lib.ple_plan_pages_workspace(0, 5) == -1 and lib.ple_plan_pages_workspace(5, 0) == -1
    assert lib.ple_plan_pages_workspace(1, 1) > 0
    # sizes that 32 bits do not hold
    assert lib.ple_plan_pages_workspace(1, 2 ** 31 - 1) > 2 ** 34


def test_a_null_struct_is_refused(lib):
    for name in FIELDS:
        assert getattr(lib, name)(ctypes.c_char_p(None), None) == NULL


def test_binding_refuses_cpu_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((4, 2, 16, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones((4, 2, 1), dtype=torch.bfloat16)
    t = torch.zeros((3, 1), dtype=torch.int32)
    m = torch.zeros((4, 1), dtype=torch.int64)
    ids = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        ple.ple_qk_norm_rope_fp8(x, x, x, i, ids, None, None, c, c, s, s, t, i[:3], i)
    with pytest.raises(ValueError, match="CUDA"):
        ple.ple_tree_attention_fp8(x, c, c, s, s, t, i[:3], i, m)
    with pytest.raises(ValueError, match="CUDA"):
        ple.ple_tree_commit_fp8(ids, t, i[:3], i, None, i[:3], t, c, c, s, s)
    with pytest.raises(ValueError, match="CUDA"):
        ple.ple_plan_pages(t, i[:3], i, i, 9, 16)
    with pytest.raises(ValueError, match="CUDA"):
        ple.ple_copy_pages(t.view(-1)[:2].view(1, 2), c, c, s, s)


def test_a_failed_workspace_query_is_not_kept(monkeypatch):
    answers, asked = [-1, 4096], []

    def query(*sizes):
        asked.append(sizes)
        return answers.pop(0)

    monkeypatch.setattr(cache, "lib",
                        lambda: types.SimpleNamespace(ple_tree_attention_fp8_workspace=query))
    monkeypatch.setattr(cache, "_workspace_sizes", {})
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    assert cache._workspace_size(5, 8, 2, 64, 0) == 0
    assert cache._workspace_size(5, 8, 2, 64, 0) == 4096
    assert cache._workspace_size(5, 8, 2, 64, 0) == 4096
    assert len(asked) == 2


# ------------------------------------------------- the plain implementations


def test_reference_elements_are_torchs():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.uniform(-4, 2, 20000),
                        ref8.VALUES, (ref8.POSITIVE[1:] + ref8.POSITIVE[:-1]) / 2,
                        -(ref8.POSITIVE[1:] + ref8.POSITIVE[:-1]) / 2, [0.0, -0.0]])
    x = x[np.abs(np.nan_to_num(x)) <= 448].astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = ref8.encode(x)
    nan = np.isnan(x)
    assert np.array_equal(got[~nan], want[~nan]) and np.all(got[nan] & 0x7F == 0x7F)


@pytest.mark.parametrize("most,k", [(448.0, 0), (448.5, 1), (224.0, -1), (1.0, -8), (1.75, -8),
                                    (1.76, -7), (0.0, -100), (2.0 ** -99, -100), (3e38, 120)])
def test_reference_scales(most, k):
    assert ref8.scale_for(most) == k


def test_reference_plan_of_a_fork_by_hand():
    table = np.array([[4, 2, 0, -1], [1, 5, -1, -1]], np.int32)
    # request 0 (11 tokens, pages of 4) forks in two that write; request 1 goes on unwritten
    got = ref8.plan(table, [11, 8], [0, 0, 1, -1], [1, 2, 0, 5], 8, 4, 8)
    assert got[0].tolist() == [[4, 2, 0, -1], [4, 2, 3, 6], [1, 5, -1, -1], [7, -1, -1, -1]]
    assert got[1].tolist() == [11, 11, 8, 0]
    assert got[2] == [(0, 3)] and got[3] == [1, 8, 1]
