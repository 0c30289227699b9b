"""Every tensor argument of the tree operators in a wrong dtype, on the host,
with a stride, and longer than the others say, in the form of a call that
allocates its outputs and in the one that is given them: the binding tests a
call's arguments in one expression and names the culprit in another, and both
have to know of each.  Refused calls launch nothing."""

import pytest
import torch

import layer_gram_embedding_gb300 as ple
from test_tree_ops import make_step, step

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

REFUSED = (TypeError, ValueError, ple.PleError)


def forms():
    s = make_step(81)
    step(s)
    T, dev = s["q"].shape[0], "cuda"

    def empty(*shape, dtype=torch.int32):
        return torch.zeros(shape, dtype=dtype, device=dev)

    bf, i64 = torch.bfloat16, torch.int64
    positions, masks = ple.ple_build_tree_index(s["parent"], s["cu"], s["ctx"], 1)
    paged = dict(k_cache=s["kc"], v_cache=s["vc"], page_table=s["table"], ctx_lens=s["ctx"],
                 cu_seqlens=s["cu"])
    index = dict(parent=s["parent"], cu_seqlens=s["cu"], ctx_lens=s["ctx"], mask_words=1)
    rows = dict(input_ids=s["ids"], parent=s["parent"], cu_seqlens=s["cu"],
                ngram_context=s["context"], layer_multipliers=s["M"], vocab_sizes=s["vocab"],
                offsets=s["off"], ngram_size=3, heads_per_ngram=2, boundary_id=7)
    norm = dict(q=s["q"], k=s["k"], v=s["v"], positions=positions, rope=s["rope"],
                q_weight=s["qw"], k_weight=s["kw"], **paged)
    alone = dict(q=s["q"], k=s["k"], v=None, positions=positions, rope=s["rope"],
                 q_weight=s["qw"], k_weight=s["kw"])
    attention = dict(q=s["q"], tree_mask=masks, **paged)
    commit = dict(input_ids=s["ids"], path=s["path"], accepted=torch.zeros_like(s["accepted"]),
                  ngram_context=s["context"], **paged)
    heads = ple.ple_prepare_heads(s["vocab"], s["off"])
    return {
        "index": (ple.ple_build_tree_index, index),
        "index, outputs given": (ple.ple_build_tree_index, dict(
            index, positions=empty(T), tree_mask=empty(T, 1, dtype=i64))),
        "row ids": (ple.ple_tree_row_ids, rows),
        "row ids, outputs given": (ple.ple_tree_row_ids, dict(
            rows, out=empty(1, T, 4, dtype=i64), heads=heads)),
        "norm": (ple.ple_qk_norm_rope, norm),
        "norm, outputs given": (ple.ple_qk_norm_rope, dict(norm, q_out=empty(T, 4, 128, dtype=bf))),
        "norm alone": (ple.ple_qk_norm_rope, alone),
        "norm alone, outputs given": (ple.ple_qk_norm_rope, dict(
            alone, q_out=empty(T, 4, 128, dtype=bf), k_out=empty(T, 2, 128, dtype=bf))),
        "attention": (ple.ple_tree_attention, attention),
        "attention, outputs given": (ple.ple_tree_attention, dict(
            attention, out=empty(T, 4, 128, dtype=bf), lse=empty(T, 4, dtype=torch.float32),
            workspace=ple.ple_tree_attention_workspace(T, 4, 2, 128))),
        "commit": (ple.ple_tree_commit, commit),
        "commit, outputs given": (ple.ple_tree_commit, dict(
            commit, next_context=empty(3, 2, dtype=i64), next_ctx_lens=empty(3))),
    }


NAMES = ["index", "index, outputs given", "row ids", "row ids, outputs given", "norm",
         "norm, outputs given", "norm alone", "norm alone, outputs given", "attention",
         "attention, outputs given", "commit", "commit, outputs given"]


def other_dtype(t):
    return t.to({torch.int32: torch.int64, torch.int64: torch.int32, torch.uint8: torch.int8,
                 torch.bfloat16: torch.float16, torch.float32: torch.float64}[t.dtype])


def strided(t):
    """The same values, every other element of a wider tensor's last dimension."""
    wide = torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype, device=t.device)
    view = wide[..., ::2]
    view.copy_(t)
    return view


def longer(t, dim):
    return torch.cat([t, t.narrow(dim, 0, 1)], dim)


# sizes that a call takes from the argument itself, by form: (argument, dimension)
FREE = {
    "index": {("parent", 0)},
    "norm": {("q", 1), ("page_table", 1)},
    "norm, outputs given": {("page_table", 1)},
    "norm alone": {("q", 1), ("k", 1)},
    "attention": {("page_table", 1), ("tree_mask", 1)},
    "attention, outputs given": {("page_table", 1), ("tree_mask", 1), ("workspace", 0)},
    "commit": {("input_ids", 0), ("path", 1), ("page_table", 1), ("ngram_context", 1)},
    "commit, outputs given": {("input_ids", 0), ("path", 1), ("page_table", 1)},
}


@pytest.mark.parametrize("name", NAMES)
def test_every_argument_is_looked_at(name):
    fn, good = forms()[name]
    fn(**good)
    for key, t in good.items():
        if not isinstance(t, torch.Tensor):
            continue
        bad = {"dtype": other_dtype(t), "host": t.cpu(), "stride": strided(t)}
        for dim in range(t.dim()):
            if (key, dim) not in FREE.get(name, ()):
                bad[f"longer in dimension {dim}"] = longer(t, dim)
        for what, wrong in bad.items():
            try:
                fn(**dict(good, **{key: wrong}))
            except REFUSED:
                continue
            pytest.fail(f"{key}: {what} was taken")
