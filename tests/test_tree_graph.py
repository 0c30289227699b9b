"""A captured verification step replayed with other lengths: the batch's
layout (prefix sums, cached lengths, trees) is read on the device, so one graph
serves every batch of its sizes."""

import numpy as np
import pytest
import torch

import layer_gram_embedding_gb300 as ple
import tree_reference as ref
from test_tree_ops import BOUNDARY, Cache, DEV, dev, row_id_inputs, rows

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

B, T, HQ, HK, D, PAGE, CAPACITY, P = 5, 60, 8, 2, 128, 16, 2000, 6


def state(rng):
    """Buffers of one shape whatever the lengths: every request has pages for CAPACITY tokens."""
    cache = Cache(rng, [CAPACITY] * B, PAGE, HK, D, torch.bfloat16)
    for c in (cache.k, cache.v):
        c.zero_()
    qkv = torch.zeros((T, HQ + 2 * HK, D), dtype=torch.bfloat16, device=DEV)
    ids, context, M, vocab, off = (dev(x) for x in row_id_inputs(rng, [T // B] * B, 3, 2, 2,
                                                                 np.int64))
    w = rows(rng, (D,), torch.bfloat16)
    return dict(parent=torch.zeros(T, dtype=torch.int32, device=DEV),
                cu=torch.zeros(B + 1, dtype=torch.int32, device=DEV),
                ctx=torch.zeros(B, dtype=torch.int32, device=DEV), ids=ids, context=context,
                M=M, vocab=vocab, off=off, qkv=qkv, w=w, rope=ple.ple_prepare_rope(D),
                k=cache.k, v=cache.v, table=dev(cache.table),
                path=torch.zeros((B, P), dtype=torch.int32, device=DEV),
                accepted=torch.zeros(B, dtype=torch.int32, device=DEV))


def step(s):
    positions, masks = ple.ple_build_tree_index(s["parent"], s["cu"], s["ctx"], 1)
    ids = ple.ple_tree_row_ids(s["ids"], s["parent"], s["cu"], s["context"], s["M"], s["vocab"],
                               s["off"], 3, 2, BOUNDARY)
    q, k, v = s["qkv"][:, :HQ], s["qkv"][:, HQ:HQ + HK], s["qkv"][:, HQ + HK:]
    q = ple.ple_qk_norm_rope(q, k, v, positions, s["rope"], s["w"], s["w"], k_cache=s["k"],
                             v_cache=s["v"], page_table=s["table"], ctx_lens=s["ctx"],
                             cu_seqlens=s["cu"])
    out, lse = ple.ple_tree_attention(q, s["k"], s["v"], s["table"], s["ctx"], s["cu"], masks,
                                      return_lse=True)
    nxt, lens = ple.ple_tree_commit(s["ids"], s["path"], s["accepted"], s["cu"], s["context"],
                                    s["ctx"], s["table"], s["k"], s["v"])
    return [positions, masks, ids, q, out, lse, nxt, lens, s["k"], s["v"]]


def batch(seed, counts, ctx):
    """New contents for the buffers: T nodes, some of them padding behind the last request's."""
    rng = np.random.default_rng(seed)
    parent = np.full(T, -1, np.int32)
    parent[:sum(counts)] = ref.trees(rng, counts)
    path, accepted = np.zeros((B, P), np.int32), np.zeros(B, np.int32)
    for r, n in enumerate(counts):
        accepted[r] = rng.integers(0, min(n, P) + 1)
        path[r, :accepted[r]] = np.sort(rng.choice(n, accepted[r], replace=False))
    shape = (B * -(-CAPACITY // PAGE) + 2, HK, PAGE, D)
    return dict(parent=dev(parent), cu=dev(ref.prefix(counts)), ctx=dev(np.array(ctx, np.int32)),
                ids=dev(rng.integers(0, 1000, T)), context=dev(rng.integers(0, 1000, (B, 2))),
                qkv=rows(rng, (T, HQ + 2 * HK, D), torch.bfloat16),
                k=rows(rng, shape, torch.bfloat16), v=rows(rng, shape, torch.bfloat16),
                path=dev(path), accepted=dev(accepted))


def test_a_graph_serves_other_lengths():
    batches = [batch(1, [12] * 5, [100, 0, 33, 7, 16]), batch(2, [1, 0, 57, 2, 0], [1900, 5, 0, 640, 1]),
               batch(3, [1] * 5, [1800, 1900, 1700, 3, 1990]), batch(4, [0, 0, 60, 0, 0], [0, 0, 1, 0, 0]),
               batch(5, [0] * 5, [4, 5, 6, 7, 8]), batch(6, [20, 20, 4, 0, 1], [0, 1000, 127, 128, 129])]
    s, plain = state(np.random.default_rng(9)), state(np.random.default_rng(9))

    def fill(t, b):
        for key, value in b.items():
            t[key].copy_(value)

    fill(s, batches[0])
    step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(s)
    for b in batches + batches[::-1]:
        fill(s, b)
        fill(plain, b)
        graph.replay()
        want = step(plain)
        torch.cuda.synchronize()
        n = int(b["cu"][-1])   # what lies behind is padding: unspecified
        for i, (x, y) in enumerate(zip(captured, want)):
            if i == 2:
                x, y = x[:, :n], y[:, :n]
            elif i < 6:
                x, y = x[:n], y[:n]
            assert torch.equal(x, y), i
