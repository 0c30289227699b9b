"""Corners of the operators on caches in 8 bits and on pages, on the GPU: queries
that are not finite, many requests, rows in place, the same tensor for both
caches, prompts and decodes in one call, captured steps that share nothing."""

import numpy as np
import pytest
import torch

import cache_reference as ref8
import layer_gram_embedding_gb300 as ple
import tree_reference as ref
from test_cache_ops import (Cache8, KERNELS, attention_inputs, check_append, check_attention,
                            check_plan, read, same)
from test_cache_steps import equal, make_step, state, step
from test_tree_ops import U, check_rows, dev, host, rows

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("counts,Hq", KERNELS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_queries_that_are_not_finite_stay_in_their_rows(counts, Hq, dtype, bad):
    rng = np.random.default_rng(91)
    q, cache, ctx, cu, masks = attention_inputs(rng, counts, [700], Hq, 2, 64, 32, 16, dtype)
    want, want_lse = check_attention(q, cache, ctx, cu, masks)
    q = q.clone()
    q[1, Hq - 1, 5] = bad
    out, lse = ple.ple_tree_attention_fp8(q, *cache.device(), dev(cache.table), dev(ctx), dev(cu),
                                          dev(masks), return_lse=True)
    assert bool(out[1, Hq - 1].isnan().all())
    out[1, Hq - 1], lse[1, Hq - 1] = want[1, Hq - 1], want_lse[1, Hq - 1]
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("counts,Hq", KERNELS)
def test_tiny_and_large_queries(counts, Hq):
    # rows of 2^-120 and of 2^100 beside others; keys as small as makes the scores ordinary
    rng = np.random.default_rng(92)
    q, cache, ctx, cu, masks = attention_inputs(rng, counts, [300], Hq, 2, 64, 32, 16,
                                                torch.bfloat16, low=-12, high=-12)
    q[0] *= 2.0 ** -120
    check_attention(q, cache, ctx, cu, masks)
    q[:] = rows(rng, tuple(q.shape), torch.bfloat16, 2.0 ** 90)
    live = cache.k_scale == 2.0 ** -12
    cache.k_scale[live] = 2.0 ** -98
    check_attention(q, cache, ctx, cu, masks)


@pytest.mark.parametrize("nodes", [1, 6])
def test_many_requests(nodes):
    # more requests than a block has threads
    rng = np.random.default_rng(93)
    B = 1100
    counts = [nodes if i % 7 else 0 for i in range(B)]
    ctx = [int(x) for x in rng.integers(0, 60, B)]
    q, cache, ctx, cu, masks = attention_inputs(rng, counts, ctx, 8, 2, 32, 16, 16, torch.bfloat16)
    check_attention(q, cache, ctx, cu, masks)
    qkv = [rows(rng, (sum(counts), h, 32), torch.bfloat16) for h in (8, 2, 2)]
    caches = cache.device()
    before = read(caches)
    got = ple.ple_qk_norm_rope_fp8(*qkv, None, None, None, None, *caches, dev(cache.table),
                                   dev(ctx), dev(cu))
    assert torch.equal(got, qkv[0])
    after = read(caches)
    for i in (0, 1):
        x = host(qkv[i + 1])
        check_append((after[i][0], after[i + 2][0]), (before[i][0], before[i + 2][0]), x,
                     np.zeros(x.shape), cache.table, ctx, cu, exact=True)


def test_prompts_and_decodes_in_one_call():
    rng = np.random.default_rng(94)
    counts = [1, 200, 1, 1, 64, 1, 1, 17, 1, 1]
    ctx = [900, 0, 15, 16, 300, 2000, 1, 31, 0, 77]
    args = attention_inputs(rng, counts, ctx, 8, 2, 128, 64, 32, torch.bfloat16)
    check_attention(*args)


@pytest.mark.parametrize("D,R", [(128, 128), (64, 32)])
def test_queries_in_place(D, R):
    rng = np.random.default_rng(95)
    qkv = rows(rng, (40, 8, D), torch.bfloat16)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    positions = rng.integers(0, 2 ** 31, 40).astype(np.int32)
    cache = Cache8(rng, [40], 48, 16, 2, D)
    w = ref.inverse_frequencies(R, 10000.0)
    want, size = ref.norm_rope(host(q), None, positions, w, 0.0, False, 1.0)
    got = ple.ple_qk_norm_rope_fp8(q, k, v, dev(positions), ple.ple_prepare_rope(R), None, None,
                                   *cache.device(), dev(cache.table), dev(np.zeros(1, np.int32)),
                                   dev(np.array([0, 40], np.int32)), q_out=q)
    assert got is q
    check_rows(q, want, size, U[torch.bfloat16], "q")


@pytest.mark.parametrize("page,block,D", [(128, 128, 256), (128, 64, 256), (256, 128, 128)])
@pytest.mark.parametrize("Hk", [1, 40, 140])
def test_append_whose_angles_come_in_parts(page, block, D, Hk):
    # blocks whose angles are worked out table by table: parts of blocks, infinities in one part
    # and not in another, heads enough for more tasks a warp than it walks with at once
    rng = np.random.default_rng(96)
    counts, ctx = [300, 1, 100, 40], np.array([0, 5, 70, 127], np.int32)
    cu, T = ref.prefix(counts), 441
    q, k, v = (rows(rng, (T, h, D), torch.float16) for h in (2, Hk, Hk))
    k[130, 0, 3] = v[131, 0, 7] = float("inf")
    v[260, -1, 9] = float("nan")
    k[50:70] *= 30
    cache = Cache8(rng, [int(c) + n for c, n in zip(ctx, counts)], page, block, Hk, D)
    for r in range(4):
        cache.fill(rng, r, int(ctx[r]) // block * block, int(ctx[r]), -20, -4, any_scale=r == 3)
    positions = rng.integers(0, 100000, T).astype(np.int32)
    kw = rows(rng, (D,), torch.float16)
    w = ref.inverse_frequencies(D, 1e6)
    caches = cache.device()
    before = read(caches)
    ple.ple_qk_norm_rope_fp8(q, k, v, dev(positions), ple.ple_prepare_rope(D, 1e6), None, kw,
                             *caches, dev(cache.table), dev(ctx), dev(cu))
    after = read(caches)
    with np.errstate(invalid="ignore"):
        want, size = ref.norm_rope(host(k), host(kw), positions, w, 1e-6, False, 1.0)
    check_append((after[0][0], after[2][0]), (before[0][0], before[2][0]), want,
                 2.0 ** -20 * size + 2.0 ** -40, cache.table, ctx, cu, exact=False)
    check_append((after[1][0], after[3][0]), (before[1][0], before[3][0]), host(v),
                 np.zeros(v.shape), cache.table, ctx, cu, exact=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("counts", [[5, 4, 3, 4], [8, 0, 7, 1], [1, 30, 0, 0], [2, 2, 3, 3]])
def test_page_tables_with_room_for_long_contexts(D, counts):
    # the kernel is chosen by rows a key head and the tables' width: 8 to 32 rows in wide ones
    rng = np.random.default_rng(103)
    q, cache, ctx, cu, masks = attention_inputs(rng, counts, [700, 3, 129, 64], 16, 4, D, 128, 32,
                                                torch.bfloat16)
    narrow = check_attention(q, cache, ctx, cu, masks)
    cache.table = np.concatenate([cache.table, np.full((4, 2000), -1, np.int32)], 1)
    wide = check_attention(q, cache, ctx, cu, masks)
    assert narrow[0].shape == wide[0].shape


def test_one_tensor_for_keys_and_values():
    # attention reads them alone: they may be one
    rng = np.random.default_rng(97)
    q, cache, ctx, cu, masks = attention_inputs(rng, [3, 40], [200, 100], 4, 2, 64, 16, 16,
                                                torch.bfloat16)
    cache.v, cache.v_scale = cache.k, cache.k_scale
    k, _, s, _ = cache.device()
    check_attention(q, cache, ctx, cu, masks, caches=(k, k, s, s))


def test_scales_that_are_broadcast():
    # one scale for all pages and heads, read alone
    rng = np.random.default_rng(98)
    q, cache, ctx, cu, masks = attention_inputs(rng, [2], [200], 4, 2, 64, 32, 16, torch.bfloat16)
    one = torch.tensor([2.0 ** -6, 2.0 ** -8], dtype=torch.bfloat16, device=DEV)
    shape = cache.k_scale.shape[1:]
    k, v, _, _ = cache.device()
    cache.k_scale = cache.v_scale = np.broadcast_to(np.array([2.0 ** -6, 2.0 ** -8]), (1, *shape))
    check_attention(q, cache, ctx, cu, masks, caches=(k, v, one.expand(shape), one.expand(shape)))


def test_two_captured_steps_replayed_in_turn():
    s, t = make_step(99), make_step(100)
    want_s, want_t = make_step(99), make_step(100)
    graphs, got = [], []
    for x in (s, t):
        before = [y.clone() for y in state(x)]
        step(x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(step(x))
        for y, z in zip(state(x), before):
            y.copy_(z)
        graphs.append(graph)
    for _ in range(3):
        for graph, out, x, y in zip(graphs, got, (s, t), (want_s, want_t)):
            graph.replay()
            want = step(y)
            torch.cuda.synchronize()
            assert equal(out, want) and equal(state(x), state(y))


@pytest.mark.parametrize("rows_,max_pages", [(1, 5000), (3, 700), (9000, 1), (257, 129)])
def test_plans_of_long_rows_and_many(rows_, max_pages):
    rng = np.random.default_rng(101)
    B, page = 2, 16
    pages = B * max_pages + 3 * rows_ + 40
    table = rng.permutation(pages)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
    ctx = rng.integers(0, max_pages * page + 1, B).astype(np.int32)
    for limit in (None, pages // 2, 17):
        check_plan(table, ctx, rng.integers(-1, B, rows_), rng.integers(0, 40, rows_), pages, page,
                   limit)


def test_commit_of_everything_and_nothing_at_once():
    # whole chains accepted in place (nothing moves), others not at all, blocks at their borders
    rng = np.random.default_rng(102)
    counts, ctx = [16, 16, 32, 1], np.array([16, 15, 0, 31], np.int32)
    cu = ref.prefix(counts)
    cache = Cache8(rng, [int(c) + n for c, n in zip(ctx, counts)], 32, 16, 3, 48, layers=2)
    for r, n in enumerate(counts):
        cache.fill(rng, r, 0, int(ctx[r]) + n, -20, -4)
    path = np.tile(np.arange(32, dtype=np.int32), (4, 1))
    accepted = np.array([16, 0, 32, 1], np.int32)
    caches = cache.device()
    ple.ple_tree_commit_fp8(dev(np.zeros(65, np.int64)), dev(path), dev(accepted), dev(cu), None,
                            dev(ctx), dev(cache.table), *caches)
    after = read(caches)
    for i, (c, s) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        want, scales = ref8.commit(path, accepted, cu, ctx, cache.table, c, s)
        assert same(after[i], want) and same(after[i + 2], scales)
        assert same(want, c)      # rows stay under the scales that they had
