"""Faults that the operators on caches in 8 bits and on pages once had, on the GPU: a
test for each, against plain 64-bit host implementations (cache_reference.py)."""

import numpy as np
import pytest
import torch

import cache_reference as ref8
import layer_gram_embedding_gb300 as ple
import tree_reference as ref
from test_cache_ops import (FP8, KERNELS, U, Cache8, attention_inputs, check_append,
                            check_attention, dev, host, read, rows, same)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("D,nodes,longest,dtype", [
    # rows a key head on the average: up to 32, 64, 128 and more
    (64, (5, 7), 60, torch.bfloat16), (64, (9, 15), 60, torch.float16),
    (64, (17, 31), 60, torch.bfloat16), (64, (33, 60), 60, torch.float16),
    (32, (5, 40), 60, torch.float16), (48, (5, 7), 60, torch.bfloat16),
    (64, (5, 7), 300, torch.float16), (64, (17, 60), 300, torch.bfloat16),
    (128, (5, 7), 60, torch.float16), (128, (17, 31), 60, torch.bfloat16),
    (256, (9, 15), 60, torch.bfloat16),
])
def test_nan_in_one_segment_of_many(D, nodes, longest, dtype):
    # Units of one tile (and some of a few), several in a row in every block: what was found in a
    # unit's drafted values stays known until its rows go out.  A NaN changes nothing but its own
    # column of the rows that see it.
    rng = np.random.default_rng(D + nodes[1] + longest)
    B, Hk, group = 160, 8, 4
    counts = [int(x) for x in rng.integers(nodes[0], nodes[1] + 1, B)]
    ctx = [int(x) for x in rng.integers(0, longest, B)]
    q, cache, ctx, cu, masks = attention_inputs(rng, counts, ctx, group * Hk, Hk, D, 32, 16, dtype)
    out, lse = check_attention(q, cache, ctx, cu, masks)
    want = out.clone()
    for r in range(0, B, 3):
        node, h, d = (int(rng.integers(n)) for n in (counts[r], Hk, D))
        p, s = cache.where(r, int(ctx[r]) + node)
        cache.v[0, p, h, s, d] = rng.choice([0x7F, 0xFF])
        sees = dev(masks[cu[r]:cu[r + 1], 0] >> node & 1 != 0)
        want[cu[r]:cu[r + 1], h * group:(h + 1) * group, d][sees] = float("nan")
    assert bool(want.isnan().any())
    got, got_lse = ple.ple_tree_attention_fp8(q, *cache.device(), dev(cache.table), dev(ctx),
                                              dev(cu), dev(masks), return_lse=True)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0)) and torch.equal(got_lse, lse)


def test_commit_under_any_two_scales():
    # Eight older tokens under one scale, eight moved behind them from a block under another: of
    # all pairs of significands, all bytes of the ones or of the others are rounded under the
    # larger scale.  Products of an element and a scale are exact in 64 bits, and so is a quotient
    # of them on the border of two elements; every other one is 2^-13 of itself away from it.
    requests, heads, D = 128, 128, 256
    pages = 2 * requests
    table = np.arange(pages, dtype=np.int32).reshape(requests, 2)
    ctx, cu = np.full(requests, 8, np.int32), ref.prefix([16] * requests)
    path = np.tile(np.arange(8, 16, dtype=np.int32), (requests, 1))
    one, two = np.broadcast_arrays(128.0 + np.arange(requests)[:, None], 128.0 + np.arange(heads))
    for exponent in (-13, -100, -139, 119):
        scales = [np.stack([one, two * step], 1) * 2.0 ** exponent for step in (1, 2)]
        caches = [dev(np.arange(256, dtype=np.uint8)).expand(pages, heads, 16, D).contiguous()
                  .view(FP8) for _ in range(2)]
        caches += [dev(s.reshape(pages, heads, 1)).to(torch.bfloat16) for s in scales]
        scales = [s.double().cpu().numpy().reshape(requests, 2, heads) for s in caches[2:]]
        ple.ple_tree_commit_fp8(dev(np.zeros(16 * requests, np.int64)), dev(path),
                                dev(np.full(requests, 8, np.int32)), dev(cu), None, dev(ctx),
                                dev(table), *caches)
        for c, now, had in zip(caches[:2], caches[2:], scales):
            got = c.view(torch.uint8).view(requests, 2, heads, 16, D)[:, 0].cpu().numpy()
            top = had.max(1)
            assert np.array_equal(now.double().cpu().numpy().reshape(had.shape)[:, 0], top)
            for part in (0, 1):
                with np.errstate(invalid="ignore"):     # NaN elements
                    want = ref8.encode(ref8.VALUES * had[:, part, :, None] / top[..., None])
                nan = np.isnan(ref8.VALUES)
                x = got[:, :, 8 * part:8 * part + 8]
                assert np.all(x[..., nan] & 0x7F == 0x7F)
                differ = x[..., ~nan] != want[:, :, None, ~nan]
                assert not differ.any(), (exponent, part, differ.mean())


@pytest.mark.parametrize("counts,Hq", KERNELS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("below", [40, 44, 48])
def test_values_far_below_a_key_that_takes_nearly_all(counts, Hq, dtype, below):
    # One key's weight is 2^below times any other's, its values are zeros and so are those of the
    # 128 slots around it: all that comes out has weights of 2^-below, which enter the product to
    # 2^-11 of themselves.  Enough requests that a block has most of a unit's tiles.
    rng = np.random.default_rng(41)
    B, c, scale = 120, 600, float(np.log(2.0))
    q, cache, ctx, cu, masks = attention_inputs(rng, counts * B, [c] * B, Hq, 2, 64, 16, 16, dtype)
    q[:] = 0
    q[..., 0] = 1
    for r in range(B):
        p, s = cache.where(r, np.arange(c + counts[0]))
        cache.k[0, p, :, s, 0] = 0
        cache.k[0, p[0], :, s[0], 0] = ref8.encode(float(below))
        cache.k_scale[0, p] = 1
        cache.v[0, p[:128], :, s[:128]] = 0
        cache.v_scale[0, p] = 2.0 ** (below - 8)
    out, lse = ple.ple_tree_attention_fp8(q, *cache.device(), dev(cache.table), dev(ctx), dev(cu),
                                          dev(masks), scale=scale, return_lse=True)
    k, v = (ref8.dequantise(x[0], y[0]) for x, y in ((cache.k, cache.k_scale),
                                                     (cache.v, cache.v_scale)))
    want, want_lse, weight = ref8.attention(host(q), k, v, cache.v_scale[0], cache.table, ctx, cu,
                                            masks, scale)[:3]
    # the output's rounding, the weights', that of exponents up to `below` (scores are exact but
    # for scale * log2(e)) and of one sum for each 16 slots
    bound = U[dtype] * (1 + 2.0 ** -8) * np.abs(want) + \
        (2.0 ** -11 + 2.0 ** -22 * below + 2.0 ** -20 + 2.0 ** -23 * c / 16) * weight
    assert np.all(np.abs(host(out) - want) <= bound)
    assert np.all(np.abs(host(lse) - want_lse) <= 2.0 ** -20 * np.abs(want_lse) + 2.0 ** -20)


@pytest.mark.parametrize("block,D,into", [(128, 128, 127), (128, 256, 65), (64, 256, 33)])
def test_older_tokens_grow_with_their_block(block, D, into):
    # angles in parts: every lane sees the scale that the block had, not the one that it gets, and
    # rounds its part of the older tokens anew
    rng = np.random.default_rng(43)
    B, Hk = 40, 8
    ctx, cu = np.full(B, into, np.int32), ref.prefix([2] * B)
    cache = Cache8(rng, [into + 2] * B, block, block, Hk, D)
    for r in range(B):
        cache.fill(rng, r, 0, into, -16, -12)
    k, v = (rows(rng, (2 * B, Hk, D), torch.bfloat16) for _ in range(2))
    positions = dev(np.zeros(2 * B, np.int32))     # turned by nothing
    args = (dev(cache.table), dev(ctx), dev(cu))
    first = None
    for _ in range(5):
        caches = cache.device()
        before = read(caches)
        ple.ple_qk_norm_rope_fp8(k[:, :0], k, v, positions, ple.ple_prepare_rope(D), None, None,
                                 *caches, *args)
        after = read(caches)
        for i, x in enumerate((k, v)):
            check_append((after[i][0], after[i + 2][0]), (before[i][0], before[i + 2][0]), host(x),
                         np.zeros(x.shape), cache.table, ctx, cu, exact=True)
        first = first or after
        assert all(same(x, y) for x, y in zip(first, after))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale", [1.5, 1.0, 255 * 2.0 ** -100])
def test_appended_zeros_keep_their_signs(dtype, scale):
    # under a scale that the block has, a power of two or not, and beside what is not finite
    cache = Cache8(np.random.default_rng(44), [12], 16, 16, 2, 64)
    cache.fill(np.random.default_rng(45), 0, 0, 4)
    p, _ = cache.where(0, 0)
    cache.k_scale[0, p] = cache.v_scale[0, p] = scale
    x = torch.zeros((8, 2, 64), dtype=dtype, device=DEV)
    x[:, :, ::3] = -0.0
    x[:, :, 1::3] = scale * 4.5
    x[5, 1, 7] = float("inf")
    ctx, cu = np.array([4], np.int32), np.array([0, 8], np.int32)
    caches = cache.device()
    before = read(caches)
    ple.ple_qk_norm_rope_fp8(x[:, :0], x, x, None, None, None, None, *caches, dev(cache.table),
                             dev(ctx), dev(cu))
    after = read(caches)
    for i in (0, 1):
        check_append((after[i][0], after[i + 2][0]), (before[i][0], before[i + 2][0]), host(x),
                     np.zeros(x.shape), cache.table, ctx, cu, exact=True)


def test_a_plan_does_not_keep_its_workspace():
    pages = 2 ** 20
    table, zero = dev(np.zeros((1, 1), np.int32)), dev(np.zeros(1, np.int32))
    got = ple.ple_plan_pages(table, zero, zero, dev(np.ones(1, np.int32)), pages, 16)
    assert got[3].tolist() == [0, 1, 0]
    assert all(t.untyped_storage().nbytes() < 2 ** 16 for t in got)
