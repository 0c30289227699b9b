"""Attention in float16 where the weights of a softmax span more binades than
float16 has, against 64 bits: a weight that is tiny beside the largest counts
for what it is, on every kernel.

Scores are set exactly: one element of the queries and keys, whose product is
the score's exponent of 2, and a scale of ln 2.  The bound is that of the
other attention tests, with the weights' rounding as it is in float16: a weight
is exact to 2^-11 of itself or to 2^-28 of the largest weight of its 128 slots
(float16 ends at 2^-25, and the largest weight of 128 slots that go together
enters as at least 2^3), so 128 slots lose at most 2^-21 of their largest
weight times their largest value.
"""

import numpy as np
import pytest
import torch

import layer_gram_embedding_gb300 as ple
import tree_reference as ref
from test_tree_ops import Cache, attention_inputs, check_attention, dev, host

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

U = 2.0 ** -11
LN2 = float(np.log(2.0))
SIGNS = (1.0, 0.5, -0.5, 0.75)   # the queries' element, by row
# nodes, query heads, key heads, page size: rows that share tiles in turn, rows of both groups,
# and the kernel for every page size
ROWS = [(1, 4, 1, 16), (40, 8, 2, 64), (3, 4, 1, 20)]


def softmax(levels, values, sign):
    """(out, weight, lost, lse, reach) over keys of exponents sign * levels, in 64 bits."""
    s = sign * levels
    p = np.exp2(s - s.max())
    total = p.sum()
    p = p / total
    pad = -len(p) % 128
    top = np.pad(p, (0, pad)).reshape(-1, 128).max(1)
    size = np.pad(np.abs(values), ((0, pad), (0, 0))).reshape(len(top), 128, -1).max(1)
    return (p @ values, p @ np.abs(values), 2.0 ** -21 * (top @ size),
            LN2 * (s.max() + np.log2(total)), LN2 * np.abs(s).max())


def check(levels, values):
    """levels [n], values [n, D] as float16 holds them, seen by every node of one request."""
    assert np.array_equal(levels, levels.astype(np.float16))
    values = values.astype(np.float16).astype(np.float64)
    want = {x: softmax(levels.astype(np.float64), values, x) for x in SIGNS}
    for rows in ROWS:
        check_rows(levels, values, want, *rows)


def check_rows(levels, values, expected, nodes, Hq, Hk, page):
    n, D = values.shape
    cache = Cache(np.random.default_rng(n), [n + nodes], page, Hk, D, torch.float16)
    i = np.arange(n)
    p, s = dev(cache.table[0][i // page].astype(np.int64)), dev(i % page)
    keys = np.zeros((n, Hk, D), np.float16)
    keys[:, :, 0] = levels[:, None]
    cache.k[p, :, s] = dev(keys)
    cache.v[p, :, s] = dev(np.repeat(values[:, None].astype(np.float16), Hk, 1))
    q = np.zeros((nodes, Hq, D), np.float16)
    sign = np.resize(SIGNS, nodes * Hq).reshape(nodes, Hq)
    q[:, :, 0] = sign
    out, lse = ple.ple_tree_attention(
        dev(q), cache.k, cache.v, dev(cache.table), dev(np.array([n], np.int32)),
        dev(np.array([0, nodes], np.int32)), torch.zeros((nodes, 1), dtype=torch.int64,
                                                         device="cuda"),
        scale=LN2, return_lse=True)
    out, lse = host(out), host(lse)
    for x in SIGNS:
        want, weight, lost, want_lse, reach = expected[x]
        # the exponent's own roundings, of the scale, the product and the shift; and those of
        # the running sums, a step for 128 slots
        score = 2.0 ** -24 * (4 * reach + n / 128) + 2.0 ** -20
        bound = U * (1 + 2.0 ** -8) * np.abs(want) + (U + 2 * score) * weight + lost + 2.0 ** -25
        err = np.abs(out[sign == x] - want)
        assert np.all(err <= bound), f"{x}, page {page}: {np.max(err / bound)} times the bound"
        assert np.all(np.abs(lse[sign == x] - want_lse)
                      <= score + 2.0 ** -20 + 2.0 ** -22 * abs(want_lse))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [20000, 131000])
@pytest.mark.parametrize("below", [25.1875, 33.0, 45.0])
@pytest.mark.parametrize("where", ["first", "last"])
def test_one_key_far_above_many(D, n, below, where):
    # an attention sink: one key whose value is nothing above a flat context
    rng = np.random.default_rng(3)
    levels = np.full(n, -below / 2)
    values = rng.uniform(50, 100, (n, D))
    sink = 0 if where == "first" else n - 1
    levels[sink] = below / 2
    values[sink // 128 * 128:sink // 128 * 128 + 128] = 0
    check(levels, values)


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kind", ["down", "up", "jumps", "slopes"])
def test_tiles_at_levels_of_their_own(D, kind):
    # each column's values lie in one tile's slots, largest where the weights are least
    rng = np.random.default_rng(4)
    tiles = 45
    level = {"down": -2.5 * np.arange(tiles), "up": 2.5 * np.arange(tiles) - 100,
             "jumps": rng.integers(-50, 51, tiles), "slopes": 10 * rng.integers(-3, 4, tiles)}[kind]
    n = 128 * tiles - 37
    levels = np.repeat(level, 128)[:n].astype(np.float64)
    if kind == "slopes":  # within a tile too
        levels = levels + rng.integers(-160, 161, n) / 16
    values = np.zeros((n, D))
    columns = rng.integers(0, tiles, D)
    for c, tile in enumerate(columns):
        at = slice(128 * tile, min(128 * tile + 128, n))
        values[at, c] = rng.uniform(0.5, 1.0, at.stop - at.start) * rng.choice([1.0, 30000.0])
    check(levels, values)


@pytest.mark.parametrize("D", [64, 128, 96, 160])
def test_large_scores_in_half(D):
    # a softmax of few weights, whose running maximum moves often and far
    rng = np.random.default_rng(9)
    q, cache, ctx, cu, masks = attention_inputs(rng, [12], [700], 8, 2, D, 16, torch.float16,
                                                size=20.0)
    for i in range(712):
        p, s = cache.where(0, i)
        cache.k[int(p), :, s] *= 0.02 * (1 + i // 30)
    check_attention(q, cache, ctx, cu, masks)
    # and falling ones, the last above all others
    for i in range(712):
        p, s = cache.where(0, i)
        cache.k[int(p), :, s] *= 30.0 / (1 + i // 30) ** 2 if i < 705 else 1.0
    check_attention(q, cache, ctx, cu, masks)


def test_hidden_slots_do_not_set_the_level():
    # drafted nodes whose masks hide the tile's largest scores, and rows that see one node alone
    rng = np.random.default_rng(5)
    q, cache, ctx, cu, masks = attention_inputs(rng, [300], [200], 4, 2, 128, 16, torch.float16)
    masks = np.zeros_like(masks)
    for j in range(300):
        masks[j, j // 64] = np.uint64(1 << (j % 64)).astype(np.int64)
    for j in range(0, 300, 2):
        p, s = cache.where(0, 200 + j)
        cache.k[int(p), :, s] *= 20.0
    check_attention(q, cache, ctx, cu, masks)
    ctx0 = np.array([0], np.int32)
    positions, _ = ref.tree_index(np.full(300, -1, np.int32), cu, ctx0, 5)
    assert positions.max() == 0
    check_attention(q, cache, ctx0, cu, masks)
