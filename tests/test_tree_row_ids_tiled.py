"""Row ids of drafted trees in batches that take the tiled kernel (more than
small_batch_max_rows() row ids a call): branches, both id types, both output
types, prepared constants, every ngram size, divisors off the 32-bit path, many
requests in a tile; and the limits of what a malformed layout reads."""

import numpy as np
import pytest
import torch

import layer_gram_embedding_gb300 as ple
import tree_reference as ref
from test_tree_ops import BOUNDARY, dev, row_id_inputs

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def expected(ids, parent, cu, ctx, M, vocab, off, hpn):
    """tree_reference.tree_row_ids, whole tokens at a time."""
    V = ref.tree_windows(ids, parent, cu, ctx, BOUNDARY)
    L, N = M.shape
    out = np.zeros((L, len(ids), vocab.shape[1]), np.int64)
    with np.errstate(over="ignore", divide="ignore"):
        for l in range(L):
            mix = V[:, 0] * M[l, 0]
            for s in range(1, N):
                mix = mix ^ (V[:, s] * M[l, s])
                for h in range((s - 1) * hpn, s * hpn):
                    v = vocab[l, h]
                    out[l, :, h] = (np.remainder(mix, v) if v else 0) + off[l, h]
    return out


def test_expected_is_the_references():
    rng = np.random.default_rng(1)
    counts = [5, 0, 9]
    parent, cu = ref.trees(rng, counts), ref.prefix(counts)
    ids, ctx, M, vocab, off = row_id_inputs(rng, counts, 4, 2, 3, np.int64, 2 ** 62)
    vocab[0, 1], vocab[1, 2] = -vocab[0, 1], 0
    a = (ids, parent, cu, ctx, M, vocab, off, 2)
    assert np.array_equal(expected(*a), ref.tree_row_ids(*a, BOUNDARY))


def counts_of(rng, T, most):
    out = []
    while sum(out) < T:
        out.append(int(min(rng.integers(0, most + 1), T - sum(out))))
    return out


# N, heads of an order, layers, nodes of a request at most
SHAPES = [(2, 1, 3, 60), (2, 3, 7, 9), (2, 255, 1, 40), (3, 2, 9, 1), (3, 4, 20, 33), (4, 4, 11, 63),
          (4, 7, 5, 200), (5, 8, 48, 63), (5, 64, 1, 5), (6, 5, 4, 70), (8, 3, 6, 2), (8, 32, 2, 50),
          (9, 4, 3, 130), (16, 1, 8, 17), (16, 16, 2, 64), (3, 1, 40, 2), (17 - 1, 3, 4, 1)]


@pytest.mark.parametrize("dtype", [np.int32, np.int64])
@pytest.mark.parametrize("N,hpn,L,most", SHAPES)
def test_tiled_kernel(N, hpn, L, most, dtype):
    rng = np.random.default_rng(N * 1000 + hpn)
    H = (N - 1) * hpn
    T = ple.small_batch_max_rows() // (H * L) + 45  # a ragged last tile
    assert T * H * L > ple.small_batch_max_rows()
    counts = counts_of(rng, T, most)
    parent, cu = ref.trees(rng, counts), ref.prefix(counts)
    ids, ctx, M, vocab, off = row_id_inputs(rng, counts, N, hpn, L, dtype)
    want = expected(ids, parent, cu, ctx, M, vocab, off, hpn)
    args = [dev(x) for x in (ids, parent, cu, ctx, M, vocab, off)]
    heads = ple.ple_prepare_heads(args[5], args[6])
    for prepared in (None, heads):
        got = ple.ple_tree_row_ids(*args, N, hpn, BOUNDARY, heads=prepared)
        assert np.array_equal(got.cpu().numpy(), want)
        low = ple.ple_tree_row_ids(*args, N, hpn, BOUNDARY, heads=prepared, out_dtype=torch.int32)
        assert np.array_equal(low.cpu().numpy(), want.astype(np.int32))


@pytest.mark.parametrize("N,hpn", [(3, 8), (4, 7), (5, 8), (7, 2)])
def test_tiled_kernel_large_vocab_sizes_and_signs(N, hpn):
    # heads on the 32-bit path among heads off it: large, negative and zero divisors
    rng = np.random.default_rng(N)
    H, L = (N - 1) * hpn, 6
    T = ple.small_batch_max_rows() // (H * L) + 33
    counts = counts_of(rng, T, 40)
    parent, cu = ref.trees(rng, counts), ref.prefix(counts)
    ids, ctx, M, vocab, off = row_id_inputs(rng, counts, N, hpn, L, np.int64, 2 ** 62)
    vocab[:, 1::3] = rng.integers(1, 2 ** 29 + 1, vocab[:, 1::3].shape)
    vocab[0, ::4] *= -1
    vocab[1, 3], vocab[2, 0], vocab[2, 1] = 0, 2 ** 29, 2 ** 29 + 1
    vocab[3, 0], vocab[3, 1], vocab[3, 2] = 1, -1, 2 ** 63 - 1
    want = expected(ids, parent, cu, ctx, M, vocab, off, hpn)
    args = [dev(x) for x in (ids, parent, cu, ctx, M, vocab, off)]
    for prepared in (None, ple.ple_prepare_heads(args[5], args[6])):
        got = ple.ple_tree_row_ids(*args, N, hpn, BOUNDARY, heads=prepared)
        assert np.array_equal(got.cpu().numpy(), want)


def test_parents_that_are_no_earlier_node_count_as_none():
    rng = np.random.default_rng(7)
    counts = counts_of(rng, 5000, 50)
    cu = ref.prefix(counts)
    parent = rng.integers(-3, 60, 5000).astype(np.int32)
    parent[rng.random(5000) < 0.1] = 2 ** 31 - 1
    parent[rng.random(5000) < 0.1] = -2 ** 31
    ids, ctx, M, vocab, off = row_id_inputs(rng, counts, 5, 8, 1, np.int64)
    want = expected(ids, parent, cu, ctx, M, vocab, off, 8)
    got = ple.ple_tree_row_ids(*[dev(x) for x in (ids, parent, cu, ctx, M, vocab, off)], 5, 8,
                               BOUNDARY)
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("T,L", [(200, 2), (6000, 3)])  # the small kernel and the tiled one
def test_malformed_layout_reads_nothing_outside(T, L):
    # rows of a malformed layout are unspecified, but they are made of the arguments alone: what lies
    # around ids, parents, contexts and prefix sums in memory changes none of them
    rng = np.random.default_rng(11)
    N, hpn, B, guard = 5, 8, 90, 4096
    _, _, M, vocab, off = (dev(x) for x in row_id_inputs(rng, [1], N, hpn, L, np.int64))
    ids = rng.integers(0, 1000, T)
    ctx = rng.integers(0, 1000, (B, N - 1))

    def inside(a, fill):
        a = np.asarray(a)
        whole = torch.full((a.size + 2 * guard,), int(fill), dtype=dev(a).dtype, device="cuda")
        view = whole[guard:guard + a.size]
        view.copy_(dev(a.reshape(-1)))
        return view.view(a.shape)

    layouts = [rng.integers(-2 ** 31, 2 ** 31, B + 1), rng.integers(-50, T + 50, B + 1),
               np.sort(rng.integers(-50, T + 50, B + 1)), np.full(B + 1, T), np.zeros(B + 1),
               np.sort(rng.integers(0, T + 1, B + 1))[::-1]]
    for k, cu in enumerate(layouts):
        parent = rng.integers(-2 ** 31, 2 ** 31, T) if k % 2 else rng.integers(-3, T, T)
        got = []
        for fill in (0, 1, -1, 12345):
            a = [inside(x.astype(kind), fill) for x, kind in
                 ((ids, np.int64), (parent, np.int32), (np.asarray(cu), np.int32),
                  (ctx, np.int64))]
            got.append(ple.ple_tree_row_ids(*a, M, vocab, off, N, hpn, BOUNDARY))
        for x in got[1:]:
            assert torch.equal(x, got[0]), k
