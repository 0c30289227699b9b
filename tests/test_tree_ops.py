"""The tree-verification operators on the GPU against plain 64-bit host
implementations (tree_reference.py).

Integer outputs and moved rows are compared bit for bit.  Floating outputs are
held to bounds that follow from the arithmetic: results are computed in 32
bits and rounded once to the element type (unit roundoff u: half the spacing at
1, 2^-8 for bfloat16 and 2^-11 for float16), and the attention's weights are
rounded to it before they meet the values.
"""

import numpy as np
import pytest
import torch

import layer_gram_embedding_gb300 as ple
import tree_reference as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = torch.device("cuda:0")
U = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16)}
BOUNDARY = 7


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def rows(rng, shape, dtype, size=1.0):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * size).to(dtype).to(DEV)


def host(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------- tree index


@pytest.mark.parametrize("counts,words", [
    ([1], 1), ([4], 1), ([0, 3, 0, 64, 1], 1), ([65, 127, 128, 0], 2), ([130, 192], 3),
    ([256, 1], 4), ([300], 5), ([383], 6), ([448], 7), ([512, 511], 8), ([3] * 700, 1),
])
def test_tree_index(counts, words):
    rng = np.random.default_rng(sum(counts) + words)
    for reach in (1, 6):  # chains (the deepest trees) and branches
        parent = ref.trees(rng, counts, roots=0.0 if reach == 1 else 0.1, reach=reach)
        cu = ref.prefix(counts)
        ctx = rng.integers(0, 200000, len(counts)).astype(np.int32)
        positions, masks = ref.tree_index(parent, cu, ctx, words)
        got = ple.ple_build_tree_index(dev(parent), dev(cu), dev(ctx), words)
        assert np.array_equal(got[0].cpu().numpy(), positions)
        assert np.array_equal(got[1].cpu().numpy(), masks)


def test_tree_index_parents_that_are_no_earlier_node_count_as_none():
    parent = np.array([-1, 0, 2, 7, -5, 3, 2 ** 31 - 1, -2 ** 31], dtype=np.int32)
    cu, ctx = np.array([0, 8], dtype=np.int32), np.array([10], dtype=np.int32)
    positions, masks = ref.tree_index(parent, cu, ctx, 1)
    got = ple.ple_build_tree_index(dev(parent), dev(cu), dev(ctx), 1)
    assert np.array_equal(got[0].cpu().numpy(), positions)
    assert np.array_equal(got[1].cpu().numpy(), masks)


def test_tree_index_nodes_without_a_bit():
    # 70 nodes in one word: the first 64 as ever, the others without bits
    parent = np.arange(-1, 69, dtype=np.int32)
    cu, ctx = np.array([0, 70], dtype=np.int32), np.array([5], dtype=np.int32)
    positions, masks = ple.ple_build_tree_index(dev(parent), dev(cu), dev(ctx), 1)
    assert positions.tolist() == [5 + j for j in range(64)] + [5] * 6
    assert [m & (2 ** 64 - 1) for m in masks[:, 0].tolist()] == \
        [2 ** (j + 1) - 1 for j in range(64)] + [0] * 6


# -------------------------------------------------------------- tree row ids


def row_id_inputs(rng, counts, N, hpn, L, dtype, vocab_hi=2 ** 20):
    H = (N - 1) * hpn
    T = sum(counts)
    ids = rng.integers(0, 1000, T).astype(dtype)
    ids[rng.random(T) < 0.15] = BOUNDARY
    ctx = rng.integers(0, 1000, (len(counts), N - 1)).astype(dtype)
    ctx[rng.random(ctx.shape) < 0.15] = BOUNDARY
    M = rng.integers(-2 ** 63, 2 ** 63, (L, N), dtype=np.int64)
    vocab = rng.integers(1, vocab_hi, (L, H), dtype=np.int64)
    off = rng.integers(0, 2 ** 40, (L, H), dtype=np.int64)
    return ids, ctx, M, vocab, off


@pytest.mark.parametrize("dtype", [np.int32, np.int64])
@pytest.mark.parametrize("counts,N,hpn,L", [
    ([1], 3, 2, 1), ([9], 3, 2, 1), ([3, 0, 17, 1, 40], 5, 8, 3), ([33] * 5, 4, 4, 2),
    ([20, 5], 2, 1, 2), ([12, 30], 16, 3, 1), ([7] * 40, 3, 4, 5), ([64, 31, 1], 4, 7, 2),
    ([50], 2, 255, 1), ([40, 40], 5, 64, 2),
])
def test_tree_row_ids(counts, N, hpn, L, dtype):
    rng = np.random.default_rng(N * 1000 + hpn)
    parent, cu = ref.trees(rng, counts), ref.prefix(counts)
    ids, ctx, M, vocab, off = row_id_inputs(rng, counts, N, hpn, L, dtype)
    expect = ref.tree_row_ids(ids, parent, cu, ctx, M, vocab, off, hpn, BOUNDARY)
    args = [dev(x) for x in (ids, parent, cu, ctx, M, vocab, off)]
    got = ple.ple_tree_row_ids(*args, N, hpn, BOUNDARY)
    assert np.array_equal(got.cpu().numpy(), expect)
    low = ple.ple_tree_row_ids(*args, N, hpn, BOUNDARY, out_dtype=torch.int32)
    assert np.array_equal(low.cpu().numpy(), expect.astype(np.int32))
    heads = ple.ple_prepare_heads(args[5], args[6])
    got = ple.ple_tree_row_ids(*args, N, hpn, BOUNDARY, heads=heads)
    assert np.array_equal(got.cpu().numpy(), expect)


def test_tree_row_ids_large_vocab_sizes_and_signs():
    # divisors off the 32-bit path, negative and zero ones among them
    rng = np.random.default_rng(5)
    counts = [31, 2]
    parent, cu = ref.trees(rng, counts), ref.prefix(counts)
    ids, ctx, M, vocab, off = row_id_inputs(rng, counts, 4, 4, 3, np.int64, 2 ** 62)
    vocab[0, ::3] *= -1
    vocab[1, 5] = 0
    expect = ref.tree_row_ids(ids, parent, cu, ctx, M, vocab, off, 4, BOUNDARY)
    got = ple.ple_tree_row_ids(*[dev(x) for x in (ids, parent, cu, ctx, M, vocab, off)], 4, 4,
                               BOUNDARY)
    assert np.array_equal(got.cpu().numpy(), expect)


@pytest.mark.parametrize("N,hpn,L", [(3, 2, 1), (5, 8, 48), (4, 4, 8), (4, 7, 3)])
@pytest.mark.parametrize("counts", [[1, 5, 0, 700], [2000, 33, 4096, 1]])
def test_tree_row_ids_of_chains_are_a_prefills(counts, N, hpn, L):
    rng = np.random.default_rng(sum(counts) + L)
    cu = ref.prefix(counts)
    parent = np.concatenate([np.arange(-1, n - 1) for n in counts]).astype(np.int32)
    ids, ctx, M, vocab, off = (dev(x) for x in row_id_inputs(rng, counts, N, hpn, L, np.int64))
    got = ple.ple_tree_row_ids(ids, dev(parent), dev(cu), ctx, M, vocab, off, N, hpn, BOUNDARY)
    want = ple.ple_row_ids(ids, None, None, ctx, M, vocab, off, N, hpn, BOUNDARY,
                           cu_seqlens=dev(cu))
    assert torch.equal(got, want)


def test_tree_row_ids_malformed_layout_stays_in_bounds():
    # any parents and cu_seqlens: rows are unspecified, every access is clamped
    rng = np.random.default_rng(11)
    counts = [100, 57, 43]
    ids, ctx, M, vocab, off = (dev(x) for x in row_id_inputs(rng, counts, 5, 8, 2, np.int64))
    for _ in range(4):
        parent = rng.integers(-2 ** 31, 2 ** 31, 200).astype(np.int32)
        cu = rng.integers(-2 ** 31, 2 ** 31, 4).astype(np.int32)
        ple.ple_tree_row_ids(ids, dev(parent), dev(cu), ctx, M, vocab, off, 5, 8, BOUNDARY)
    torch.cuda.synchronize()


# ------------------------------------------------------------ rotation, norms


@pytest.mark.parametrize("R", [2, 4, 64, 128, 256])
@pytest.mark.parametrize("scaling,factor", [("plain", 1.0), ("linear", 4.0), ("base", 8.0),
                                            ("parts", 4.0)])
def test_prepare_rope(R, scaling, factor):
    w = ref.inverse_frequencies(R, 10000.0, scaling, factor, 4096.0)
    got = ple.ple_prepare_rope(R, 10000.0, scaling, factor, 4096.0)
    turns = got.cpu().numpy().astype(np.float64) / 2.0 ** 64
    # pow and three roundings in 64 bits, and the truncation to 2^-64 turns
    assert np.all(np.abs(turns - w / (2 * np.pi)) <= 2.0 ** -49 * turns + 2.0 ** -64)


class Cache:
    """A paged cache in drawn order, NaN wherever nothing lives, laid out in memory as `order` says."""

    def __init__(self, rng, lengths, page, heads, dim, dtype, order="phsd", layers=None, spare=2):
        per = [max(1, -(-n // page)) for n in lengths]
        pages = sum(per) + spare
        at = rng.permutation(pages)
        table, k = np.full((len(lengths), max(per) if per else 1), 2 ** 30, dtype=np.int32), 0
        for r, n in enumerate(per):
            table[r, :n] = at[k:k + n]
            k += n
        sizes = dict(l=layers or 1, p=pages, h=heads, s=page, d=dim)
        order = ("l" if layers else "") + order
        shape = [sizes[c] for c in order]
        logical = ("l" if layers else "") + "phsd"

        def make():
            t = torch.full(shape, float("nan"), dtype=dtype, device=DEV)
            return t.permute([order.index(c) for c in logical])

        self.k, self.v, self.table, self.page = make(), make(), table, page

    def where(self, r, i):
        return self.table[r, i // self.page], i % self.page

    def fill(self, rng, r, first, last, size=1.0):
        """Live keys and values for cached tokens first .. last - 1 of request r."""
        i = np.arange(first, last)
        if len(i) == 0:
            return
        p, s = dev(self.table[r][i // self.page].astype(np.int64)), dev(i % self.page)
        for c in (self.k, self.v):
            # [.., n, heads, dim] in the order that the two indices give
            shape = (len(i), c.shape[-3], c.shape[-1])
            if c.dim() == 5:
                shape = (len(i), c.shape[0]) + shape[1:]
                c[:, p, :, s] = rows(rng, shape, c.dtype, size)
            else:
                c[p, :, s] = rows(rng, shape, c.dtype, size)


NORM_CASES = [
    # counts, ctx, Hq, Hk, D, R, interleaved, page
    ([1], [900], 32, 8, 128, 128, False, 64),
    ([3, 0, 33, 1], [0, 5, 120000, 63], 8, 2, 64, 64, False, 16),
    ([3, 0, 33, 1], [0, 5, 120000, 63], 8, 2, 64, 32, True, 16),
    ([17, 2], [100, 7], 5, 5, 96, 48, False, 48),
    ([17, 2], [100, 7], 4, 1, 80, 40, False, 1),
    ([17, 2], [100, 7], 4, 1, 80, 40, True, 7),
    ([5], [1000], 3, 1, 256, 256, False, 128),
    ([5], [1000], 3, 1, 256, 12, False, 32),
    ([9, 9], [31, 32], 2, 2, 8, 6, False, 16),
    ([9, 9], [31, 32], 2, 2, 8, 0, False, 16),
    ([40], [11], 1, 3, 16, 2, True, 5),
    ([3000, 2500], [1, 2], 4, 2, 128, 64, False, 64),   # four tokens a block
    ([1300] * 4, [0, 9, 1, 2], 2, 1, 64, 64, True, 16),
]


def check_rows(got, want, size, u, what):
    """want in 64 bits; size: |y_a| + |y_b| of each element's pair."""
    # rounding to the element type; 32-bit norm, products and angle (2e-7 radians); subnormals of float16
    bound = u * np.abs(want) * (1 + 2.0 ** -8) + 2.0 ** -20 * size + 2.0 ** -25
    err = np.abs(host(got) - want)
    assert np.all(err <= bound), f"{what}: {np.max(err - bound)} over the bound"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", NORM_CASES)
@pytest.mark.parametrize("form", ["fused", "plain", "odd strides"])
def test_qk_norm_rope(case, dtype, form):
    counts, ctx, Hq, Hk, D, R, interleaved, page = case
    rng = np.random.default_rng(sum(counts) + D + R)
    T, B = sum(counts), len(counts)
    qkv = rows(rng, (T, Hq + 2 * Hk, D), dtype, 3.0)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    order = "phsd"
    if form == "plain":
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    if form == "odd strides":  # head-major rows, slots outside heads in the cache
        q = q.transpose(0, 1).contiguous().transpose(0, 1)
        order = "pshd"
    qw, kw = rows(rng, (D,), dtype), rows(rng, (D,), dtype)
    ctx = np.array(ctx, dtype=np.int32)
    lengths = [int(c) + n for c, n in zip(ctx, counts)]
    cu = ref.prefix(counts)
    positions = (np.repeat(ctx, counts) + rng.integers(0, 40, T)).astype(np.int32)
    rope = ple.ple_prepare_rope(R, 1e6, "parts", 4.0, 4096.0) if R else None
    w = ref.inverse_frequencies(R, 1e6, "parts", 4.0, 4096.0)
    # 120000-token contexts need only the pages behind them
    cache = Cache(rng, lengths, page, Hk, D, dtype, order)
    before = cache.k.clone(), cache.v.clone()
    got = ple.ple_qk_norm_rope(q, k, v, dev(positions) if R else None, rope, qw, kw,
                               k_cache=cache.k, v_cache=cache.v, page_table=dev(cache.table),
                               ctx_lens=dev(ctx), cu_seqlens=dev(cu), eps=1e-5,
                               interleaved=interleaved, rope_scale=1.25)
    want, size = ref.norm_rope(host(q), host(qw), positions, w, 1e-5, interleaved, 1.25)
    check_rows(got, want, size, U[dtype], "q")
    want, size = ref.norm_rope(host(k), host(kw), positions, w, 1e-5, interleaved, 1.25)
    page_at, slot_at = [], []
    for r in range(B):
        for j in range(counts[r]):
            p, s = cache.where(r, int(ctx[r]) + j)
            page_at.append(int(p))
            slot_at.append(int(s))
    check_rows(cache.k[page_at, :, slot_at], want, size, U[dtype], "k")
    assert torch.equal(cache.v[page_at, :, slot_at], v)
    # nothing else was written
    for now, old in zip((cache.k, cache.v), before):
        now = now.clone()
        now[page_at, :, slot_at] = float("nan")
        assert torch.equal(now.isnan(), old.isnan())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rotation_without_cache_or_norm_in_place(dtype):
    rng = np.random.default_rng(2)
    q, k = rows(rng, (70, 6, 64), dtype), rows(rng, (70, 3, 64), dtype)
    positions = rng.integers(0, 2 ** 20, 70).astype(np.int32)
    w = ref.inverse_frequencies(64, 10000.0)
    want = [ref.norm_rope(host(x), None, positions, w, 0.0, False, 1.0) for x in (q, k)]
    rope = ple.ple_prepare_rope(64)
    a, b = ple.ple_qk_norm_rope(q, k, None, dev(positions), rope, q_out=q, k_out=k)
    assert a is q and b is k
    check_rows(q, *want[0], U[dtype], "q")
    check_rows(k, *want[1], U[dtype], "k")


@pytest.mark.parametrize("D,Hq,Hk", [(64, 3, 2), (128, 1, 4), (96, 2, 1)])
@pytest.mark.parametrize("which", ["q", "k"])
def test_norm_of_queries_or_keys_alone(which, D, Hq, Hk):
    rng = np.random.default_rng(D)
    q, k = rows(rng, (9, Hq, D), torch.bfloat16, 2.0), rows(rng, (9, Hk, D), torch.bfloat16, 2.0)
    w = rows(rng, (D,), torch.bfloat16)
    positions = rng.integers(0, 5000, 9).astype(np.int32)
    freq = ref.inverse_frequencies(D, 10000.0)
    a, b = ple.ple_qk_norm_rope(q, k, None, dev(positions), ple.ple_prepare_rope(D),
                                w if which == "q" else None, w if which == "k" else None)
    for got, x, name in ((a, q, "q"), (b, k, "k")):
        want, size = ref.norm_rope(host(x), host(w) if name == which else None, positions, freq,
                                   1e-6, False, 1.0)
        check_rows(got, want, size, U[torch.bfloat16], name)


def test_norm_of_extreme_rows():
    # zeros stay zeros (eps), an infinity makes its row NaN and no other's
    q = torch.ones((4, 2, 64), dtype=torch.bfloat16, device=DEV)
    q[0] = 0
    q[1, 0, 3] = float("inf")
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    out, _ = ple.ple_qk_norm_rope(q, q.clone(), None, None, None, w, w)
    assert torch.all(out[0] == 0)
    assert out[1, 0].isnan().any() and not out[1, 1].isnan().any()
    assert torch.all(out[2:] == 1)


def test_append_outside_the_page_table_is_dropped():
    rng = np.random.default_rng(3)
    q, k, v = (rows(rng, (40, 1, 64), torch.bfloat16) for _ in range(3))
    cache = Cache(rng, [32], 16, 1, 64, torch.bfloat16)
    cache.table[0, 1] = -1
    ple.ple_qk_norm_rope(q, k, v, None, None, k_cache=cache.k, v_cache=cache.v,
                         page_table=dev(cache.table), ctx_lens=dev(np.array([4], np.int32)),
                         cu_seqlens=dev(np.array([0, 40], np.int32)))
    written = ~cache.v.isnan().all(-1)
    assert int(written.sum()) == 12  # slots 4 .. 15 of the only page
    assert torch.equal(cache.v[int(cache.table[0, 0]), 0, 4:], v[:12, 0])


def test_padding_tokens_append_nothing():
    # seven tokens of a fixed shape, four of them nodes; the last request has room behind its own
    rng = np.random.default_rng(19)
    q, k, v = (rows(rng, (7, 1, 64), torch.float16) for _ in range(3))
    cache = Cache(rng, [16, 32], 16, 1, 64, torch.float16)
    ple.ple_qk_norm_rope(q, k, v, None, None, k_cache=cache.k, v_cache=cache.v,
                         page_table=dev(cache.table), ctx_lens=dev(np.array([4, 9], np.int32)),
                         cu_seqlens=dev(np.array([0, 3, 4], np.int32)))
    assert int((~cache.v.isnan().all(-1)).sum()) == 4
    assert int((~cache.k.isnan().all(-1)).sum()) == 4
    assert torch.equal(cache.v[int(cache.table[0, 0]), 0, 4:7], v[:3, 0])
    assert torch.equal(cache.v[int(cache.table[1, 0]), 0, 9], v[3, 0])


# ------------------------------------------------------------------ attention


def host_attention(q, cache, ctx, cu, masks, scale):
    return ref.attention(host(q), host(cache.k), host(cache.v), cache.table, ctx, cu, masks, scale)


def check_attention(q, cache, ctx, cu, masks, scale=None, what="", workspace=None, sanitize=False,
                    reference=host_attention):
    """The call against the reference.  Errors: the output's rounding u |o|; the weights' rounding and the 32-bit scores'
    error (D + 8 roundings of the products' sum, and a few of the exponent) on sum p |v|."""
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    u = U[q.dtype]
    out, lse = ple.ple_tree_attention(q, cache.k, cache.v, dev(cache.table), dev(ctx), dev(cu),
                                      dev(masks), scale=scale, return_lse=True,
                                      workspace=workspace)
    want, want_lse, weight, reach = reference(q, cache, ctx, cu, masks, scale)
    D = q.shape[-1]
    score = 2.0 ** -24 * (D + 8) * reach + 2.0 ** -20
    bound = u * (1 + 2.0 ** -8) * np.abs(want) + (u + 2 * score[..., None]) * weight + 2.0 ** -25
    got = host(out)
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fine), what
    if sanitize:
        assert np.array_equal(np.isnan(got), np.isnan(want)), what
    with np.errstate(invalid="ignore"):
        err = np.abs(got - want)
    assert np.all(err[fine] <= bound[fine]), f"{what}: {np.max((err - bound)[fine])} over the bound"
    got = host(lse)
    fine = np.isfinite(want_lse)
    assert np.array_equal(got[~fine & ~np.isnan(want_lse)], want_lse[~fine & ~np.isnan(want_lse)])
    err = np.abs(got[fine] - want_lse[fine])
    assert np.all(err <= (score + 2.0 ** -20 + 2.0 ** -22 * np.abs(want_lse))[fine]), what
    return out, lse


def attention_inputs(rng, counts, ctx, Hq, Hk, D, page, dtype, order="phsd", size=1.0):
    ctx = np.array(ctx, dtype=np.int32)
    cu = ref.prefix(counts)
    lengths = [int(c) + n for c, n in zip(ctx, counts)]
    cache = Cache(rng, lengths, page, Hk, D, dtype, order)
    for r, n in enumerate(lengths):
        cache.fill(rng, r, 0, n)
    words = max(1, -(-max(counts) // 64))
    _, masks = ref.tree_index(ref.trees(rng, counts), cu, ctx, words)
    q = rows(rng, (sum(counts), Hq, D), dtype, size)
    return q, cache, ctx, cu, masks


ATTENTION_CASES = [
    # counts, ctx, Hq, Hk, D, page, order
    ([1], [0], 1, 1, 64, 16, "phsd"),
    ([1], [700], 32, 8, 128, 64, "phsd"),
    ([1, 1, 1], [127, 128, 129], 4, 1, 128, 64, "phsd"),
    ([5, 0, 33, 1], [0, 9, 511, 64], 8, 2, 64, 16, "phsd"),
    ([64, 3], [300, 1], 16, 2, 128, 32, "phsd"),
    ([17], [1000], 10, 2, 128, 128, "pshd"),
    ([70, 129], [50, 257], 8, 4, 128, 64, "phsd"),
    ([200], [3], 4, 4, 64, 256, "phsd"),
    ([33], [95], 5, 1, 64, 8, "phsd"),
    ([9, 2], [40, 77], 6, 2, 96, 16, "phsd"),
    ([9, 2], [40, 77], 9, 1, 256, 48, "pshd"),
    ([9, 2], [40, 77], 3, 3, 8, 16, "phsd"),
    ([9, 2], [40, 77], 8, 2, 128, 7, "phsd"),
    ([4] * 37, list(range(0, 370, 10)), 4, 2, 64, 16, "phsd"),
    ([2], [5000], 4, 1, 128, 64, "phsd"),
    ([512], [130], 2, 1, 64, 64, "phsd"),
    # more tiles than the device has SMs: shares of many tiles and requests
    ([2] * 40, [100 + 19 * i for i in range(40)], 16, 8, 128, 16, "phsd"),
    ([3, 0, 1, 30] * 12, [37 * i for i in range(48)], 16, 4, 64, 64, "phsd"),
    ([40, 64, 33], [2500, 900, 3000], 32, 4, 64, 32, "phsd"),
    ([18], [9001], 32, 4, 128, 64, "phsd"),
    ([1, 1], [20000, 11], 4, 2, 128, 128, "phsd"),
    # other widths, and page sizes of the other kernel: split slots, more heads than a block takes
    ([1, 3], [5000, 0], 20, 2, 256, 16, "phsd"),
    ([1], [3001], 3, 1, 128, 20, "pshd"),
    ([1, 40], [3001, 129], 6, 2, 128, 24, "pshd"),
    ([33, 2], [500, 1000], 8, 2, 120, 40, "phsd"),
    ([9, 9], [1000, 20], 4, 1, 40, 384, "phsd"),
    ([60, 70], [90, 300], 8, 8, 80, 16, "phsd"),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", ATTENTION_CASES)
def test_tree_attention(case, dtype):
    counts, ctx, Hq, Hk, D, page, order = case
    rng = np.random.default_rng(sum(counts) + D + page)
    q, cache, ctx, cu, masks = attention_inputs(rng, counts, ctx, Hq, Hk, D, page, dtype, order)
    check_attention(q, cache, ctx, cu, masks, what=str(case))


@pytest.mark.parametrize("D", [64, 128, 96, 160])
def test_attention_is_the_same_every_time(D):
    rng = np.random.default_rng(8)
    q, cache, ctx, cu, masks = attention_inputs(rng, [20, 3, 64], [900, 2000, 31], 8, 2, D, 16,
                                                torch.bfloat16)
    first = check_attention(q, cache, ctx, cu, masks)
    for _ in range(3):
        again = check_attention(q, cache, ctx, cu, masks)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def dense_attention(q, cache, ctx, cu, masks, scale):
    """The reference in 64 bits on the device, a request at a time: for sizes the host is too slow for."""
    T, Hq, D = q.shape
    Hk = cache.k.shape[1]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=DEV)
    weight, lse = out.clone(), torch.full((T, Hq), -np.inf, dtype=torch.float64, device=DEV)
    reach = torch.zeros((T, Hq), dtype=torch.float64, device=DEV)
    for r in range(len(cu) - 1):
        n, first = int(cu[r + 1] - cu[r]), int(cu[r])
        if n == 0:
            continue
        length = int(ctx[r]) + n
        at = np.arange(length)
        p, s = dev(cache.table[r][at // cache.page].astype(np.int64)), dev(at % cache.page)
        k, v = (c[p, :, s].double().transpose(0, 1) for c in (cache.k, cache.v))  # [Hk, length, D]
        bits = (dev(masks[first:first + n])[:, :, None] >> torch.arange(64, device=DEV)) & 1
        sees = torch.ones((n, length), dtype=torch.bool, device=DEV)
        sees[:, int(ctx[r]):] = bits.reshape(n, -1)[:, :n].bool()
        x = q[first:first + n].double().reshape(n, Hk, Hq // Hk, D).permute(1, 2, 0, 3)
        score = (x @ k[:, None].transpose(2, 3)) * scale
        score = score.masked_fill(~sees, -np.inf)
        p = torch.softmax(score, -1)

        def back(t):
            return t.permute(2, 0, 1, 3).reshape(n, Hq, -1)

        out[first:first + n] = back(p @ v[:, None])
        weight[first:first + n] = back(p @ v[:, None].abs())
        lse[first:first + n] = back(torch.logsumexp(score, -1, keepdim=True))[..., 0]
        reach[first:first + n] = back((x.abs() @ k[:, None].abs().transpose(2, 3))
                                      .amax(-1, keepdim=True))[..., 0] * abs(scale)
    return tuple(t.cpu().numpy() for t in (out, lse, weight, reach))


@pytest.mark.parametrize("seed", range(24))
def test_attention_random_batches(seed):
    rng = np.random.default_rng(1000 + seed)
    D = int(rng.choice([64, 128, 128, 96, 72, 32]))
    page = int(rng.choice([8, 16, 32, 64, 128, 256, 384, 24, 80]))
    dtype = [torch.bfloat16, torch.float16][seed % 2]
    Hk = int(rng.choice([1, 2, 4, 8]))
    Hq = Hk * int(rng.choice([1, 2, 3, 4, 7, 8, 16]))
    B = int(rng.integers(1, 40))
    most = int(rng.choice([1, 3, 17, 64, 90, 200]))
    counts = [int(rng.integers(0 if B > 1 else 1, most + 1)) for _ in range(B)]
    counts[0] = max(counts[0], 1)
    room = max(1, int(3e6 / max(sum(counts) * Hq, 1) * B))  # scores of the reference
    ctx = [int(rng.integers(0, min(room, 9000) + 1)) for _ in range(B)]
    q, cache, ctx, cu, masks = attention_inputs(rng, counts, ctx, Hq, Hk, D, page, dtype,
                                                str(rng.choice(["phsd", "pshd"])))
    first = check_attention(q, cache, ctx, cu, masks, what=str((counts, ctx, Hq, Hk, D, page)),
                            reference=dense_attention)
    for _ in range(20):  # nothing depends on timing
        again = ple.ple_tree_attention(q, cache.k, cache.v, dev(cache.table), dev(ctx), dev(cu),
                                       dev(masks), return_lse=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# Heads in two parts: one tile, cut units, more than a unit's 128 rows, a part of one
# piece, tiles of several pages; then pages of the other kernel.
WIDE_CASES = [
    ([1], [0], 1, 1, 256, 64, "phsd"),
    ([1], [127], 8, 1, 256, 64, "pshd"),
    ([1, 1, 1], [20000, 0, 300], 8, 2, 256, 64, "phsd"),
    ([40, 64, 33], [900, 2500, 1], 8, 2, 256, 16, "phsd"),
    ([33, 0, 200], [3001, 5, 130], 16, 4, 192, 32, "pshd"),
    ([18], [9001], 16, 2, 136, 128, "phsd"),
    ([65], [4000], 6, 2, 248, 8, "phsd"),
    ([9, 3], [700, 64], 20, 2, 256, 12, "phsd"),
    ([5], [2000], 4, 4, 192, 20, "pshd"),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", WIDE_CASES)
def test_attention_of_wide_heads(case, dtype):
    counts, ctx, Hq, Hk, D, page, order = case
    rng = np.random.default_rng(sum(counts) + D + page)
    q, cache, ctx, cu, masks = attention_inputs(rng, counts, ctx, Hq, Hk, D, page, dtype, order)
    check_attention(q, cache, ctx, cu, masks, what=str(case))


@pytest.mark.parametrize("seed", range(12))
def test_attention_random_batches_of_wide_heads(seed):
    rng = np.random.default_rng(2000 + seed)
    D = int(rng.choice([256, 256, 192, 136, 160, 200]))
    page = int(rng.choice([8, 16, 32, 64, 128, 24]))
    dtype = [torch.bfloat16, torch.float16][seed % 2]
    Hk = int(rng.choice([1, 2, 4, 8]))
    Hq = Hk * int(rng.choice([1, 2, 3, 4, 8]))
    B = int(rng.integers(1, 40))
    most = int(rng.choice([1, 3, 17, 64, 90]))
    counts = [int(rng.integers(0 if B > 1 else 1, most + 1)) for _ in range(B)]
    counts[0] = max(counts[0], 1)
    room = max(1, int(3e6 / max(sum(counts) * Hq, 1) * B))  # scores of the reference
    ctx = [int(rng.integers(0, min(room, 9000) + 1)) for _ in range(B)]
    q, cache, ctx, cu, masks = attention_inputs(rng, counts, ctx, Hq, Hk, D, page, dtype,
                                                str(rng.choice(["phsd", "pshd"])))
    first = check_attention(q, cache, ctx, cu, masks, what=str((counts, ctx, Hq, Hk, D, page)),
                            reference=dense_attention)
    for _ in range(20):  # nothing depends on timing
        again = ple.ple_tree_attention(q, cache.k, cache.v, dev(cache.table), dev(ctx), dev(cu),
                                       dev(masks), return_lse=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_attention_many_short_units_again_and_again():
    # blocks with several units of a few tiles each, 300 times
    rng = np.random.default_rng(16)
    q, cache, ctx, cu, masks = attention_inputs(rng, [2] * 40, [100 + 19 * i for i in range(40)],
                                                16, 8, 128, 16, torch.bfloat16)
    args = (q, cache.k, cache.v, dev(cache.table), dev(ctx), dev(cu), dev(masks))
    first = ple.ple_tree_attention(*args)
    for _ in range(300):
        assert torch.equal(ple.ple_tree_attention(*args), first)


@pytest.mark.parametrize("D", [64, 128, 96, 160])
def test_attention_large_scores(D):
    # a softmax of few weights, whose running maximum moves often and far
    rng = np.random.default_rng(9)
    q, cache, ctx, cu, masks = attention_inputs(rng, [12], [700], 8, 2, D, 16, torch.bfloat16,
                                                size=20.0)
    # rising keys: every tile holds a new maximum
    for i in range(712):
        p, s = cache.where(0, i)
        cache.k[int(p), :, s] *= 0.02 * (1 + i // 30)
    check_attention(q, cache, ctx, cu, masks)


@pytest.mark.parametrize("D", [64, 128, 96, 160])
def test_nodes_that_see_nothing(D):
    rng = np.random.default_rng(4)
    q, cache, ctx, cu, masks = attention_inputs(rng, [6, 5, 70], [0, 40, 0], 4, 2, D, 16,
                                                torch.float16)
    masks = masks.copy()
    masks[[0, 3, 7, 12, 60]] = 0  # rows 0, 3 and 12, 60 have neither context nor nodes
    out, lse = check_attention(q, cache, ctx, cu, masks)
    for t in (0, 3, 12, 60):
        assert torch.all(out[t] == 0) and torch.all(lse[t] == float("-inf"))


@pytest.mark.parametrize("D", [64, 128, 96, 160])
def test_nothing_unseen_has_an_effect(D):
    # nodes no row sees hold NaN; a node that some rows see holds infinities, which reach those rows alone
    rng = np.random.default_rng(6)
    q, cache, ctx, cu, masks = attention_inputs(rng, [40, 9], [100, 13], 8, 2, D, 16,
                                                torch.bfloat16)
    masks = masks.copy()
    for hidden in (11, 25):
        masks[:40, 0] &= ~np.int64(1 << hidden)
        p, s = cache.where(0, 100 + hidden)
        cache.k[int(p), :, s] = float("nan")
        cache.v[int(p), :, s] = float("inf")
    plain, plain_lse = check_attention(q, cache, ctx, cu, masks)
    for bad in (float("inf"), float("nan")):
        p, s = cache.where(0, 100 + 7)
        old = cache.v[int(p), :, s].clone()
        cache.v[int(p), :, s, 5] = bad
        out, lse = check_attention(q, cache, ctx, cu, masks, sanitize=True)
        sees = dev(((masks[:, 0] >> 7) & 1).astype(bool) & (np.arange(49) < 40))
        assert not out[sees][:, :, 5].isfinite().any()
        out[sees] = plain[sees]
        assert torch.equal(out, plain) and torch.equal(lse, plain_lse)
        cache.v[int(p), :, s] = old


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
@pytest.mark.parametrize("D", [64, 96, 160])
def test_attention_scales(D, scale):
    rng = np.random.default_rng(19)
    q, cache, ctx, cu, masks = attention_inputs(rng, [5, 70], [200, 31], 4, 2, D, 16,
                                                torch.bfloat16)
    check_attention(q, cache, ctx, cu, masks, scale=scale)


def test_attention_masks_bits_past_the_nodes_are_ignored():
    rng = np.random.default_rng(12)
    q, cache, ctx, cu, masks = attention_inputs(rng, [5, 3], [30, 2], 4, 2, 128, 16,
                                                torch.bfloat16)
    plain = check_attention(q, cache, ctx, cu, masks)
    more = masks.copy()
    more[:5] |= ~np.int64(31)
    more[5:] |= ~np.int64(7)
    out = ple.ple_tree_attention(q, cache.k, cache.v, dev(cache.table), dev(ctx), dev(cu),
                                 dev(more), return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(out, plain))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_of_long_drafts(D, dtype):
    # masks of any bits in eight words, drafted tiles at odd places in them, and values that
    # are not finite in a few nodes' first, last and middle elements
    rng = np.random.default_rng(17)
    q, cache, ctx, cu, masks = attention_inputs(rng, [512, 300, 65], [77, 1000, 191], 2, 1, D, 16,
                                                dtype)
    masks = rng.integers(-2 ** 63, 2 ** 63, masks.shape, dtype=np.int64)
    masks[rng.random(masks.shape) < 0.3] = 0
    check_attention(q, cache, ctx, cu, masks)
    for r, node, element, bad in [(0, 511, D - 1, np.inf), (0, 200, 3, -np.inf),
                                  (0, 63, 0, np.nan), (1, 299, D // 2, np.inf), (1, 0, 7, np.nan),
                                  (2, 64, D - 2, -np.inf)]:
        p, s = cache.where(r, int(ctx[r]) + node)
        cache.v[int(p), :, s, element] = float(bad)
    check_attention(q, cache, ctx, cu, masks, sanitize=True)


@pytest.mark.parametrize("D", [64, 128, 96, 160])
def test_attention_pages_outside_the_cache_read_as_zeros(D):
    rng = np.random.default_rng(13)
    q, cache, ctx, cu, masks = attention_inputs(rng, [4], [60], 4, 2, D, 16, torch.bfloat16)
    lost = int(cache.table[0, 1])
    out = []
    for page in (-1, 2 ** 31 - 1, None):
        if page is None:  # the same page, holding zeros
            cache.table[0, 1] = lost
            cache.k[lost] = 0
            cache.v[lost] = 0
        else:
            cache.table[0, 1] = page
        out.append(ple.ple_tree_attention(q, cache.k, cache.v, dev(cache.table), dev(ctx), dev(cu),
                                          dev(masks)))
    assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[2])


def test_attention_on_another_stream_keeps_its_workspace():
    # the call's own workspace is not handed out again while the other stream still needs it
    rng = np.random.default_rng(18)
    args = attention_inputs(rng, [20], [3001], 8, 2, 64, 16, torch.bfloat16)
    q, cache, ctx, cu, masks = args
    call = (q, cache.k, cache.v, dev(cache.table), dev(ctx), dev(cu), dev(masks))
    out, want = torch.empty_like(q), ple.ple_tree_attention(*call)
    size = ple.ple_tree_attention_workspace(20, 8, 2, 64).shape[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    block = torch.empty(size, dtype=torch.uint8, device=DEV)
    taken = block.data_ptr()
    del block
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # some tens of ms
    ple.ple_tree_attention(*call, out=out, stream=side)
    again = torch.empty(size, dtype=torch.uint8, device=DEV)
    assert not side.query() and again.data_ptr() != taken
    side.synchronize()
    assert torch.equal(out, want)


def test_attention_strided_queries_and_preallocated_outputs():
    rng = np.random.default_rng(14)
    q, cache, ctx, cu, masks = attention_inputs(rng, [9, 30], [77, 500], 8, 4, 64, 32,
                                                torch.float16)
    wide = torch.zeros((39, 12, 72), dtype=torch.float16, device=DEV)
    wide[:, 2:10, :64] = q
    view = wide[:, 2:10, :64]
    plain = check_attention(q, cache, ctx, cu, masks)
    out = torch.empty_like(q)
    lse = torch.empty((39, 8), dtype=torch.float32, device=DEV)
    workspace = ple.ple_tree_attention_workspace(39, 8, 4, 64)
    workspace.fill_(255)  # need not be cleared
    got = ple.ple_tree_attention(view, cache.k, cache.v, dev(cache.table), dev(ctx), dev(cu),
                                 dev(masks), out=out, lse=lse, workspace=workspace)
    assert got is out
    assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])


@pytest.mark.parametrize("D", [128, 80])
def test_attention_offsets_past_32_bits(D):
    # a cache of more than 2^32 elements, the request's pages at its far end
    page, heads = 64, 2
    pages = 2 ** 32 // (page * heads * D) + 40
    k = torch.zeros((pages, heads, page, D), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    rng = np.random.default_rng(15)
    k[-4:] = rows(rng, (4, heads, page, D), torch.bfloat16)
    v[-4:] = rows(rng, (4, heads, page, D), torch.bfloat16)
    small = Cache(rng, [200], page, heads, D, torch.bfloat16, spare=0)
    small.k, small.v = k[-4:], v[-4:]
    small.table = np.array([[3, 0, 2, 1]], dtype=np.int32)
    q = rows(rng, (3, 4, D), torch.bfloat16)
    ctx, cu = np.array([197], np.int32), np.array([0, 3], np.int32)
    masks = np.array([[1], [3], [5]], dtype=np.int64)
    want = check_attention(q, small, ctx, cu, masks)
    out = ple.ple_tree_attention(q, k, v, dev(small.table + (pages - 4)), dev(ctx), dev(cu),
                                 dev(masks), return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(out, want))


# --------------------------------------------------------------------- commit


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("counts,ctx,P,layers,Hk,D,page,order", [
    ([9], [700], 3, 1, 8, 128, 64, "phsd"),
    ([9, 0, 33, 1], [0, 5, 63, 16], 9, 3, 2, 64, 16, "phsd"),
    ([200, 130], [1, 30], 150, 2, 3, 8, 5, "pshd"),
    ([12] * 20, list(range(20)), 6, 4, 1, 256, 48, "phsd"),
])
def test_tree_commit(counts, ctx, P, layers, Hk, D, page, order, dtype):
    rng = np.random.default_rng(sum(counts) + P)
    ctx, cu = np.array(ctx, np.int32), ref.prefix(counts)
    cache = Cache(rng, [int(c) + n for c, n in zip(ctx, counts)], page, Hk, D, dtype, order,
                  layers)
    for r, n in enumerate(counts):
        cache.fill(rng, r, 0, int(ctx[r]) + n)
    path = np.zeros((len(counts), P), np.int32)
    accepted = np.zeros(len(counts), np.int32)
    for r, n in enumerate(counts):
        accepted[r] = rng.integers(0, min(n, P) + 1)
        path[r, :accepted[r]] = np.sort(rng.choice(n, accepted[r], replace=False))
    ids = rng.integers(0, 2 ** 40, sum(counts))
    context = rng.integers(0, 2 ** 40, (len(counts), 4))
    want = [ref.commit(path, accepted, cu, ctx, cache.table, host(c)) for c in (cache.k, cache.v)]
    for kind in (np.int64, np.int32):
        again = Cache.__new__(Cache)
        again.k, again.v = cache.k.clone(), cache.v.clone()
        got = ple.ple_tree_commit(dev(ids.astype(kind)), dev(path), dev(accepted), dev(cu),
                                  dev(context.astype(kind)), dev(ctx), dev(cache.table), again.k,
                                  again.v)
        for c, w in zip((again.k, again.v), want):
            assert np.array_equal(host(c), w, equal_nan=True)
        assert np.array_equal(got[0].cpu().numpy(),
                              ref.next_context(ids.astype(kind), path, accepted, cu,
                                               context.astype(kind)))
        assert np.array_equal(got[1].cpu().numpy(), ctx + accepted)


def test_commit_of_one_layer_without_a_context():
    rng = np.random.default_rng(21)
    cache = Cache(rng, [30], 16, 2, 64, torch.bfloat16)
    cache.fill(rng, 0, 0, 30)
    old = cache.k.clone()
    ids = torch.zeros(10, dtype=torch.int64, device=DEV)
    path, accepted = dev(np.array([[0, 4, 9]], np.int32)), dev(np.array([3], np.int32))
    nxt, lens = ple.ple_tree_commit(ids, path, accepted, dev(np.array([0, 10], np.int32)), None,
                                    dev(np.array([20], np.int32)), dev(cache.table), cache.k,
                                    cache.v)
    assert nxt is None and lens.tolist() == [23]
    for j, node in enumerate((0, 4, 9)):
        a, b = cache.where(0, 20 + node), cache.where(0, 20 + j)
        assert torch.equal(cache.k[int(b[0]), :, int(b[1])], old[int(a[0]), :, int(a[1])])


def test_commit_refuses_to_leave_the_request():
    # path entries past the nodes, or before their own place, leave their slots; accepted is clamped
    rng = np.random.default_rng(22)
    cache = Cache(rng, [26], 16, 1, 64, torch.bfloat16)
    cache.fill(rng, 0, 0, 26)
    old = cache.k.clone()
    path, accepted = np.array([[0, 0, 6, -3, 2 ** 31 - 1, 5]], np.int32), np.array([99], np.int32)
    _, lens = ple.ple_tree_commit(torch.zeros(6, dtype=torch.int32, device=DEV), dev(path),
                                  dev(accepted), dev(np.array([0, 6], np.int32)), None,
                                  dev(np.array([20], np.int32)), dev(cache.table), cache.k,
                                  cache.v)
    assert lens.tolist() == [26]
    assert torch.equal(cache.k.nan_to_num(), old.nan_to_num())


# ------------------------------------------------------- streams, graphs, sizes


def test_empty_batches():
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    cu, ctx = dev(np.array([0], np.int32)), z
    p, m = ple.ple_build_tree_index(z, cu, ctx, 1)
    assert p.shape == (0,) and m.shape == (0, 1)
    cache = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16, device=DEV)
    table = torch.zeros((0, 1), dtype=torch.int32, device=DEV)
    q = torch.zeros((0, 1, 64), dtype=torch.bfloat16, device=DEV)
    assert ple.ple_tree_attention(q, cache, cache, table, ctx, cu, m).shape == (0, 1, 64)
    assert ple.ple_qk_norm_rope(q, q, q, None, None, k_cache=cache, v_cache=cache,
                                page_table=table, ctx_lens=ctx,
                                cu_seqlens=cu).shape == (0, 1, 64)


def step_inputs(rng, D=128):
    counts, ctx = [7, 1, 20], np.array([50, 300, 9], np.int32)
    cu = ref.prefix(counts)
    cache = Cache(rng, [int(c) + n for c, n in zip(ctx, counts)], 16, 2, D, torch.bfloat16)
    for r in range(3):
        cache.fill(rng, r, 0, int(ctx[r]))
    return counts, ctx, cu, cache


def step(s):
    """One layer of a verification step, as a user runs it."""
    positions, masks = ple.ple_build_tree_index(s["parent"], s["cu"], s["ctx"], 1)
    row_ids = ple.ple_tree_row_ids(s["ids"], s["parent"], s["cu"], s["context"], s["M"],
                                   s["vocab"], s["off"], 3, 2, BOUNDARY)
    q = ple.ple_qk_norm_rope(s["q"], s["k"], s["v"], positions, s["rope"], s["qw"], s["kw"],
                             k_cache=s["kc"], v_cache=s["vc"], page_table=s["table"],
                             ctx_lens=s["ctx"], cu_seqlens=s["cu"])
    out, lse = ple.ple_tree_attention(q, s["kc"], s["vc"], s["table"], s["ctx"], s["cu"], masks,
                                      return_lse=True)
    nxt, lens = ple.ple_tree_commit(s["ids"], s["path"], s["accepted"], s["cu"], s["context"],
                                    s["ctx"], s["table"], s["kc"], s["vc"])
    return [row_ids, out, lse, nxt, lens, s["kc"], s["vc"]]


def make_step(seed):
    rng = np.random.default_rng(seed)
    counts, ctx, cu, cache = step_inputs(rng)
    T = sum(counts)
    ids, context, M, vocab, off = (dev(x) for x in row_id_inputs(rng, counts, 3, 2, 1, np.int64))
    qkv = rows(rng, (T, 8, 128), torch.bfloat16)
    w = rows(rng, (128,), torch.bfloat16)
    return dict(parent=dev(ref.trees(rng, counts)), cu=dev(cu), ctx=dev(ctx), ids=ids,
                context=context, M=M, vocab=vocab, off=off, q=qkv[:, :4], k=qkv[:, 4:6],
                v=qkv[:, 6:], rope=ple.ple_prepare_rope(128), qw=w, kw=w, kc=cache.k, vc=cache.v,
                table=dev(cache.table), path=dev(np.array([[0, 2, 5]] * 3, np.int32)),
                accepted=dev(np.array([3, 1, 2], np.int32)))


def same(a, b):
    return all(torch.equal(x.nan_to_num() if x.is_floating_point() else x,
                           y.nan_to_num() if y.is_floating_point() else y) for x, y in zip(a, b))


def test_a_step_on_another_stream_and_in_a_graph():
    # the commit moves rows within the nodes' slots, which the next pass appends anew: a pass may be repeated
    s, t = make_step(31), make_step(31)
    torch.cuda.synchronize()
    want = [x.clone() for x in step(s)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(t)
        got = step(t)
    side.synchronize()
    assert same(got, want)
    u = make_step(32)
    other = [x.clone() for x in step(make_step(32))]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(t)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert same(captured, want)
    for key, value in u.items():  # fresh inputs in the captured buffers
        t[key].copy_(value)
    graph.replay()
    torch.cuda.synchronize()
    assert same(captured, other)


def test_programmatic_launch_does_not_change_the_step():
    want = [x.clone() for x in step(make_step(33))]
    before = ple.set_programmatic_launch(False)
    try:
        got = step(make_step(33))
        torch.cuda.synchronize()
        assert same(got, want)
    finally:
        ple.set_programmatic_launch(before)


# ------------------------------------------------------------------- refusals


def test_refusals():
    s = make_step(40)
    T, bf = s["q"].shape[0], torch.bfloat16
    mask = torch.zeros((T, 1), dtype=torch.int64, device=DEV)

    def attention(**kw):
        a = dict(q=s["q"], k_cache=s["kc"], v_cache=s["vc"], page_table=s["table"],
                 ctx_lens=s["ctx"], cu_seqlens=s["cu"], tree_mask=mask)
        return ple.ple_tree_attention(**dict(a, **kw))

    def norm(**kw):
        a = dict(q=s["q"], k=s["k"], v=s["v"], positions=s["parent"], rope=s["rope"],
                 k_cache=s["kc"], v_cache=s["vc"], page_table=s["table"], ctx_lens=s["ctx"],
                 cu_seqlens=s["cu"])
        return ple.ple_qk_norm_rope(**dict(a, **kw))

    def commit(**kw):
        a = dict(input_ids=s["ids"], path=s["path"], accepted=s["accepted"], cu_seqlens=s["cu"],
                 ngram_context=s["context"], ctx_lens=s["ctx"], page_table=s["table"],
                 k_cache=s["kc"], v_cache=s["vc"])
        return ple.ple_tree_commit(**dict(a, **kw))

    def index(**kw):
        a = dict(parent=s["parent"], cu_seqlens=s["cu"], ctx_lens=s["ctx"], mask_words=1)
        return ple.ple_build_tree_index(**dict(a, **kw))

    def row_ids(**kw):
        a = dict(input_ids=s["ids"], parent=s["parent"], cu_seqlens=s["cu"],
                 ngram_context=s["context"], layer_multipliers=s["M"], vocab_sizes=s["vocab"],
                 offsets=s["off"], ngram_size=3, heads_per_ngram=2, boundary_id=BOUNDARY)
        return ple.ple_tree_row_ids(**dict(a, **kw))

    half = s["kc"].half()
    for error, call in [
        (TypeError, lambda: attention(q=s["q"].float())),
        (TypeError, lambda: attention(k_cache=half, v_cache=half)),
        (ValueError, lambda: attention(q=s["q"][0])),
        (ValueError, lambda: attention(q=s["q"][:, :3])),          # heads not divided
        (ValueError, lambda: attention(q=s["q"][..., :64])),
        (ValueError, lambda: attention(v_cache=s["vc"][:-1])),
        (ValueError, lambda: attention(cu_seqlens=s["cu"][:-1])),
        (ValueError, lambda: attention(tree_mask=mask[:-1])),
        (TypeError, lambda: attention(tree_mask=mask.int())),
        (ValueError, lambda: attention(page_table=s["table"][:2])),
        (ValueError, lambda: attention(page_table=s["table"].cpu())),
        (ValueError, lambda: attention(lse=torch.zeros(T, device=DEV))),
        (ValueError, lambda: attention(out=torch.zeros((T, 4, 64), dtype=bf, device=DEV))),
        (ple.PleError, lambda: attention(workspace=torch.zeros(0, dtype=torch.uint8, device=DEV))),
        (ple.PleError, lambda: attention(scale=float("nan"))),
        (ple.PleError, lambda: attention(tree_mask=torch.zeros((T, 9), dtype=torch.int64,
                                                               device=DEV))),
        (TypeError, lambda: norm(q=s["q"].float())),
        (TypeError, lambda: norm(k=s["k"].half())),
        (ValueError, lambda: norm(v=None)),
        (ValueError, lambda: norm(positions=None)),
        (ValueError, lambda: norm(k_out=s["k"])),
        (ValueError, lambda: norm(k_cache=None)),
        (ValueError, lambda: norm(q_weight=s["qw"][:64])),
        (ValueError, lambda: norm(k=s["k"][:, :1], v=s["v"][:, :1])),
        (ValueError, lambda: norm(q=s["q"].transpose(1, 2).contiguous().transpose(1, 2))),
        (ple.PleError, lambda: norm(rope=torch.zeros(65, dtype=torch.int64, device=DEV))),
        (ple.PleError, lambda: norm(eps=-1.0)),
        (TypeError, lambda: commit(path=s["path"].long())),
        (ValueError, lambda: commit(accepted=s["accepted"][:2])),
        (ValueError, lambda: commit(ngram_context=None, next_context=s["context"])),
        (TypeError, lambda: commit(input_ids=s["ids"].float())),
        (TypeError, lambda: commit(k_cache=s["kc"].float(), v_cache=s["vc"].float())),
        (TypeError, lambda: index(parent=s["parent"].long())),
        (ValueError, lambda: index(ctx_lens=s["ctx"][:2])),
        (ple.PleError, lambda: index(mask_words=9)),
        (ValueError, lambda: index(tree_mask=mask, mask_words=2)),
        (ValueError, lambda: row_ids(ngram_size=4)),
        (ValueError, lambda: row_ids(heads_per_ngram=3)),          # the library's geometry check
        (TypeError, lambda: row_ids(ngram_context=s["context"].int())),
        (TypeError, lambda: row_ids(out_dtype=torch.float32)),
        (ValueError, lambda: row_ids(parent=s["parent"][:-1])),
        (ValueError, lambda: ple.ple_prepare_rope(64, scaling="other")),
        (ple.PleError, lambda: ple.ple_prepare_rope(64, factor=0.5, scaling="linear")),
    ]:
        with pytest.raises(error):
            call()
