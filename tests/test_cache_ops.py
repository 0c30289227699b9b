"""The operators on caches in 8 bits and on pages, on the GPU, against plain
64-bit host implementations (cache_reference.py).

Moved and planned numbers are compared bit for bit, and so are elements and
scales wherever they follow from the inputs without a rounding before the one
to 8 bits (half a step of a normal element is 2^-4 of it, of the others 2^-10
scales).  The other bounds follow from the arithmetic and stand where they are
used."""

import numpy as np
import pytest
import torch

import cache_reference as ref8
import layer_gram_embedding_gb300 as ple
import tree_reference as ref
from test_tree_ops import U, check_rows, dev, host, rows

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = torch.device("cuda:0")
FP8 = torch.float8_e4m3fn
ODD_SCALES = np.array([np.nan, np.inf, -np.inf, 0.0, -1.0])


class Cache8:
    """A paged cache in 8 bits in drawn order: any bytes, NaN among them, and scales of any kind
    wherever nothing lives.  Host copies in k, v, k_scale, v_scale; `order` is the caches' layout in
    memory, and scales lie blocks after heads with `gap` numbers between pages."""

    def __init__(self, rng, lengths, page, block, heads, dim, order="phsd", layers=1, spare=2,
                 gap=0, odd=ODD_SCALES):
        per = [max(1, -(-n // page)) for n in lengths]
        pages = sum(per) + spare
        at = rng.permutation(pages)
        self.table = np.full((len(lengths), max(per)), 2 ** 30, np.int32)
        done = 0
        for r, n in enumerate(per):
            self.table[r, :n] = at[done:done + n]
            done += n
        self.page, self.block, self.order, self.gap = page, block, order, gap
        shape = (layers, pages, heads, page, dim)
        self.k, self.v = (rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2))
        self.k_scale, self.v_scale = (rng.choice(odd, (layers, pages, heads, page // block))
                                      for _ in range(2))

    def where(self, r, i):
        return self.table[r][np.asarray(i) // self.page], np.asarray(i) % self.page

    def fill(self, rng, r, first, last, low=-9, high=-5, any_scale=False):
        """Live keys and values in slots first .. last - 1 of request r: elements around 2^5 under
        scales between 2^low and 2^high."""
        i = np.arange(first, last)
        if len(i) == 0:
            return
        p, s = self.where(r, i)
        for c, scales in ((self.k, self.k_scale), (self.v, self.v_scale)):
            c[:, p, :, s] = ref8.encode(40.0 * rng.standard_normal(
                (len(i), c.shape[0], c.shape[2], c.shape[4])))
            new = 2.0 ** rng.integers(low, high + 1, scales.shape)
            if any_scale:
                new = torch.from_numpy(new * rng.uniform(1, 2, new.shape))
                new = new.bfloat16().double().numpy()
            live = np.zeros(scales.shape, bool)
            live[:, p, :, s // self.block] = True
            scales[live] = new[live]

    def device(self):
        """(k, v, k_scale, v_scale) on the GPU, without a first dimension for one layer."""
        out = []
        for c in (self.k, self.v):
            c = dev(c).view(FP8)
            if self.order == "pshd":
                c = c.view(torch.uint8).transpose(2, 3).contiguous().transpose(2, 3).view(FP8)
            out.append(c)
        for s in (self.k_scale, self.v_scale):
            L, P, H, blocks = s.shape
            wide = torch.full((L, P, H * blocks + self.gap), float("nan"), device=DEV,
                              dtype=torch.bfloat16)
            view = wide[:, :, :H * blocks].unflatten(2, (H, blocks))
            view.copy_(dev(s))
            out.append(view)
        return [x[0] for x in out] if self.k.shape[0] == 1 else out


def read(caches):
    """Host copies (bytes, bytes, scales, scales), a first dimension for one layer."""
    out = [c.view(torch.uint8).cpu().numpy() for c in caches[:2]]
    out += [s.double().cpu().numpy() for s in caches[2:]]
    return [x[None] if caches[0].dim() == 4 else x for x in out]


def same(a, b):
    return np.array_equal(a, b, equal_nan=a.dtype.kind == "f")


# --------------------------------------------------------------------- append


def check_append(got, before, new, error, table, ctx, cu, exact):
    """One layer's bytes and scales after the call against what they were.  new [T, heads, D] is
    what was appended, known to `error`."""
    (bytes_, scales), (old, old_scales) = got, before
    kept = old.copy(), old_scales.copy()
    for page, block_at, held, slots, low, high in ref8.append(new, error, old, old_scales, table,
                                                              ctx, cu):
        size = old.shape[2] // old_scales.shape[2]
        at = block_at * size
        for h in range(old.shape[1]):
            s = scales[page, h, block_at]
            least, most = 2.0 ** low[h], 2.0 ** high[h]
            if held:
                least = max(least, old_scales[page, h, block_at])
                most = max(most, old_scales[page, h, block_at])
            assert least <= s <= most, (page, h, block_at, s, least, most)
            kept[1][page, h, block_at] = s
            if held and s > old_scales[page, h, block_at]:
                rows_at = slice(at, at + min(held, size))
                shrunk = ref8.encode(ref8.VALUES[old[page, h, rows_at]] *
                                     (old_scales[page, h, block_at] / s))
                nan = np.isnan(ref8.VALUES[shrunk])
                assert np.array_equal(bytes_[page, h, rows_at][~nan], shrunk[~nan])
                assert np.all(bytes_[page, h, rows_at][nan] & 0x7F == 0x7F)
                kept[0][page, h, rows_at] = bytes_[page, h, rows_at]
            slot, token = (list(x) for x in zip(*slots))
            slot = [at + i for i in slot]
            e, want, around = bytes_[page, h, slot], new[token, h], error[token, h]
            if exact:
                assert np.array_equal(e, ref8.encode(want / s))
            else:
                fine = np.isfinite(want)
                assert np.all(e[~fine] & 0x7F == 0x7F)
                err = np.abs(ref8.VALUES[e] * s - want)[fine]
                bound = np.maximum(2.0 ** -4 * np.abs(want), s * 2.0 ** -10)[fine] + \
                    1.125 * around[fine]
                assert np.all(err <= bound), np.max(err - bound)
            kept[0][page, h, slot] = e
    # nothing else was written
    assert same(bytes_, kept[0]) and same(scales, kept[1])


APPEND_CASES = [
    # counts, ctx, Hq, Hk, D, R, interleaved, page, block
    ([1], [900], 32, 8, 128, 128, False, 64, 64),
    ([1], [0], 4, 1, 64, 64, False, 16, 16),
    ([1, 1, 1], [15, 16, 17], 4, 2, 64, 64, False, 32, 16),
    ([3, 0, 33, 1], [0, 5, 120000, 63], 8, 2, 64, 64, False, 16, 16),
    ([3, 0, 33, 1], [0, 5, 120000, 63], 8, 2, 64, 32, True, 32, 32),
    ([17, 2], [100, 7], 5, 5, 96, 48, False, 48, 16),
    ([17, 2], [100, 7], 4, 1, 80, 40, True, 128, 128),
    ([5], [1000], 3, 1, 256, 256, False, 128, 128),
    ([300], [77], 3, 1, 256, 12, False, 256, 128),
    ([9, 9], [31, 32], 2, 2, 16, 6, False, 16, 16),
    ([9, 9], [31, 32], 2, 2, 16, 0, True, 64, 16),
    ([40], [11], 0, 3, 16, 2, True, 160, 32),
    ([2000, 1500], [1, 2], 4, 2, 128, 64, False, 64, 32),
    ([1300] * 3, [0, 9, 1], 2, 1, 64, 64, True, 128, 128),
    ([257, 1, 130], [31, 63, 64], 6, 2, 112, 112, False, 192, 64),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", APPEND_CASES)
@pytest.mark.parametrize("form", ["fused", "odd strides", "growing"])
def test_qk_norm_rope_fp8(case, dtype, form):
    counts, ctx, Hq, Hk, D, R, interleaved, page, block = case
    rng = np.random.default_rng(sum(counts) + D + R)
    T, B = sum(counts), len(counts)
    qkv = rows(rng, (T, Hq + 2 * Hk, D), dtype, 3.0)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    if form == "odd strides":
        k = k.transpose(0, 1).contiguous().transpose(0, 1)
    qw, kw = rows(rng, (D,), dtype), rows(rng, (D,), dtype)
    ctx = np.array(ctx, np.int32)
    cu = ref.prefix(counts)
    positions = (np.repeat(ctx, counts) + rng.integers(0, 40, T)).astype(np.int32)
    rope = ple.ple_prepare_rope(R, 1e6, "parts", 4.0, 4096.0) if R else None
    w = ref.inverse_frequencies(R, 1e6, "parts", 4.0, 4096.0)
    cache = Cache8(rng, [int(c) + n for c, n in zip(ctx, counts)], page, block, Hk, D,
                   "pshd" if form == "odd strides" else "phsd",
                   gap=3 if form == "odd strides" else 0)
    for r in range(B):
        # what the new tokens join: under scales that stay, or that they outgrow
        low = -30 if form == "growing" else -7
        cache.fill(rng, r, int(ctx[r]) // block * block, int(ctx[r]), low, low + 12,
                   any_scale=form == "odd strides")
    caches = cache.device()
    before = read(caches)
    got = ple.ple_qk_norm_rope_fp8(q, k, v, dev(positions) if R else None, rope, qw, kw, *caches,
                                   dev(cache.table), dev(ctx), dev(cu), eps=1e-5,
                                   interleaved=interleaved, rope_scale=1.25)
    want, size = ref.norm_rope(host(q), host(qw), positions, w, 1e-5, interleaved, 1.25)
    check_rows(got, want, size, U[dtype], "q")
    want, size = ref.norm_rope(host(k), host(kw), positions, w, 1e-5, interleaved, 1.25)
    after = read(caches)
    # 32-bit norm, products and angle (2e-7 radians)
    check_append((after[0][0], after[2][0]), (before[0][0], before[2][0]), want,
                 2.0 ** -20 * size + 2.0 ** -40, cache.table, ctx, cu, exact=False)
    check_append((after[1][0], after[3][0]), (before[1][0], before[3][0]), host(v),
                 np.zeros(v.shape), cache.table, ctx, cu, exact=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_append_without_norm_or_rotation_is_exact(dtype):
    # keys as they come: extremes of the types, signed zeros, infinities, NaN, rows of zeros
    rng = np.random.default_rng(5)
    k, v = (rows(rng, (50, 2, 64), dtype) for _ in range(2))
    for x in (k, v):
        x[3] = 0
        x[4, 0, 5] = -0.0
        x[7, 1, 2] = float("inf")
        x[9, 0, 3] = float("-inf")
        x[20, 1, 9] = float("nan")
        x[30:32] = float("nan")
        x[33, 0, 0] = torch.finfo(dtype).max
        x[34, 1, 1] = torch.finfo(dtype).tiny
    ctx, cu = np.array([5, 40], np.int32), ref.prefix([30, 20])
    cache = Cache8(rng, [35, 60], 32, 16, 2, 64)
    for r in range(2):
        cache.fill(rng, r, 0, int(ctx[r]))
    caches = cache.device()
    before = read(caches)
    q = rows(rng, (50, 4, 64), dtype)
    got = ple.ple_qk_norm_rope_fp8(q, k, v, None, None, None, None, *caches, dev(cache.table),
                                   dev(ctx), dev(cu))
    assert torch.equal(got, q)
    after = read(caches)
    for i, x in ((0, k), (1, v)):
        check_append((after[i][0], after[i + 2][0]), (before[i][0], before[i + 2][0]), host(x),
                     np.zeros(x.shape), cache.table, ctx, cu, exact=True)


def test_append_of_nothing_that_is_finite():
    k = torch.full((1, 1, 16), float("nan"), dtype=torch.bfloat16, device=DEV)
    cache = Cache8(np.random.default_rng(6), [1], 16, 16, 1, 16)
    caches = cache.device()
    ple.ple_qk_norm_rope_fp8(k[:, :0], k, torch.zeros_like(k), None, None, None, None, *caches,
                             dev(cache.table), dev(np.array([0], np.int32)),
                             dev(np.array([0, 1], np.int32)))
    after = read(caches)
    p = cache.table[0, 0]
    assert after[2][0, p, 0, 0] == 2.0 ** -100 and after[3][0, p, 0, 0] == 2.0 ** -100
    assert np.all(after[0][0, p, 0, 0] & 0x7F == 0x7F) and np.all(after[1][0, p, 0, 0] == 0)


def test_append_outside_the_page_table_is_dropped():
    rng = np.random.default_rng(3)
    k, v = (rows(rng, (60, 1, 64), torch.bfloat16) for _ in range(2))
    cache = Cache8(rng, [48], 16, 16, 1, 64)
    for bad in (-1, 10 ** 6):
        cache.table[0, 1] = bad
        caches = cache.device()
        before = read(caches)
        ctx, cu = np.array([4], np.int32), np.array([0, 60], np.int32)
        cache.fill(rng, 0, 0, 0)
        ple.ple_qk_norm_rope_fp8(k, k, v, None, None, None, None, *caches, dev(cache.table),
                                 dev(ctx), dev(cu))
        after = read(caches)
        p = [int(cache.table[0, 0]), int(cache.table[0, 2])]
        assert np.array_equal(np.unique(np.nonzero(after[1] != before[1])[1]), np.sort(p))
        # slots 32 .. 47: tokens 28 .. 43
        s = after[3][0, p[1], 0, 0]
        assert np.array_equal(after[1][0, p[1], 0], ref8.encode(host(v)[28:44, 0] / s))


def test_padding_tokens_append_nothing():
    # seven tokens of a fixed shape, four of them nodes; the last request has room behind its own
    rng = np.random.default_rng(19)
    k, v = (rows(rng, (7, 1, 64), torch.float16) for _ in range(2))
    cache = Cache8(rng, [16, 32], 16, 16, 1, 64)
    ctx, cu = np.array([0, 16], np.int32), np.array([0, 3, 4], np.int32)
    caches = cache.device()
    before = read(caches)
    ple.ple_qk_norm_rope_fp8(k, k, v, None, None, None, None, *caches, dev(cache.table), dev(ctx),
                             dev(cu))
    after = read(caches)
    for i, x in ((0, k), (1, v)):
        check_append((after[i][0], after[i + 2][0]), (before[i][0], before[i + 2][0]), host(x),
                     np.zeros(x.shape), cache.table, ctx, cu, exact=True)


def guarded(caches):
    """The same caches inside wider memory whose first and last pages hold a pattern."""
    wide = []
    for c in caches:
        c = c.view(torch.uint8) if c.dtype == FP8 else c
        w = torch.full((c.shape[0] + 4, *c.shape[1:]), 5, dtype=c.dtype, device=DEV)
        w[2:-2] = c
        wide.append(w)
    inner = [w[2:-2].view(FP8) if w.dtype == torch.uint8 else w[2:-2] for w in wide]
    return inner, lambda: all(bool((w[:2] == 5).all()) and bool((w[-2:] == 5).all()) for w in wide)


def test_append_of_any_layout_stays_in_bounds():
    # any prefix sums, lengths, pages and positions: what is written is unspecified, where is not
    rng = np.random.default_rng(11)
    q, k, v = (rows(rng, (90, 2, 64), torch.bfloat16) for _ in range(3))
    cache = Cache8(rng, [64] * 3, 16, 16, 2, 64)
    for i in range(8):
        caches, intact = guarded(cache.device())
        table, ctx, cu, positions = (rng.integers(-2 ** 31, 2 ** 31, n).astype(np.int32)
                                     for n in ((3, 4), 3, 4, 90))
        if i % 2:
            table, ctx, cu = rng.integers(-2, 16, (3, 4)).astype(np.int32), ctx % 80, cu % 100
        ple.ple_qk_norm_rope_fp8(q, k, v, dev(positions), ple.ple_prepare_rope(64), None, None,
                                 *caches, dev(table), dev(ctx), dev(cu))
        assert intact()


# ------------------------------------------------------------------ attention


def attention_inputs(rng, counts, ctx, Hq, Hk, D, page, block, dtype, order="phsd", any_scale=False,
                     low=-9, high=-5):
    ctx = np.array(ctx, np.int32)
    cu = ref.prefix(counts)
    lengths = [int(c) + n for c, n in zip(ctx, counts)]
    cache = Cache8(rng, lengths, page, block, Hk, D, order, gap=5 if order == "pshd" else 0)
    for r, n in enumerate(lengths):
        cache.fill(rng, r, 0, n, low, high, any_scale)
    words = max(1, -(-max(counts) // 64))
    _, masks = ref.tree_index(ref.trees(rng, counts), cu, ctx, words)
    q = rows(rng, (sum(counts), Hq, D), dtype)
    return q, cache, ctx, cu, masks


def check_attention(q, cache, ctx, cu, masks, scale=None, what="", caches=None, **kw):
    """The call against the formula.  Errors: queries enter as sums of elements or as halves (what
    lies below 2^-17 of the row's largest is lost); 32-bit scores (D + 16 roundings); the output's
    rounding; weights times value scales as halves, to 2^-11 of each or 2^-27 of the largest near
    it; one 32-bit sum for each 16 slots; an approximated logarithm (2^-18, as its error in the
    exponent counts twice) of scales that are no powers of two."""
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    caches = cache.device() if caches is None else caches
    out, lse = ple.ple_tree_attention_fp8(q, *caches, dev(cache.table), dev(ctx), dev(cu),
                                          dev(masks), scale=scale, return_lse=True, **kw)
    n = int(cu[-1])
    k, v = (ref8.dequantise(c[0], s[0]) for c, s in ((cache.k, cache.k_scale),
                                                     (cache.v, cache.v_scale)))
    want, want_lse, weight, reach, spread, flush = ref8.attention(
        host(q)[:n], k, v, cache.v_scale[0], cache.table, ctx, cu, masks[:n], scale)
    u, D = U[q.dtype], q.shape[-1]
    score = 2.0 ** -23 * (D + 16) * reach + 2.0 ** -17 * spread + 2.0 ** -20
    steps = (max([int(c) for c in ctx], default=0) + 1024) / 16
    bound = u * (1 + 2.0 ** -8) * np.abs(want) + 2.0 ** -25 + 2.0 ** -27 * flush + \
        (2.0 ** -11 * (1 + 2.0 ** -8) + 2.0 ** -18 + 2.0 ** -23 * steps +
         2 * score[..., None]) * weight
    got = host(out)[:n]
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    err = np.abs(got - want)
    assert np.all(err[fine] <= bound[fine]), f"{what}: {np.max((err - bound)[fine])} over the bound"
    got = host(lse)[:n]
    fine = np.isfinite(want_lse)
    assert np.array_equal(got[~fine & ~np.isnan(want_lse)], want_lse[~fine & ~np.isnan(want_lse)])
    err = np.abs(got[fine] - want_lse[fine])
    assert np.all(err <= (score + 2.0 ** -20 + 2.0 ** -22 * np.abs(want_lse))[fine]), what
    return out, lse


ATTENTION_CASES = [
    # counts, ctx, Hq, Hk, D, page, block, order
    ([1], [0], 1, 1, 64, 16, 16, "phsd"),
    ([1], [700], 32, 8, 128, 64, 64, "phsd"),
    ([1, 1, 1], [127, 128, 129], 4, 1, 128, 64, 32, "phsd"),
    ([5, 0, 33, 1], [0, 9, 511, 64], 8, 2, 64, 16, 16, "phsd"),
    ([64, 3], [300, 1], 16, 2, 128, 32, 32, "phsd"),
    ([17], [1000], 10, 2, 128, 128, 128, "pshd"),
    ([70, 129], [50, 257], 8, 4, 128, 64, 16, "phsd"),
    ([200], [3], 4, 4, 64, 256, 128, "phsd"),
    ([33], [95], 5, 1, 64, 16, 16, "phsd"),
    ([9, 2], [40, 77], 6, 2, 96, 16, 16, "phsd"),
    ([9, 2], [40, 77], 9, 1, 256, 48, 16, "pshd"),
    ([9, 2], [40, 77], 3, 3, 16, 16, 16, "phsd"),
    ([4] * 37, list(range(0, 370, 10)), 4, 2, 64, 16, 16, "phsd"),
    ([2], [5000], 4, 1, 128, 64, 64, "phsd"),
    ([512], [130], 2, 1, 64, 64, 64, "phsd"),
    # more tiles than the device has SMs: shares of many tiles and requests
    ([2] * 40, [100 + 19 * i for i in range(40)], 16, 8, 128, 16, 16, "phsd"),
    ([3, 0, 1, 30] * 12, [37 * i for i in range(48)], 16, 4, 64, 64, 32, "phsd"),
    ([40, 64, 33], [2500, 900, 3000], 32, 4, 64, 32, 16, "phsd"),
    ([18], [9001], 32, 4, 128, 64, 64, "phsd"),
    ([1, 1], [20000, 11], 4, 2, 128, 128, 128, "phsd"),
    # rows a key head around the borders of the rule, and other widths and pages
    ([8], [333], 2, 2, 128, 32, 16, "phsd"), ([9], [333], 2, 2, 128, 32, 16, "phsd"),
    ([16], [333], 2, 2, 64, 32, 32, "pshd"), ([17], [333], 2, 2, 64, 32, 32, "phsd"),
    ([64], [640], 4, 2, 128, 64, 64, "phsd"), ([65], [640], 4, 2, 128, 64, 64, "phsd"),
    ([64], [640], 8, 2, 256, 64, 64, "phsd"), ([50, 50], [90, 300], 8, 1, 256, 96, 32, "pshd"),
    ([1, 3], [5000, 0], 20, 2, 256, 16, 16, "phsd"),
    ([1, 40], [3001, 129], 6, 2, 112, 48, 16, "pshd"),
    ([33, 2], [500, 1000], 8, 2, 80, 384, 128, "phsd"),
    ([60, 70], [90, 300], 8, 8, 48, 16, 16, "phsd"),
    ([16, 1, 0, 2], [3000, 40000, 2, 0], 8, 8, 32, 64, 64, "phsd"),
    ([300], [700], 8, 1, 128, 64, 32, "phsd"),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", ATTENTION_CASES)
def test_tree_attention_fp8(case, dtype):
    counts, ctx, Hq, Hk, D, page, block, order = case
    rng = np.random.default_rng(sum(counts) + D + page)
    args = attention_inputs(rng, counts, ctx, Hq, Hk, D, page, block, dtype, order,
                            any_scale=page % 32 == 0)
    check_attention(*args, what=str(case))


# rows a key head: those of few rows (one product of 8 and of 16) and those of many (128, 256)
KERNELS = [([2], 4), ([6], 4), ([14], 4), ([40], 8)]


@pytest.mark.parametrize("counts,Hq", KERNELS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_of_scales_far_apart(counts, Hq, dtype):
    # a block's values 2^60 times another's: what is small keeps its own bits where it is seen
    # alone; keys of ordinary sizes, or scores would be single keys
    rng = np.random.default_rng(21)
    q, cache, ctx, cu, masks = attention_inputs(rng, counts, [400], Hq, 2, 64, 32, 16, dtype)
    live = np.isfinite(cache.v_scale)
    cache.v_scale[live] = np.where(cache.v_scale[live] > 0,
                                   2.0 ** rng.integers(-40, 6, live.sum()), cache.v_scale[live])
    check_attention(q, cache, ctx, cu, masks)


@pytest.mark.parametrize("counts,Hq", KERNELS)
def test_attention_of_small_and_odd_scales(counts, Hq):
    rng = np.random.default_rng(22)
    args = attention_inputs(rng, counts, [400], Hq, 2, 128, 32, 16, torch.bfloat16)
    q, cache, ctx, cu, masks = args
    p, _ = cache.where(0, np.arange(400 + counts[0]))
    p = np.unique(p)
    cache.v_scale[0, p, 0] = 2.0 ** -100              # as of rows of zeros
    cache.k_scale[0, p, 1] = 2.0 ** -100              # all scores near 0
    cache.v_scale[0, p[::2], 1] = 0.0                 # values that are 0
    check_attention(*args)


@pytest.mark.parametrize("counts,Hq", KERNELS)
@pytest.mark.parametrize("scale", [0.0, -0.3, 40.0])
def test_attention_of_other_scores(counts, Hq, scale):
    rng = np.random.default_rng(23)
    args = attention_inputs(rng, counts, [700], Hq, 2, 64, 64, 32, torch.float16, low=-9, high=-8)
    check_attention(*args, scale=scale)


@pytest.mark.parametrize("counts,Hq", KERNELS)
def test_attention_of_rising_scores(counts, Hq):
    # references move again and again: scores rise along the context, value scales fall, and
    # the other way round in the second head
    rng = np.random.default_rng(24)
    q, cache, ctx, cu, masks = attention_inputs(rng, counts, [3000], Hq, 2, 64, 16, 16,
                                                torch.bfloat16)
    n = 3000 + counts[0]
    p, s = cache.where(0, np.arange(n))
    rise = np.linspace(0, 1, n)
    q[..., 0] = 8.0
    for h, way in ((0, rise), (1, rise[::-1])):
        cache.k[0, p, h, s, 0] = ref8.encode(400 * way)
        cache.k_scale[0, p, h, s // 16] = 2.0 ** -3
        cache.v_scale[0, p, h, s // 16] = 2.0 ** np.round(-40 * way)
    check_attention(q, cache, ctx, cu, masks, scale=0.4)


@pytest.mark.parametrize("counts,Hq", KERNELS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_of_rows_that_see_nothing(counts, Hq, dtype):
    rng = np.random.default_rng(25)
    q, cache, ctx, cu, masks = attention_inputs(rng, counts, [0], Hq, 2, 64, 16, 16, dtype)
    masks[:] = 0
    out, lse = check_attention(q, cache, ctx, cu, masks)
    assert not out.any() and bool((lse == float("-inf")).all())
    masks[0] = 1      # one row that sees one slot
    check_attention(q, cache, ctx, cu, masks)


@pytest.mark.parametrize("counts,Hq", KERNELS)
@pytest.mark.parametrize("ctx", [5, 128, 300])
def test_attention_of_bad_slots(counts, Hq, ctx):
    rng = np.random.default_rng(26)
    q, cache, lens, cu, masks = attention_inputs(rng, counts, [ctx], Hq, 2, 64, 16, 16,
                                                 torch.bfloat16)
    # a drafted node's value, and another's key, are NaN in one element of one head
    p, s = cache.where(0, ctx + np.array([0, 1]))
    cache.v[0, p[0], 0, s[0], 7] = 0x7F
    cache.k[0, p[1], 1, s[1], 3] = 0xFF
    masks[:, 0] = 1 << np.arange(counts[0], dtype=np.int64)    # nodes see themselves alone
    k = ref8.dequantise(cache.k[0], cache.k_scale[0])
    out, lse = ple.ple_tree_attention_fp8(q, *cache.device(), dev(cache.table), dev(lens), dev(cu),
                                          dev(masks), return_lse=True)
    got = np.isnan(host(out)).any(-1)
    want = np.zeros(got.shape, bool)
    want[0, :Hq // 2] = want[1, Hq // 2:] = True
    assert np.array_equal(got, want) and np.isnan(k).any()
    # of a cached slot: every row of the head
    p, s = cache.where(0, ctx - 2)
    cache.v[0, p, 1, s, 9] = 0x7F
    out = ple.ple_tree_attention_fp8(q, *cache.device(), dev(cache.table), dev(lens), dev(cu),
                                     dev(masks))
    want[:, Hq // 2:] = True
    assert np.array_equal(np.isnan(host(out)).any(-1), want)


@pytest.mark.parametrize("counts,Hq", KERNELS)
def test_attention_of_blocks_that_no_row_sees(counts, Hq):
    # scales and elements of the last node's block may be anything when nobody sees that node
    rng = np.random.default_rng(27)
    n = counts[0]
    ctx = 48 - (n - 1)
    q, cache, lens, cu, masks = attention_inputs(rng, counts, [ctx], Hq, 2, 64, 16, 16,
                                                 torch.float16)
    masks[:] &= (1 << (n - 1)) - 1
    masks[n - 1] = 1
    p, s = cache.where(0, ctx + n - 1)
    assert s == 0
    for bad in (np.nan, np.inf, -np.inf, 0.0):
        cache.k_scale[0, p, :, 0] = cache.v_scale[0, p, :, 0] = bad
        cache.k[0, p, :, 0], cache.v[0, p, :, 0] = 0x7F, 0xFF
        check_attention(q, cache, lens, cu, masks, what=str(bad))


@pytest.mark.parametrize("counts,Hq", KERNELS)
def test_attention_padding_rows_and_outputs_given(counts, Hq):
    # rows behind the last request's stay as they were
    rng = np.random.default_rng(28)
    q, cache, ctx, cu, masks = attention_inputs(rng, counts + [3], [77, 200], Hq, 2, 128, 32, 16,
                                                torch.bfloat16)
    n = int(cu[-1])
    wide = torch.zeros((n + 5, Hq + 3, 136), dtype=q.dtype, device=DEV)
    wide[:n, 2:Hq + 2, :128] = q
    view = wide[:, 2:Hq + 2, :128]
    view[n:] = float("nan")
    more = np.concatenate([masks, np.full((5, masks.shape[1]), -1)])
    out = torch.full((n + 5, Hq, 128), 9.0, dtype=q.dtype, device=DEV)
    lse = torch.full((n + 5, Hq), 9.0, device=DEV)
    workspace = ple.ple_tree_attention_fp8_workspace(n + 5, Hq, 2, 128)
    workspace.fill_(255)  # need not be cleared
    got = check_attention(view, cache, ctx, cu, more, out=out, lse=lse, workspace=workspace)
    assert got[0] is out and got[1] is lse
    assert bool((out[n:] == 9).all()) and bool((lse[n:] == 9).all())


@pytest.mark.parametrize("counts,Hq", KERNELS)
def test_attention_pages_outside_the_cache_read_as_zeros(counts, Hq):
    rng = np.random.default_rng(29)
    q, cache, ctx, cu, masks = attention_inputs(rng, counts + counts, [400, 333], Hq, 2, 64, 16, 16,
                                                torch.bfloat16)
    lost = int(cache.table[0, 3])
    out = []
    for page in (-1, 2 ** 31 - 1, -2 ** 31, None):
        if page is None:  # the same page, holding zeros under scales of 1
            cache.table[0, 3] = lost
            cache.k[0, lost] = cache.v[0, lost] = 0
            cache.k_scale[0, lost] = cache.v_scale[0, lost] = 1
        else:
            cache.table[0, 3] = page
        out.append(ple.ple_tree_attention_fp8(q, *cache.device(), dev(cache.table), dev(ctx),
                                              dev(cu), dev(masks), return_lse=True))
    for o in out[:3]:
        assert torch.equal(o[0], out[3][0]) and torch.equal(o[1], out[3][1])


@pytest.mark.parametrize("counts,Hq", KERNELS)
def test_attention_of_any_lengths_and_pages_stays_in_bounds(counts, Hq):
    rng = np.random.default_rng(30)
    q, cache, ctx, cu, masks = attention_inputs(rng, counts * 3, [40, 33, 7], Hq, 2, 64, 16, 16,
                                                torch.float16)
    caches, intact = guarded(cache.device())
    for _ in range(4):
        table = rng.integers(-2 ** 31, 2 ** 31, cache.table.shape).astype(np.int32)
        lens = rng.integers(-2 ** 31, 2 ** 31, 3).astype(np.int32)
        words = rng.integers(-2 ** 63, 2 ** 63, masks.shape)
        for t, l in ((table, ctx), (cache.table, lens), (table, lens)):
            ple.ple_tree_attention_fp8(q, *caches, dev(t), dev(l), dev(cu), dev(words))
    torch.cuda.synchronize()
    assert intact()


@pytest.mark.parametrize("counts,Hq", KERNELS)
def test_attention_is_the_same_every_time(counts, Hq):
    rng = np.random.default_rng(31)
    q, cache, ctx, cu, masks = attention_inputs(rng, counts, [6000], Hq, 2, 128, 64, 64,
                                                torch.bfloat16)
    args = (q, *cache.device(), dev(cache.table), dev(ctx), dev(cu), dev(masks))
    want = ple.ple_tree_attention_fp8(*args, return_lse=True)
    for _ in range(20):
        got = ple.ple_tree_attention_fp8(*args, return_lse=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("counts,Hq", [([3], 4), ([40], 4)])
def test_attention_offsets_past_32_bits(counts, Hq):
    # a cache of more than 2^32 elements, the request's pages at its far end
    page, heads, D = 64, 2, 128
    pages = 2 ** 32 // (page * heads * D) + 40
    rng = np.random.default_rng(15)
    q, cache, ctx, cu, masks = attention_inputs(rng, counts, [197], Hq, heads, D, page, 16,
                                                torch.bfloat16)
    few = cache.k.shape[1]
    want = check_attention(q, cache, ctx, cu, masks)
    small = cache.device()
    k, v = (torch.zeros((pages, heads, page, D), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((pages, heads, 4), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for t, s in zip((k, v, ks, vs), small):
        t[-few:] = s.view(torch.uint8) if s.dtype == FP8 else s
    out = ple.ple_tree_attention_fp8(q, k.view(FP8), v.view(FP8), ks, vs,
                                     dev(cache.table + (pages - few)), dev(ctx), dev(cu),
                                     dev(masks), return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(out, want))


# --------------------------------------------------------------------- commit


def commit_inputs(rng, counts, ctx, P, layers, Hk, D, page, block, order, any_scale):
    ctx, cu = np.array(ctx, np.int32), ref.prefix(counts)
    cache = Cache8(rng, [int(c) + n for c, n in zip(ctx, counts)], page, block, Hk, D, order,
                   layers, gap=1 if order == "pshd" else 0)
    for r, n in enumerate(counts):
        cache.fill(rng, r, 0, int(ctx[r]) + n, -12, -4, any_scale)
    path = np.zeros((len(counts), P), np.int32)
    accepted = np.zeros(len(counts), np.int32)
    for r, n in enumerate(counts):
        kept = int(rng.integers(0, min(n, P) + 1))
        accepted[r] = kept
        path[r, :kept] = np.sort(rng.choice(n, kept, replace=False))
    ids, context = rng.integers(0, 1000, sum(counts)), rng.integers(0, 1000, (len(counts), 2))
    return ctx, cu, cache, path, accepted, ids, context


def check_commit(inputs, exact=True):
    ctx, cu, cache, path, accepted, ids, context = inputs
    caches = cache.device()
    nxt, lens = ple.ple_tree_commit_fp8(dev(ids), dev(path), dev(accepted), dev(cu), dev(context),
                                        dev(ctx), dev(cache.table), *caches)
    kept = np.minimum(np.minimum(np.maximum(accepted, 0), path.shape[1]), np.diff(cu))
    assert np.array_equal(lens.cpu().numpy(), ctx + kept)
    after = read(caches)
    for i, (c, s) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        want, want_scales = ref8.commit(path, accepted, cu, ctx, cache.table, c, s)
        assert same(after[i + 2], want_scales)
        if exact:
            assert same(after[i], want)
        else:
            # quotients of scales that are no powers of two are rounded (2^-24): elements at
            # the border between two may fall to the other side
            differ = after[i] != want
            assert differ.mean() < 2.0 ** -10
            assert np.all(np.abs(after[i][differ].astype(int) - want[differ]) <= 1)
    return nxt


@pytest.mark.parametrize("counts,ctx,P,layers,Hk,D,page,block,order", [
    ([9], [700], 3, 1, 8, 128, 64, 64, "phsd"),
    ([9, 0, 33, 1], [0, 5, 63, 16], 9, 3, 2, 64, 16, 16, "phsd"),
    ([200, 130], [1, 30], 150, 2, 3, 16, 160, 32, "pshd"),
    ([12] * 20, list(range(20)), 6, 4, 1, 256, 48, 16, "phsd"),
    ([300, 2], [100, 127], 290, 1, 5, 96, 128, 128, "pshd"),
    ([70], [13], 60, 2, 40, 48, 32, 32, "phsd"),
])
@pytest.mark.parametrize("any_scale", [False, True])
def test_tree_commit_fp8(counts, ctx, P, layers, Hk, D, page, block, order, any_scale):
    rng = np.random.default_rng(sum(counts) + P)
    inputs = commit_inputs(rng, counts, ctx, P, layers, Hk, D, page, block, order, any_scale)
    nxt = check_commit(inputs, exact=not any_scale)
    ctx, cu, cache, path, accepted, ids, context = inputs
    assert np.array_equal(nxt.cpu().numpy(), ref.next_context(ids, path, accepted, cu, context))


def test_commit_of_paths_and_pages_that_are_not_sound():
    # nodes below their place or past the request's leave their slot; pages that are none are
    # passed over; counts past the path's length and below 0 are cut
    rng = np.random.default_rng(41)
    inputs = commit_inputs(rng, [20, 20, 20, 20], [10, 25, 40, 3], 8, 2, 2, 64, 16, 16, "phsd",
                           False)
    ctx, cu, cache, path, accepted, ids, context = inputs
    path[0] = [3, 0, 19, 2, 25, 2 ** 31 - 1, -2 ** 31, 7]
    path[1] = [0, 1, 2, 3, 4, 5, 6, 7]
    path[2] = [5, 6, 7, 9, 11, 13, 15, 19]
    path[3] = [2, 4, 6, 8, 10, 12, 14, 16]
    accepted[:] = [100, 8, 8, -5]
    cache.table[2, 3] = 10 ** 6      # where the nodes from 8 on are
    check_commit(inputs)
    cache.table[2, 2] = -1           # where they go
    check_commit(inputs)


# ---------------------------------------------------------------- plan, copies


def check_plan(table, ctx, source, want, pages, page_size, limit=None):
    table, ctx, source, want = (np.asarray(x, np.int32) for x in (table, ctx, source, want))
    got = ple.ple_plan_pages(dev(table), dev(ctx), dev(source), dev(want), pages, page_size, limit)
    limit = pages if limit is None else limit
    nxt, lens, copies, counts = ref8.plan(table, ctx, source, want, pages, page_size, limit)
    assert np.array_equal(got[0].cpu().numpy(), nxt)
    assert np.array_equal(got[1].cpu().numpy(), lens)
    listed = got[2].cpu().numpy()
    assert listed.shape == (len(source) + pages - limit, 2)
    assert listed[:len(copies)].tolist() == [list(c) for c in copies]
    assert np.all(listed[len(copies):] == -1)
    assert got[3].tolist() == counts
    return got


def batch_of(rng, B, max_pages, page_size, pages, shared=0.3):
    """Tables as of plans before: requests that share the pages of their common past."""
    table, ctx = np.full((B, max_pages), -1, np.int32), np.zeros(B, np.int32)
    free = list(rng.permutation(pages))
    for r in range(B):
        if r and rng.random() < shared:
            s = int(rng.integers(0, r))
            common = int(rng.integers(0, ctx[s] // page_size + 1))
            table[r, :common] = table[s, :common]
        else:
            common = 0
        most = min(max_pages, common + len(free))
        ctx[r] = rng.integers(common * page_size, most * page_size + 1)
        for e in range(common, -(-int(ctx[r]) // page_size)):
            table[r, e] = free.pop()
    return table, ctx


@pytest.mark.parametrize("B,N,max_pages,page_size,pages", [
    (1, 1, 1, 1, 1), (1, 4, 8, 16, 40), (3, 5, 7, 48, 64), (16, 16, 10, 16, 300),
    (40, 64, 33, 5, 1500), (5, 300, 12, 16, 2000), (300, 3, 4, 128, 1200),
    (256, 256, 60, 64, 17000), (2, 9000, 2, 16, 12000),
])
@pytest.mark.parametrize("limited", [False, True])
def test_plan_pages(B, N, max_pages, page_size, pages, limited):
    rng = np.random.default_rng(B + N + pages)
    for part in (0.5, 0.95):
        # how much of the pages the old requests may hold: with the second, pages run out
        table, ctx = batch_of(rng, B, max_pages, page_size, max(1, int(pages * part)))
        table[table >= 0] = rng.permutation(pages)[table[table >= 0]]
        source = rng.integers(-1, B, N)
        want = rng.choice([0, 1, 2, page_size, 3 * page_size + 1, -7], N)
        limit = int(rng.integers(0, pages + 1)) if limited else None
        check_plan(table, ctx, source, want, pages, page_size, limit)


def test_plan_of_tables_that_are_not_sound():
    # numbers that are no page, lengths out of range, sources out of range, a page twice in a row
    table = np.array([[2 ** 30, 3, -1, 5], [3, 3, 7, 0], [1, 2, 4, 6]], np.int32)
    ctx = np.array([50, 2 ** 31 - 1, -9], np.int32)
    check_plan(table, ctx, [0, 1, 2, 3, -2 ** 31, 0, 1], [5, 2, 2 ** 31 - 1, 1, 0, 0, 3], 12, 16)
    check_plan(table, ctx, [0, 1, 2, 3, -2 ** 31, 0, 1], [5, 2, 2 ** 31 - 1, 1, 0, 0, 3], 12, 16, 4)
    rng = np.random.default_rng(42)
    for _ in range(4):
        check_plan(rng.integers(-2 ** 31, 2 ** 31, (3, 4)), rng.integers(-2 ** 31, 2 ** 31, 3),
                   rng.integers(-3, 6, 9), rng.integers(-2 ** 31, 2 ** 31, 9), 30, 16, 11)


def test_plan_of_an_empty_batch():
    got = check_plan(np.zeros((0, 5), np.int32), [], [0, -1], [70, 16], 9, 16)
    assert got[0].tolist() == [[0, 1, 2, 3, 4], [5, -1, -1, -1, -1]]
    check_plan([[0, 1]], [20], [0], [0], 2, 16, 0)      # nothing may stay, and nothing can move


@pytest.mark.parametrize("layers,pages,Hk,page,D,order", [
    (1, 9, 2, 16, 64, "phsd"), (3, 40, 8, 64, 128, "phsd"), (2, 30, 3, 48, 16, "pshd"),
    (48, 12, 1, 16, 256, "phsd"),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, FP8])
@pytest.mark.parametrize("count", [0, 1, 2, 100])
def test_copy_pages(layers, pages, Hk, page, D, order, dtype, count):
    rng = np.random.default_rng(layers + D + count)
    cache = Cache8(rng, [1], page, 16, Hk, D, order, layers, spare=pages - 1, gap=count % 3,
                   odd=np.array([1.0, 2.0, -3.0, 0.0, 2.0 ** -100]))
    caches = cache.device()
    if layers == 1:
        caches = [c.unsqueeze(0) for c in caches]
    if dtype != FP8:
        # any two bytes
        caches = [(c.view(torch.uint8).to(torch.int16) * 257 - 9).view(dtype) for c in caches[:2]]
    bits = torch.uint8 if dtype == FP8 else torch.int16
    before = [c.view(bits).clone() if c.dtype == dtype else c.clone() for c in caches]
    n = min(count, pages // 2)
    numbers = rng.permutation(pages)
    copies = np.stack([numbers[:n], numbers[n:2 * n]], 1).astype(np.int32)
    listed = np.full((count, 2), -1, np.int32)
    listed[np.sort(rng.choice(count, n, replace=False))] = copies
    # numbers that are no page are passed over
    for i in range(count):
        if listed[i, 0] < 0:
            listed[i] = [[-1, -1], [0, pages], [pages, 0], [-2 ** 31, 1], [0, -1]][i % 5]
    if layers == 1:
        ple.ple_copy_pages(dev(listed), *[c[0] for c in caches])
    else:
        ple.ple_copy_pages(dev(listed), *caches)
    for now, old in zip(caches, before):
        want = old.clone()
        want[:, copies[:, 1]] = old[:, copies[:, 0]]
        assert torch.equal(now.view(bits) if now.dtype == dtype else now, want)


def test_copy_offsets_past_32_bits():
    pages = 2 ** 32 // (64 * 2 * 128) + 9
    k = torch.zeros((pages, 2, 64, 128), dtype=torch.uint8, device=DEV)
    k[pages - 1] = torch.randint(0, 256, k.shape[1:], dtype=torch.uint8, device=DEV)
    s = torch.ones((pages, 2, 4), dtype=torch.bfloat16, device=DEV)
    s[pages - 1] = 3
    copies = dev(np.array([[pages - 1, pages - 4], [-1, -1]], np.int32))
    # one memory for both caches: the same bytes arrive
    ple.ple_copy_pages(copies, k.view(FP8), k.view(FP8), s, s)
    assert torch.equal(k[pages - 4], k[pages - 1]) and bool((s[pages - 4] == 3).all())
    assert not k[pages - 3].any() and not k[pages - 5].any()
