"""Plain 64-bit implementations of the operators on caches in 8 bits and on
pages, on host arrays, for the tests to compare with.  A cache is bytes
[pages, heads, page_size, D]; scales are 64-bit numbers [pages, heads, blocks]."""

import math

import numpy as np
import torch

import tree_reference as ref

# the value of every byte: four significant bits down to 2^-6, a spacing of 2^-9 below, no
# infinities; both signs of 0x7F are NaN
VALUES = torch.arange(256).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
POSITIVE = VALUES[:0x7F]    # ascending
LEAST = -100                # exponent of the least scale that is written


def encode(x):
    """The nearest elements, ties to even, the largest past 448; NaN where x is not finite."""
    x = np.asarray(x, np.float64)
    size = np.abs(np.where(np.isfinite(x), x, 0.0))
    with np.errstate(divide="ignore"):
        e = np.maximum(np.floor(np.log2(size)), -6.0)
    size = np.minimum(np.rint(size * 2.0 ** (3 - e)) * 2.0 ** (e - 3), 448.0)
    out = np.searchsorted(POSITIVE, size).astype(np.uint8)
    out = out | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isfinite(x), out, 0x7F).astype(np.uint8)


def scale_for(most):
    """The exponent of the least scale for a largest amount."""
    if most <= 448.0 * 2.0 ** LEAST:
        return LEAST
    k = math.ceil(math.log2(most / 448.0))
    while most > 448.0 * 2.0 ** k:
        k += 1
    while most <= 448.0 * 2.0 ** (k - 1):
        k -= 1
    return k


def dequantise(bytes_, scales):
    """The cache in 64 bits."""
    block = bytes_.shape[2] // scales.shape[2]
    with np.errstate(invalid="ignore"):    # 0 under an infinite scale, where nothing lives
        return VALUES[bytes_] * np.repeat(scales, block, 2)[..., None]


def append(new, error, bytes_, scales, table, ctx, cu):
    """For every cache block that new rows [T, heads, D] (finite or not, known to `error`) go to:
    (its page, its place in the page, live slots of before, [(slot in the block, token)], least
    and most exponent of the scale that they need, by head)."""
    page, blocks = bytes_.shape[2], scales.shape[2]
    block = page // blocks
    out = []
    for r in range(len(cu) - 1):
        n, c = int(cu[r + 1] - cu[r]), max(int(ctx[r]), 0)
        for first in range(c // block * block, c + n, block):
            at = first // page
            if at >= table.shape[1] or not 0 <= table[r, at] < bytes_.shape[0]:
                continue
            slots = [(i, int(cu[r]) + first + i - c) for i in range(block)
                     if c <= first + i < c + n]
            if not slots:
                continue
            rows = new[[t for _, t in slots]]
            around = error[[t for _, t in slots]]
            fine = np.isfinite(rows)
            size = np.where(fine, np.abs(np.where(fine, rows, 0)), 0)
            around = np.where(fine, around, 0)
            low = [scale_for(float((size - around)[:, h].max())) for h in range(rows.shape[1])]
            high = [scale_for(float((size + around)[:, h].max())) for h in range(rows.shape[1])]
            out.append((int(table[r, at]), first % page // block, max(c - first, 0), slots, low,
                        high))
    return out


def attention(q, k, v, v_scales, table, ctx, cu, masks, scale):
    """(out, lse, weight, reach, spread, flush) over caches k, v in 64 bits: as
    tree_reference.attention, and of each row also the largest scale * sum_d |k_d| times its
    largest |q|, and the largest weight times value scale times the sum of all elements seen,
    column by column."""
    T, Hq, D = q.shape
    group = Hq // k.shape[1]
    out, weight, flush = (np.zeros((T, Hq, D)) for _ in range(3))
    lse, reach, spread = np.full((T, Hq), -np.inf), np.zeros((T, Hq)), np.zeros((T, Hq))
    of_slots = np.repeat(v_scales, v.shape[2] // v_scales.shape[2], 2)[..., None]
    for r in range(len(cu) - 1):
        n, c = int(cu[r + 1] - cu[r]), int(ctx[r])
        if n == 0:
            continue
        kk, vv, bb = (ref.gather_cache(x, table[r], c + n) for x in (k, v, of_slots))
        rows = slice(int(cu[r]), int(cu[r + 1]))
        seen = np.zeros((n, c + n), bool)
        seen[:, :c] = True
        for i in range(min(n, 64 * masks.shape[1])):
            seen[:, c + i] = (masks[rows, i // 64] >> np.int64(i % 64)) & 1 != 0
        empty = ~seen.any(1)
        for h in range(Hq):
            x, at = q[rows, h].astype(np.float64), h // group
            with np.errstate(all="ignore"):
                s = np.where(seen, x @ kk[at].T * scale, -np.inf)
                top = np.where(empty, 0.0, s.max(1))
                p = np.where(seen, np.exp(s - top[:, None]), 0.0)
                total = np.where(empty, 1.0, p.sum(1))[:, None]
                sizes = np.abs(kk[at])
                some = seen.any(0)
                # what no row sees may be anything; what some row sees is held against those only
                values = np.where(some[:, None], vv[at], 0.0)
                scales = np.where(some, bb[at][:, 0], 0.0)
                bad = np.isnan(values).any(1)
                clean = np.where(bad[:, None], 0.0, values)
                o = p @ clean / total
                w = p @ np.abs(clean) / total
                by = np.abs(scales)[:, None]
                elements = np.where(by != 0, np.abs(clean) / by, 0)
                f = (p * np.abs(scales)).max(1, keepdims=True) * (seen @ elements) / total
                if bad.any():
                    touched = (seen & bad[None]).any(1)
                    o[touched] = (p[touched] @ values) / total[touched]
                out[rows, h], weight[rows, h], flush[rows, h] = o, w, f
                lse[rows, h] = np.where(empty, -np.inf, top + np.log(total[:, 0]))
                amounts = np.where(seen, np.abs(x) @ sizes.T, 0.0)
                reach[rows, h] = np.nanmax(amounts, 1) * abs(scale)
                spread[rows, h] = np.abs(x).max(1) * np.nanmax(
                    np.where(seen, sizes.sum(1)[None], 0.0), 1) * abs(scale)
    return out, lse, weight, reach, spread, flush


def commit(path, accepted, cu, ctx, table, bytes_, scales):
    """(bytes [layers, pages, ...], scales) after the moves, into copies."""
    out, out_scales = bytes_.copy(), scales.copy()
    layers, pages, heads, page, D = bytes_.shape
    block = page // scales.shape[3]

    def place(r, slot):
        at = slot // page
        number = int(table[r, at]) if at < table.shape[1] else -1
        return (number, slot % page) if 0 <= number < pages else None

    for r in range(len(cu) - 1):
        n, c = int(cu[r + 1] - cu[r]), int(ctx[r])
        kept = min(max(int(accepted[r]), 0), path.shape[1], n)
        if kept == 0:
            continue
        for first in range(c // block * block, c + kept, block):
            here = place(r, first)
            if here is None:
                continue
            rows, had = [], []
            for slot in range(first, min(first + block, c + kept)):
                source = place(r, slot)
                if slot >= c:
                    node = int(path[r, slot - c])
                    if slot - c < node < n:
                        source = place(r, c + node) or source
                rows.append(bytes_[:, source[0], :, source[1]])
                had.append(scales[:, source[0], :, source[1] // block])
            had = np.stack(had)                              # [slots, layers, heads]
            now = had.max(0)
            for i, x in enumerate(rows):
                factor = had[i] / now
                moved = np.where((factor == 1.0)[..., None], x,
                                 encode(VALUES[x] * factor[..., None]))
                out[:, here[0], :, here[1] + i] = moved
            out_scales[:, here[0], :, here[1] // block] = now
    return out, out_scales


def plan(table, ctx, source, want, pages, page_size, limit):
    """(next_table, next_ctx_lens, copies, counts) as lists and arrays."""
    B, M = table.shape
    N = len(source)
    rows, carried, writers = [], set(), {}
    for i in range(N):
        s = int(source[i]) if 0 <= source[i] < B else -1
        c = 0 if s < 0 else min(max(int(ctx[s]), 0), M * page_size)
        n = max(int(want[i]), 0)
        held = -(-c // page_size)
        need = min(-(-(c + n) // page_size), M)
        have = [int(table[s, e]) if 0 <= table[s, e] < pages else -1 for e in range(held)]
        written = held - 1 if n > 0 and c % page_size else -1
        for e, p in enumerate(have):
            if p >= 0 and e != written:
                carried.add(p)
            if p >= 0 and e == written:
                writers.setdefault(p, i)
        rows.append([c, have, need, written])
    used = carried | set(writers)
    free = [p for p in range(limit) if p not in used]
    moving = sorted(p for p in used if p >= limit)
    missing = max(len(moving) - len(free), 0)
    moved = dict(zip(moving, free))
    copies = [(p, moved[p]) for p in moving if p in moved]
    free = free[len(moving):]
    taken = 0
    out = np.full((N, M), -1, np.int32)

    def fresh():
        nonlocal taken, missing
        if taken < len(free):
            taken += 1
            return free[taken - 1]
        missing += 1
        return -1

    for i, (c, have, need, written) in enumerate(rows):
        for e, p in enumerate(have):
            if e == written and not (p >= 0 and p not in carried and writers[p] == i):
                to = fresh()
                if p >= 0 and to >= 0:
                    copies.append((p, to))
            else:
                to = moved.get(p, p)
            out[i, e] = to
        for e in range(len(have), need):
            out[i, e] = fresh()
    lens = np.array([r[0] for r in rows], np.int32)
    return out, lens, copies, [len(copies), len(used) + taken, missing]
