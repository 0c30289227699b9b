"""Plain 64-bit implementations of the tree-verification operators, on host
arrays, one token at a time, for the tests to compare with."""

import math

import numpy as np


def trees(rng, counts, roots=0.1, reach=6):
    """Random parents, packed: a node's parent is one of the `reach` nodes before it, or -1."""
    out = []
    for n in counts:
        for j in range(n):
            out.append(-1 if j == 0 or rng.random() < roots
                       else int(rng.integers(max(0, j - reach), j)))
    return np.array(out, dtype=np.int32)


def prefix(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def ancestors(parent):
    """For every node of one tree, the set of itself and its ancestors."""
    sets = []
    for j, p in enumerate(parent):
        sets.append({j} | (sets[p] if 0 <= p < j else set()))
    return sets


def tree_index(parent, cu, ctx_lens, words):
    positions = np.zeros(len(parent), dtype=np.int32)
    masks = np.zeros((len(parent), words), dtype=np.uint64)
    for r in range(len(cu) - 1):
        for j, s in enumerate(ancestors(parent[cu[r]:cu[r + 1]])):
            positions[cu[r] + j] = ctx_lens[r] + len(s) - 1
            for i in s:
                masks[cu[r] + j, i // 64] |= np.uint64(1 << (i % 64))
    return positions, masks.view(np.int64)


def tree_windows(ids, parent, cu, context, boundary):
    """[T, N] windows: the node's id, its ancestors' and the context's, the boundary id behind the first boundary."""
    N = context.shape[1] + 1
    out = np.zeros((len(ids), N), dtype=np.int64)
    for r in range(len(cu) - 1):
        for j in range(cu[r + 1] - cu[r]):
            line, at = [], j
            while at >= 0:
                line.append(int(ids[cu[r] + at]))
                p = parent[cu[r] + at]
                at = p if 0 <= p < at else -1
            line += [int(x) for x in context[r][::-1]]
            valid = True
            out[cu[r] + j, 0] = line[0]
            for s in range(1, N):
                valid = valid and line[s] != boundary
                out[cu[r] + j, s] = line[s] if valid else boundary
    return out


def tree_row_ids(ids, parent, cu, context, M, vocab, offsets, hpn, boundary):
    V = tree_windows(ids, parent, cu, context, boundary)
    L, N = M.shape
    out = np.zeros((L, len(ids), vocab.shape[1]), dtype=np.int64)
    wrap = 1 << 64
    for l in range(L):
        for t in range(len(ids)):
            mix = int(V[t, 0]) * int(M[l, 0]) % wrap
            for s in range(1, N):
                mix ^= int(V[t, s]) * int(M[l, s]) % wrap
                signed = mix - wrap if mix >= wrap // 2 else mix
                for h in range((s - 1) * hpn, s * hpn):
                    v = int(vocab[l, h])
                    row = (signed % v if v else 0) + int(offsets[l, h])
                    row %= wrap
                    out[l, t, h] = row - wrap if row >= wrap // 2 else row
    return out


def inverse_frequencies(R, base, scaling="plain", factor=1.0, trained=0.0, fast=32.0, slow=1.0):
    if scaling == "base" and R > 2:
        base = base * factor ** (R / (R - 2))
    out = []
    for i in range(R // 2):
        w = base ** (-2.0 * i / R)
        if scaling == "linear":
            w /= factor
        if scaling == "parts":
            g = min(max((trained * w / (2 * math.pi) - slow) / (fast - slow), 0.0), 1.0)
            w = g * w + (1 - g) * w / factor
        out.append(w)
    return np.array(out)


def norm_rope(x, weight, positions, w, eps, interleaved, scale):
    """(rows, bound): head rows x [T, H, D] in 64 bits and, for each element, |y_a| + |y_b| of its pair."""
    y = x.astype(np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    size = np.abs(y)
    R = 2 * len(w)
    if R:
        angle = positions.astype(np.float64)[:, None] * w
        c, s = np.cos(angle)[:, None] * scale, np.sin(angle)[:, None] * scale
        a = slice(0, R, 2) if interleaved else slice(0, R // 2)
        b = slice(1, R, 2) if interleaved else slice(R // 2, R)
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
        size[..., a] = size[..., b] = (np.abs(ya) + np.abs(yb)) * abs(scale)
    return y, size


def gather_cache(cache, table, length):
    """[heads, length, D] of one request from a paged cache [pages, heads, page_size, D]."""
    size = cache.shape[2]
    rows = [cache[table[i // size], :, i % size] for i in range(length)]
    return np.stack(rows, 1) if rows else np.zeros((cache.shape[1], 0, cache.shape[3]))


def attention(q, k_cache, v_cache, table, ctx_lens, cu, masks, scale):
    """(out, lse, weight, reach): also sum_j p_j |v_j| and the largest scale * sum |q_d k_d| of each row, from which the
    rounding errors of a 32-bit computation follow."""
    T, Hq, D = q.shape
    Hk = k_cache.shape[1]
    out, weight = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, reach = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for r in range(len(cu) - 1):
        n = cu[r + 1] - cu[r]
        if n == 0:
            continue
        k = gather_cache(k_cache, table[r], ctx_lens[r] + n).astype(np.float64)
        v = gather_cache(v_cache, table[r], ctx_lens[r] + n).astype(np.float64)
        for j in range(n):
            t = cu[r] + j
            seen = list(range(ctx_lens[r]))
            seen += [ctx_lens[r] + i for i in range(n)
                     if i < 64 * masks.shape[1] and (int(masks[t, i // 64]) >> (i % 64)) & 1]
            if not seen:
                continue
            for h in range(Hq):
                kk, vv = k[h // (Hq // Hk)][seen], v[h // (Hq // Hk)][seen]
                x = q[t, h].astype(np.float64)
                s = kk @ x * scale
                with np.errstate(invalid="ignore", over="ignore"):
                    top = s.max()
                    p = np.exp(s - top)
                    total = p.sum()
                    out[t, h] = (p[:, None] * vv).sum(0) / total
                    weight[t, h] = (p[:, None] * np.abs(vv)).sum(0) / total
                    lse[t, h] = top + np.log(total)
                    reach[t, h] = (np.abs(kk) @ np.abs(x)).max() * abs(scale)
    return out, lse, weight, reach


def commit(path, accepted, cu, ctx_lens, table, cache):
    """The cache [layers, pages, heads, page_size, D] after the moves, into a copy."""
    out, size = cache.copy(), cache.shape[3]
    for r in range(len(cu) - 1):
        n = cu[r + 1] - cu[r]
        for j in range(min(max(accepted[r], 0), path.shape[1], n)):
            node = path[r, j]
            if j < node < n:
                a, b = ctx_lens[r] + node, ctx_lens[r] + j
                out[:, table[r, b // size], :, b % size] = cache[:, table[r, a // size], :,
                                                                 a % size]
    return out


def next_context(ids, path, accepted, cu, context):
    out = np.zeros_like(context)
    C = context.shape[1]
    for r in range(len(cu) - 1):
        kept = min(max(accepted[r], 0), path.shape[1], cu[r + 1] - cu[r])
        line = list(context[r]) + [ids[cu[r] + path[r, j]] for j in range(kept)]
        out[r] = line[len(line) - C:]
    return out
