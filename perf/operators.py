"""The operators of a speculative verification step, as cases to be timed and compared.

A model with per-layer n-gram embeddings that verifies a tree of drafted tokens
in one step needs, next to the row ids of an ordinary batch:

  tree_index    positions and ancestor masks of the drafted trees
  tree_row_ids  the n-gram row ids of the nodes, each window along its branch
  qk_norm_rope  norms of queries and keys, the position rotation, and the append
                of keys and values to the paged cache, in one pass
  attention     the nodes' attention over the paged cache and their own branch
  commit        the accepted branch's keys and values moved together in the cache
                of every layer, with the next step's context and lengths

Each case is one call of one of them.  Where `own` is false, run() computes it
from elementary torch operations in 32 bits, rounded once at the end; where it
is true, it makes the calls that a user makes.
"""

import math
import random

import torch

own = False

VOCAB = 151936
BOUNDARY = 151643
EPS = 1e-6
ROPE_BASE = 1000000.0
TRAINED_POSITIONS = 32768  # the context that the rotation's scaling starts from
BETA_FAST, BETA_SLOW = 32.0, 1.0


# ------------------------------------------------------------------- the cases


def listed():
    return [
        # one user, a short chain of drafts: pure latency
        dict(name="index one chain", op="tree_index", requests=1, nodes_lo=4, nodes_hi=4, words=1),
        # a full serving batch of ragged trees, once per step
        dict(name="index 256 trees", op="tree_index", requests=256, nodes_lo=1, nodes_hi=127,
             words=2),
        # one user's tree through the smallest embedding (one layer, four heads)
        dict(name="row ids one tree", op="tree_row_ids", requests=1, nodes_lo=9, nodes_hi=9,
             ngram=3, hpn=2, layers=1, wide=True),
        # a full batch of trees, every one of 48 layers of 32 heads in one call
        dict(name="row ids 256 trees x 48", op="tree_row_ids", requests=256, nodes_lo=1,
             nodes_hi=63, ngram=5, hpn=8, layers=48, wide=True),
        # an ordinary decode step of one user
        dict(name="norm rope one token", op="qk_norm_rope", requests=1, nodes_lo=1, nodes_hi=1,
             ctx_lo=900, ctx_hi=900, q_heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, half=False, page=64, scaling=1.0),
        # ragged trees far into long contexts: scaled rotation of half of each head
        dict(name="norm rope 64 trees", op="qk_norm_rope", requests=64, nodes_lo=1, nodes_hi=33,
             ctx_lo=5, ctx_hi=120001, q_heads=64, kv_heads=8, dim=128, rotary=64,
             interleaved=True, half=True, page=16, scaling=4.0),
        # four prompts of thousands of tokens: bound by memory
        dict(name="norm rope prompts", op="qk_norm_rope", requests=4, nodes_lo=7001,
             nodes_hi=9001, ctx_lo=0, ctx_hi=1000, q_heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, half=False, page=64, scaling=1.0),
        # one user, one token, a short context: latency
        dict(name="attention one token", op="attention", requests=1, nodes_lo=1, nodes_hi=1,
             ctx_lo=701, ctx_hi=701, q_heads=32, kv_heads=8, dim=128, half=False, page=64),
        # one user's large tree over a very long context: 512 rows for each key head
        dict(name="attention long tree", op="attention", requests=1, nodes_lo=64, nodes_hi=64,
             ctx_lo=130981, ctx_hi=130981, q_heads=64, kv_heads=8, dim=128, half=True, page=64),
        # a serving batch, ragged in contexts and trees: bound by the cache's bytes
        dict(name="attention 32 ragged", op="attention", requests=32, nodes_lo=1, nodes_hi=32,
             ctx_lo=17, ctx_hi=32749, q_heads=32, kv_heads=8, dim=128, half=False, page=16),
        # one user's accepted branch in one layer's cache
        dict(name="commit one branch", op="commit", requests=1, nodes_lo=9, nodes_hi=9, ctx_lo=700,
             ctx_hi=700, accept_lo=3, accept_hi=3, kv_heads=8, dim=128, half=False, page=64,
             layers=1, ngram=3),
        # a batch's accepted branches in the caches of all 48 layers
        dict(name="commit 64 branches x 48", op="commit", requests=64, nodes_lo=12, nodes_hi=33,
             ctx_lo=20, ctx_hi=9000, accept_lo=1, accept_hi=9, kv_heads=8, dim=128, half=False,
             page=16, layers=48, ngram=5),
    ]


def log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree_index", "tree_row_ids", "qk_norm_rope", "attention", "attention",
                     "commit"])
    c = dict(op=op, requests=log_int(rng, 1, 256))
    if op == "tree_index":
        c["nodes_hi"] = log_int(rng, 1, 127)
        c["nodes_lo"] = rng.randint(0, c["nodes_hi"])
        c["words"] = (c["nodes_hi"] + 63) // 64
    elif op == "tree_row_ids":
        c["nodes_hi"] = log_int(rng, 1, 63)
        c["nodes_lo"] = rng.randint(0, c["nodes_hi"])
        c["ngram"], c["hpn"] = rng.choice([(2, 3), (3, 2), (3, 4), (4, 4), (5, 8), (4, 7)])
        c["layers"] = log_int(rng, 1, 48)
        c["wide"] = rng.random() < 0.6
    else:
        c["half"] = rng.random() < 0.4
        c["page"] = rng.choice([16, 32, 64, 128])
        c["dim"] = rng.choice([64, 128, 128])
        c["kv_heads"] = rng.choice([1, 2, 4, 8])
    if op == "qk_norm_rope":
        prompt = rng.random() < 0.4
        c["requests"] = log_int(rng, 1, 8 if prompt else 128)
        c["nodes_hi"] = log_int(rng, 16, 8000) if prompt else log_int(rng, 1, 64)
        c["nodes_lo"] = rng.randint(0, c["nodes_hi"])
        while c["requests"] * c["nodes_hi"] > 30000:
            c["requests"] -= 1
        c["ctx_hi"] = log_int(rng, 1, 120000)
        c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
        c["q_heads"] = c["kv_heads"] * rng.choice([1, 2, 4, 8])
        c["q_heads"] = min(c["q_heads"], 32)
        if (c["q_heads"] + 2 * c["kv_heads"]) * c["dim"] == 3072:
            c["q_heads"] //= 2
        c["rotary"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2, c["dim"] // 4])
        c["interleaved"] = rng.random() < 0.5
        c["scaling"] = rng.choice([1.0, 1.0, 4.0, 8.0])
    elif op == "attention":
        c["requests"] = log_int(rng, 1, 64)
        c["nodes_hi"] = log_int(rng, 1, 64)
        c["nodes_lo"] = rng.randint(0, c["nodes_hi"])
        c["q_heads"] = c["kv_heads"] * rng.choice([1, 2, 4, 5, 8])
        room = 32 * 32000 // c["requests"]  # the cache's size, then the scores'
        room = min(room, (1 << 29) // (c["requests"] * c["nodes_hi"] * c["q_heads"]), 131000)
        c["ctx_hi"] = log_int(rng, 1, max(1, room))
        c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
    elif op == "commit":
        c["requests"] = log_int(rng, 1, 64)
        c["nodes_hi"] = log_int(rng, 4, 33)
        c["nodes_lo"] = rng.randint(3, c["nodes_hi"])
        c["accept_hi"] = rng.randint(0, (c["nodes_lo"] - 1) // 2 + 1)
        c["accept_lo"] = rng.randint(0, c["accept_hi"])
        c["ctx_hi"] = log_int(rng, 1, 9000)
        c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
        c["layers"] = log_int(rng, 1, 48)
        c["ngram"] = rng.choice([2, 3, 4, 5])
    if c["nodes_hi"] and not c["nodes_lo"] and c["requests"] == 1:
        c["nodes_lo"] = c["nodes_hi"]
    return c


def spread(lo, hi, n):
    """n whole numbers from lo to hi at even steps (hi alone for n = 1): their order is drawn, their sum is not."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


# ------------------------------------------------------------------ the inputs


def prefix(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return cu


def draw_parents(rng, counts):
    """Trees in order: a node's parent is an earlier node of its request, or -1.  The first node is the token sampled last;
    drafts follow a few nodes behind their parents, and a few start at the context itself."""
    out = []
    for n in counts:
        for j in range(n):
            out.append(-1 if j == 0 or rng.random() < 0.04 else rng.randrange(max(0, j - 8), j))
    return out


def masks_of(parents, counts, words):
    """[T, words] int64: node i sees node j of its request where bit j is set (itself and its ancestors)."""
    rows, at = [], 0
    for n in counts:
        bits = []
        for j in range(n):
            p = parents[at + j]
            bits.append((bits[p] if p >= 0 else 0) | (1 << j))
        for b in bits:
            words_of = [(b >> (64 * w)) & (2 ** 64 - 1) for w in range(words)]
            rows.append([w - 2 ** 64 if w >= 2 ** 63 else w for w in words_of])
        at += n
    return torch.tensor(rows, dtype=torch.int64).reshape(-1, words)


def depths_of(parents, counts):
    out, at = [], 0
    for n in counts:
        d = []
        for j in range(n):
            p = parents[at + j]
            d.append(d[p] + 1 if p >= 0 else 0)
        out += d
        at += n
    return out


def inverse_frequencies(rotary, scaling):
    """[rotary / 2] float64: the rotation by parts for a context `scaling` times the trained one -- pairs that turn often keep
    their speed, pairs that turn less than once are slowed by `scaling`, and those between are mixed."""
    i = torch.arange(rotary // 2, dtype=torch.float64)
    inv = ROPE_BASE ** (-2.0 * i / rotary)
    if scaling == 1.0:
        return inv
    turns = TRAINED_POSITIONS * inv / (2.0 * math.pi)
    keep = ((turns - BETA_SLOW) / (BETA_FAST - BETA_SLOW)).clamp(0.0, 1.0)
    return inv * keep + inv / scaling * (1.0 - keep)


def rope_scale(scaling):
    return 1.0 if scaling == 1.0 else 0.1 * math.log(scaling) + 1.0


def lay_pages(rng, slots, counts, first, page):
    """A page table, int32 [B, most], over slots[r] cached tokens for each request: pages in drawn order.  Only pages that hold
    a slot at or behind first[r] get memory of their own where `first` is given (the step touches no other)."""
    most = max(1, max((-(-s // page) for s in slots), default=1))
    held = [[p for p in range(-(-s // page)) if first is None or (p + 1) * page > first[r]]
            for r, s in enumerate(slots)]
    # room that does not depend on how contexts and trees meet
    total = 1 + (sum(map(len, held)) if first is None else sum(n // page + 2 for n in counts))
    order = list(range(total))
    rng.shuffle(order)
    table, at = [[order[total - 1]] * most for _ in slots], 0
    for r, h in enumerate(held):
        for p in h:
            table[r][p] = order[at]
            at += 1
    return torch.tensor(table, dtype=torch.int32), total


def prepare(case, seed):
    c = case
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device="cuda", dtype=torch.int64)

    def put(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device="cuda")

    def shuffled(lo, hi):
        v = spread(lo, hi, c["requests"])
        rng.shuffle(v)
        return v

    s = dict(case=c)
    B = c["requests"]
    counts = shuffled(c["nodes_lo"], c["nodes_hi"])
    T = sum(counts)
    s["cu_seqlens"] = put(prefix(counts))
    s["tokens"], s["nodes_hi"] = T, c["nodes_hi"]
    ctx = None
    if "ctx_hi" in c:
        ctx = shuffled(c["ctx_lo"], c["ctx_hi"])
        s["ctx_lens"] = put(ctx)
    dtype = torch.float16 if c.get("half") else torch.bfloat16

    if c["op"] == "tree_index":
        s["parent"] = put(draw_parents(rng, counts))
        s["ctx_lens"] = whole(0, 131072, B).to(torch.int32)
    elif c["op"] == "tree_row_ids":
        s["parent"] = put(draw_parents(rng, counts))
        L, N, H = c["layers"], c["ngram"], (c["ngram"] - 1) * c["hpn"]
        kind = torch.int64 if c["wide"] else torch.int32

        def ids(*shape):
            v = whole(0, VOCAB, *shape)
            v[torch.rand(shape, generator=gen, device="cuda") < 0.05] = BOUNDARY
            return v.to(kind)

        s["ids"], s["ngram_context"] = ids(T), ids(B, N - 1)
        s["multipliers"] = whole(-2 ** 62, 2 ** 62, L, N) * 2 + 1
        s["vocab_sizes"] = whole(2 ** 16, 2 ** 22, L, H) | 1
        s["offsets"] = s["vocab_sizes"].cumsum(1) - s["vocab_sizes"]
    elif c["op"] == "qk_norm_rope":
        Hq, Hk, D = c["q_heads"], c["kv_heads"], c["dim"]
        # one product of the layer gives queries, keys and values side by side
        qkv = normal(T, Hq + 2 * Hk, D, dtype=dtype) * 3
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        s["q_weight"] = (1 + 0.2 * normal(D, dtype=torch.float32)).to(dtype)
        s["k_weight"] = (1 + 0.2 * normal(D, dtype=torch.float32)).to(dtype)
        if c["nodes_hi"] > 64:  # prompts: a chain each
            depth = [j for n in counts for j in range(n)]
        else:
            depth = depths_of(draw_parents(rng, counts), counts)
        start = [ctx[r] for r, n in enumerate(counts) for _ in range(n)]
        s["positions"] = put([a + d for a, d in zip(start, depth)])
        # the angle for each position, in 2**-64 turns
        s["rope"] = (inverse_frequencies(c["rotary"], c["scaling"]) / (2 * math.pi)
                     * 2.0 ** 64).to(torch.int64).cuda()
        table, pages = lay_pages(rng, [a + n for a, n in zip(ctx, counts)], counts, ctx,
                                 c["page"])
        s["page_table"] = table.cuda()
        s["k_cache"] = normal(pages, Hk, c["page"], D, dtype=dtype)
        s["v_cache"] = normal(pages, Hk, c["page"], D, dtype=dtype)
    elif c["op"] == "attention":
        Hq, Hk, D = c["q_heads"], c["kv_heads"], c["dim"]
        words = (c["nodes_hi"] + 63) // 64
        s["q"] = normal(T, Hq, D, dtype=dtype) * 1.5
        s["tree_mask"] = masks_of(draw_parents(rng, counts), counts, words).cuda()
        table, pages = lay_pages(rng, [a + n for a, n in zip(ctx, counts)], counts, None,
                                 c["page"])
        s["page_table"] = table.cuda()
        s["k_cache"] = normal(pages, Hk, c["page"], D, dtype=dtype)
        s["v_cache"] = normal(pages, Hk, c["page"], D, dtype=dtype)
    elif c["op"] == "commit":
        Hk, D, L = c["kv_heads"], c["dim"], c["layers"]
        accepted = shuffled(c["accept_lo"], c["accept_hi"])
        paths = []
        for n, a in zip(counts, accepted):
            # the sampled token is accepted first; a branch goes on behind its first sibling
            rest = sorted(rng.sample(range(2, n), max(0, a - 1)))
            paths.append(([0] + rest + [0] * c["accept_hi"])[:max(1, c["accept_hi"])])
        s["path"], s["accepted"] = put(paths), put(accepted)
        s["ids"] = whole(0, VOCAB, T)
        s["ngram_context"] = whole(0, VOCAB, B, c["ngram"] - 1)
        table, pages = lay_pages(rng, [a + n for a, n in zip(ctx, counts)], counts, ctx,
                                 c["page"])
        s["page_table"] = table.cuda()
        s["k_cache"] = normal(L, pages, Hk, c["page"], D, dtype=dtype)
        s["v_cache"] = normal(L, pages, Hk, c["page"], D, dtype=dtype)
    return s


# ------------------------------------------------------------------ the passes


def run(state):
    op = state["case"]["op"]
    if own:
        return OWN[op](state, state["case"])
    return PLAIN[op](state, state["case"])


def own_tree_index(s, c):
    import layer_gram_embedding_gb300 as ple

    return ple.ple_build_tree_index(s["parent"], s["cu_seqlens"], s["ctx_lens"], c["words"])


def own_tree_row_ids(s, c):
    import layer_gram_embedding_gb300 as ple

    return ple.ple_tree_row_ids(s["ids"], s["parent"], s["cu_seqlens"], s["ngram_context"],
                                s["multipliers"], s["vocab_sizes"], s["offsets"], c["ngram"],
                                c["hpn"], BOUNDARY)


def own_qk_norm_rope(s, c):
    import layer_gram_embedding_gb300 as ple

    q = ple.ple_qk_norm_rope(s["q"], s["k"], s["v"], s["positions"], s["rope"], s["q_weight"],
                             s["k_weight"], k_cache=s["k_cache"], v_cache=s["v_cache"],
                             page_table=s["page_table"], ctx_lens=s["ctx_lens"],
                             cu_seqlens=s["cu_seqlens"], eps=EPS, interleaved=c["interleaved"],
                             rope_scale=rope_scale(c["scaling"]))
    return q, s["k_cache"], s["v_cache"]


def own_attention(s, c):
    import layer_gram_embedding_gb300 as ple

    return ple.ple_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"],
                                  s["ctx_lens"], s["cu_seqlens"], s["tree_mask"],
                                  return_lse=True)


def own_commit(s, c):
    import layer_gram_embedding_gb300 as ple

    context, lens = ple.ple_tree_commit(s["ids"], s["path"], s["accepted"], s["cu_seqlens"],
                                        s["ngram_context"], s["ctx_lens"], s["page_table"],
                                        s["k_cache"], s["v_cache"])
    return s["k_cache"], s["v_cache"], context, lens


OWN = dict(tree_index=own_tree_index, tree_row_ids=own_tree_row_ids, qk_norm_rope=own_qk_norm_rope,
           attention=own_attention, commit=own_commit)


def owners(s):
    """Each token's request, and its place in it."""
    cu = s["cu_seqlens"].to(torch.int64)
    t = torch.arange(s["tokens"], device=cu.device)
    req = torch.searchsorted(cu[1:], t, right=True)
    return req, t - cu[req], cu


def plain_tree_index(s, c):
    req, local, cu = owners(s)
    B, n, W = c["requests"], s["nodes_hi"], c["words"]
    at = req * n + local
    jump = torch.full((B * n,), n, dtype=torch.int64, device=cu.device)
    jump[at] = torch.where(s["parent"] < 0, n, s["parent"].to(torch.int64))
    jump = torch.cat([jump.reshape(B, n), torch.full((B, 1), n, device=cu.device)], 1)
    # row n stands for "no parent" and sees nothing
    sees = torch.eye(n + 1, dtype=torch.bool, device=cu.device)[:, :n].repeat(B, 1, 1)
    for _ in range(max(1, n.bit_length())):  # twice as far up in each turn
        sees = sees | sees.gather(1, jump[:, :, None].expand(-1, -1, n))
        jump = jump.gather(1, jump)
    sees = sees[:, :n].reshape(B * n, n)[at]
    positions = s["ctx_lens"][req] + (sees.sum(1) - 1).to(torch.int32)
    sees = torch.nn.functional.pad(sees, (0, 64 * W - n)).reshape(-1, W, 64).to(torch.int64)
    return positions, (sees << torch.arange(64, device=cu.device)).sum(2)


def plain_tree_row_ids(s, c):
    req, local, cu = owners(s)
    N, hpn = c["ngram"], c["hpn"]
    ids, ctx = s["ids"].to(torch.int64), s["ngram_context"].to(torch.int64)
    parent = s["parent"].to(torch.int64)
    first = cu[req]
    at, valid = local, torch.ones_like(local, dtype=torch.bool)
    back = torch.full_like(local, N - 1)  # the context id read last
    mix = ids * s["multipliers"][:, :1]
    out = []
    for k in range(1, N):
        # one node up its branch, or one id back in the context behind its root
        up = torch.where(at >= 0, parent[first + at.clamp(min=0)], at)
        back = torch.where(up < 0, back - 1, back)
        word = torch.where(up >= 0, ids[first + up.clamp(min=0)],
                           ctx[req, back.clamp(0, N - 2)])
        at = up
        valid = valid & (word != BOUNDARY)
        mix = mix ^ (torch.where(valid, word, BOUNDARY) * s["multipliers"][:, k:k + 1])
        h = slice((k - 1) * hpn, k * hpn)
        out.append(torch.remainder(mix[:, :, None], s["vocab_sizes"][:, None, h])
                   + s["offsets"][:, None, h])
    return torch.cat(out, 2)


def plain_qk_norm_rope(s, c):
    R, dtype = c["rotary"], s["q"].dtype
    angle = s["positions"].float()[:, None] * (s["rope"].float() * (2 * math.pi / 2.0 ** 64))
    cos = (angle.cos() * rope_scale(c["scaling"]))[:, None]
    sin = (angle.sin() * rope_scale(c["scaling"]))[:, None]

    def one(x, weight):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + EPS) * weight.float()
        if c["interleaved"]:
            a, b = x[..., 0:R:2], x[..., 1:R:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
        else:
            a, b = x[..., :R // 2], x[..., R // 2:R]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
        return torch.cat([turned, x[..., R:]], 2).to(dtype)

    req, local, _ = owners(s)
    slot = s["ctx_lens"][req] + local
    page = s["page_table"][req, slot // c["page"]].to(torch.int64)
    s["k_cache"][page, :, slot % c["page"]] = one(s["k"], s["k_weight"])
    s["v_cache"][page, :, slot % c["page"]] = s["v"]
    return one(s["q"], s["q_weight"]), s["k_cache"], s["v_cache"]


def plain_attention(s, c):
    Hq, Hk, D = c["q_heads"], c["kv_heads"], c["dim"]
    B, n, G = c["requests"], s["nodes_hi"], c["q_heads"] // c["kv_heads"]
    req, local, cu = owners(s)
    S = s["page_table"].shape[1] * c["page"]
    pages = s["page_table"].to(torch.int64)

    def cached(x):
        return x[pages].permute(0, 2, 1, 3, 4).reshape(B, Hk, S, D).float()

    q = torch.zeros(B, n, Hk, G, D, device=cu.device)
    q[req, local] = s["q"].float().reshape(-1, Hk, G, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, Hk, n * G, D)
    # a slot is seen where it is of the context, or of a node in the mask
    place = torch.arange(S, device=cu.device) - s["ctx_lens"].to(torch.int64)[:, None]
    word = (place.clamp(min=0) // 64).clamp(max=s["tree_mask"].shape[1] - 1)
    mask = torch.zeros(B, n, s["tree_mask"].shape[1], dtype=torch.int64, device=cu.device)
    mask[req, local] = s["tree_mask"]
    bit = (mask.gather(2, word[:, None].expand(-1, n, -1)) >> (place % 64)[:, None]) & 1
    tree = (place[:, None] >= 0) & (place[:, None] < n) & (bit != 0)
    sees = ((place < 0)[:, None] | tree)[:, None, :, None].expand(B, Hk, n, G, S)
    held = place < (cu[1:] - cu[:-1])[:, None]
    score = (q @ cached(s["k_cache"]).transpose(2, 3)) * (1 / math.sqrt(D))
    score = score.masked_fill(~sees.reshape(B, Hk, n * G, S), -math.inf)
    top = score.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    weight = (score - top).exp()
    total = weight.sum(3, keepdim=True)
    values = cached(s["v_cache"]).masked_fill(~held[:, None, :, None], 0.0)
    out = (weight @ values) / torch.where(total == 0, 1.0, total)
    out = out.reshape(B, Hk, n, G, D).permute(0, 2, 1, 3, 4)[req, local]
    lse = (total.log() + top).reshape(B, Hk, n, G).permute(0, 2, 1, 3)[req, local]
    return out.reshape(-1, Hq, D).to(s["q"].dtype), lse.reshape(-1, Hq)


def plain_commit(s, c):
    N, page = c["ngram"], c["page"]
    cu = s["cu_seqlens"].to(torch.int64)
    path, accepted = s["path"].to(torch.int64), s["accepted"].to(torch.int64)
    ctx, pages = s["ctx_lens"].to(torch.int64), s["page_table"].to(torch.int64)
    P = path.shape[1]
    step = torch.arange(P, device=cu.device)
    keep = step < accepted[:, None]
    # what is not accepted moves onto itself
    to = ctx[:, None] + torch.where(keep, step, 0)
    source = ctx[:, None] + torch.where(keep, path, 0)
    held = (cu[1:] > cu[:-1])[:, None] & keep
    to, source = torch.where(held, to, 0), torch.where(held, source, 0)
    a, b = pages.gather(1, source // page).flatten(), (source % page).flatten()
    x, y = pages.gather(1, to // page).flatten(), (to % page).flatten()
    some = held.flatten()
    for cache in (s["k_cache"], s["v_cache"]):
        moved = cache[:, a, :, b]
        cache[:, x, :, y] = torch.where(some[:, None, None, None], moved, cache[:, x, :, y])
    # the last N - 1 ids of the context followed by the accepted ones
    ids = s["ids"][(cu[:-1, None] + path).clamp(max=s["tokens"] - 1)]
    line = torch.cat([s["ngram_context"], ids], 1)
    context = line.gather(1, accepted[:, None] + torch.arange(N - 1, device=cu.device))
    return s["k_cache"], s["v_cache"], context, (ctx + accepted).to(torch.int32)


PLAIN = dict(tree_index=plain_tree_index, tree_row_ids=plain_tree_row_ids,
             qk_norm_rope=plain_qk_norm_rope, attention=plain_attention, commit=plain_commit)


# --------------------------------------------------------- the work and 64 bits


def work(case):
    c = case
    B = c["requests"]
    T = sum(spread(c["nodes_lo"], c["nodes_hi"], B))
    if c["op"] == "tree_index":
        return dict(bytes=4 * (2 * B + 1) + T * (4 + 4 + 8 * c["words"]), flops=0)
    if c["op"] == "tree_row_ids":
        size, L, N, H = 8 if c["wide"] else 4, c["layers"], c["ngram"], (c["ngram"] - 1) * c["hpn"]
        return dict(bytes=T * (size + 4) + 4 * (B + 1) + B * (N - 1) * size + 8 * L * (N + 2 * H)
                    + 8 * L * T * H, flops=0)
    Hk, D = c["kv_heads"], c["dim"]
    if c["op"] == "qk_norm_rope":
        Hq = c["q_heads"]
        return dict(bytes=T * (Hq + 2 * Hk) * D * 2 * 2 + T * 4 + 8 * B + 4 * c["rotary"] + 4 * D,
                    flops=T * (Hq + Hk) * (4 * D + 3 * c["rotary"]))
    if c["op"] == "attention":
        Hq = c["q_heads"]
        # which tree meets which context is drawn: the products go by the means
        slots = T + sum(spread(c["ctx_lo"], c["ctx_hi"], B))
        return dict(bytes=slots * Hk * D * 2 * 2 + T * Hq * (D * 2 * 2 + 4) + 8 * T + 12 * B,
                    flops=4 * D * Hq * T * slots / B)
    moved = sum(max(0, a - 1) for a in spread(c["accept_lo"], c["accept_hi"], B))
    return dict(bytes=moved * c["layers"] * Hk * D * 2 * 2 * 2 + B * (16 * (c["ngram"] - 1) + 16)
                + 8 * moved, flops=0)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    cu = s["cu_seqlens"].tolist()
    ctx = s["ctx_lens"].tolist() if "ctx_hi" in c else None
    table = s["page_table"].tolist() if "page_table" in s else None
    if c["op"] == "qk_norm_rope":
        return exact_qk_norm_rope(s, c, cu, ctx, table)
    if c["op"] == "attention":
        return exact_attention(s, c, cu, ctx, table)
    if c["op"] == "commit":
        kc, vc = s["k_cache"], s["v_cache"]
        for r, a in enumerate(s["accepted"].tolist()):
            for j, node in enumerate(s["path"][r].tolist()[:a]):
                i, o = ctx[r] + node, ctx[r] + j
                for x in (kc, vc):
                    x[:, table[r][o // c["page"]], :, o % c["page"]] = x[
                        :, table[r][i // c["page"]], :, i % c["page"]]
        return kc.double(), vc.double(), None, None
    return None


def exact_qk_norm_rope(s, c, cu, ctx, table):
    R = c["rotary"]
    inv = inverse_frequencies(R, c["scaling"]).cuda()
    turn = torch.polar(torch.full((s["tokens"], R // 2), rope_scale(c["scaling"]),
                                  dtype=torch.float64, device="cuda"),
                       s["positions"].double()[:, None] * inv)

    def one(x, weight):
        x = x.double()
        x = x / (x.square().mean(2, keepdim=True) + EPS).sqrt() * weight.double()
        # a pair is a number of the complex plane
        if c["interleaved"]:
            z = torch.view_as_complex(x[..., :R].reshape(*x.shape[:2], R // 2, 2).contiguous())
            x[..., :R] = torch.view_as_real(z * turn[:, None]).reshape(*x.shape[:2], R)
        else:
            z = torch.complex(x[..., :R // 2], x[..., R // 2:R]) * turn[:, None]
            x[..., :R // 2], x[..., R // 2:R] = z.real, z.imag
        return x

    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    k, v = one(s["k"], s["k_weight"]), s["v"].double()
    for r in range(c["requests"]):
        slot = ctx[r]
        while slot < ctx[r] + cu[r + 1] - cu[r]:  # page by page
            at, end = slot % c["page"], min(ctx[r] + cu[r + 1] - cu[r],
                                            (slot // c["page"] + 1) * c["page"])
            t, p = cu[r] + slot - ctx[r], table[r][slot // c["page"]]
            kc[p, :, at:at + end - slot] = k[t:t + end - slot].transpose(0, 1)
            vc[p, :, at:at + end - slot] = v[t:t + end - slot].transpose(0, 1)
            slot = end
    return one(s["q"], s["q_weight"]), kc, vc


def exact_attention(s, c, cu, ctx, table):
    Hq, Hk, D = c["q_heads"], c["kv_heads"], c["dim"]
    if work(c)["flops"] > 6e11:
        return None
    out = torch.zeros(s["tokens"], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["tokens"], Hq, dtype=torch.float64, device="cuda")
    for r in range(c["requests"]):
        n, length = cu[r + 1] - cu[r], ctx[r] + cu[r + 1] - cu[r]
        if n == 0:
            continue
        pages = torch.tensor(table[r][:-(-length // c["page"])], device="cuda")
        sees = torch.ones(n, length, dtype=torch.bool, device="cuda")
        bits = s["tree_mask"][cu[r]:cu[r + 1]].tolist()
        sees[:, ctx[r]:] = torch.tensor([[bool((row[j // 64] >> (j % 64)) & 1) for j in range(n)]
                                         for row in bits], device="cuda")
        for h in range(Hq):  # head by head
            kv = h // (Hq // Hk)
            k = s["k_cache"][pages, kv].reshape(-1, D)[:length].double()
            v = s["v_cache"][pages, kv].reshape(-1, D)[:length].double()
            score = s["q"][cu[r]:cu[r + 1], h].double() @ k.T / math.sqrt(D)
            score[~sees] = -math.inf
            lse[cu[r]:cu[r + 1], h] = torch.logsumexp(score, 1)
            out[cu[r]:cu[r + 1], h] = torch.softmax(score, 1) @ v
    return out, lse
