"""The operators of a key and value cache held in 8 bits, and of its pages, as cases to be timed and compared.

A server whose contexts outgrow the 16-bit cache keeps keys and values as 8-bit floats (e4m3) with one scale, a power of two, for
each block of tokens and head, and moves whole pages when requests fork, end or are packed together:

  append     norms of queries and keys, the position rotation, and the append of keys and values in 8 bits to the paged cache
  attention  the drafted nodes' attention over that cache and their own branch
  commit     the accepted branch's keys and values moved together in the cache of every layer, from block to block
  plan       the next step's page tables: requests that go on, fork, end or begin, and pages packed below a limit
  copy       the pages that such a plan moves or doubles, in the caches of every layer

Each case is one call of one of them.  Where `own` is false, run() computes it from elementary torch operations in 32 bits, rounded
once at the end; where it is true, it makes the calls that a user makes.  Caches in 8 bits are returned as the values that they
stand for: element times scale, exact in bfloat16.
"""

import math
import random

import torch

own = False

EPS = 1e-6
ROPE_BASE = 1000000.0
VOCAB = 151936
ELEMENT = torch.float8_e4m3fn
LARGEST = 448.0  # of an element
LEAST_EXPONENT = -100  # of a scale


# ------------------------------------------------------------------- the cases


def listed():
    return [
        # an ordinary decode step of one user
        dict(name="append one token", op="append", requests=1, nodes_lo=1, nodes_hi=1, ctx_lo=900, ctx_hi=900, q_heads=32,
             kv_heads=8, dim=128, rotary=128, interleaved=False, half=False, page=64, block=16),
        # four prompts of thousands of tokens: bound by memory
        dict(name="append prompts", op="append", requests=4, nodes_lo=7001, nodes_hi=9001, ctx_lo=0, ctx_hi=1000, q_heads=32,
             kv_heads=8, dim=128, rotary=128, interleaved=False, half=False, page=64, block=16),
        # one user, one token, a short context: latency
        dict(name="attention one token", op="attention", requests=1, nodes_lo=1, nodes_hi=1, ctx_lo=701, ctx_hi=701, q_heads=32,
             kv_heads=8, dim=128, half=False, page=64, block=16),
        # a full batch of plain decodes: bound by the cache's bytes
        dict(name="attention 64 decodes", op="attention", requests=64, nodes_lo=1, nodes_hi=1, ctx_lo=257, ctx_hi=16385,
             q_heads=32, kv_heads=8, dim=128, half=False, page=64, block=64),
        # a serving batch, ragged in contexts and trees
        dict(name="attention 32 ragged", op="attention", requests=32, nodes_lo=1, nodes_hi=32, ctx_lo=17, ctx_hi=32749,
             q_heads=32, kv_heads=8, dim=128, half=False, page=16, block=16),
        # one user's large tree over a very long context: 512 rows for each key head
        dict(name="attention long tree", op="attention", requests=1, nodes_lo=64, nodes_hi=64, ctx_lo=130981, ctx_hi=130981,
             q_heads=64, kv_heads=8, dim=128, half=True, page=64, block=32),
        # one user's accepted branch in one layer's cache
        dict(name="commit one branch", op="commit", requests=1, nodes_lo=9, nodes_hi=9, ctx_lo=700, ctx_hi=700, accept_lo=3,
             accept_hi=3, kv_heads=8, dim=128, page=64, block=16, layers=1, ngram=3),
        # a batch's accepted branches in the caches of 16 layers
        dict(name="commit 64 branches x 16", op="commit", requests=64, nodes_lo=12, nodes_hi=33, ctx_lo=20, ctx_hi=9000,
             accept_lo=1, accept_hi=9, kv_heads=8, dim=128, page=16, block=16, layers=16, ngram=5),
        # one user's four continuations of one prompt
        dict(name="plan one prompt, four ways", op="plan", requests=1, rows=4, ctx_lo=1001, ctx_hi=1001, want_hi=9, page=16,
             spare=64, shrink=0.0, ended=0.0, forked=1.0),
        # a full batch in long contexts: some end, some fork, new ones begin, and the pool shrinks by a third
        dict(name="plan 256 requests", op="plan", requests=256, rows=256, ctx_lo=17, ctx_hi=32749, want_hi=64, page=64,
             spare=80000, shrink=0.33, ended=0.2, forked=0.2),
        # one doubled page in one layer of a 16-bit cache
        dict(name="copy one page", op="copy", copies=1, kv_heads=8, dim=128, page=64, block=16, layers=1, bits=16),
        # a batch's forked and packed pages, all layers
        dict(name="copy 97 pages x 48", op="copy", copies=97, kv_heads=8, dim=128, page=64, block=16, layers=48, bits=16),
    ]


def log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attention", "attention", "attention", "commit", "plan", "copy"])
    c = dict(op=op)
    if op == "plan":
        c["requests"] = log_int(rng, 1, 256)
        c["rows"] = log_int(rng, 1, 256)
        c["page"] = rng.choice([16, 32, 64, 128])
        c["ctx_hi"] = log_int(rng, 1, min(120000, 100000 * c["page"] // c["requests"]))
        c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
        c["want_hi"] = log_int(rng, 1, 600)
        c["spare"] = c["rows"] * (2 + c["want_hi"] // c["page"]) + log_int(rng, 1, 40000)
        c["shrink"] = rng.choice([0.0, 0.0, rng.uniform(0.0, 0.6)])
        c["ended"], c["forked"] = rng.uniform(0.0, 0.4), rng.uniform(0.0, 0.5)
        return c
    c["page"] = rng.choice([16, 32, 64, 128])
    c["block"] = rng.choice([b for b in (16, 16, 32, 64, 128) if b <= c["page"]])
    c["dim"] = rng.choice([64, 96, 128, 128, 128, 256])
    c["kv_heads"] = rng.choice([1, 2, 4, 8])
    if op == "copy":
        c["bits"] = rng.choice([8, 16])
        c["copies"] = log_int(rng, 1, 97 if c["bits"] == 16 else 16)
        c["layers"] = log_int(rng, 1, 48 if c["bits"] == 16 else 8)
        return c
    c["requests"] = log_int(rng, 1, 64)
    if op == "append":
        prompt = rng.random() < 0.5
        c["requests"] = log_int(rng, 1, 8 if prompt else 128)
        c["nodes_hi"] = log_int(rng, 16, 8000) if prompt else log_int(rng, 1, 64)
        c["nodes_lo"] = rng.randint(0, c["nodes_hi"])
        while c["requests"] * c["nodes_hi"] > 30000:
            c["requests"] -= 1
        c["ctx_hi"] = log_int(rng, 1, 120000)
        c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
        c["q_heads"] = min(c["kv_heads"] * rng.choice([1, 2, 4, 8]), 32)
        c["rotary"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2])
        c["interleaved"] = rng.random() < 0.5
        c["half"] = rng.random() < 0.4
    elif op == "attention":
        c["nodes_hi"] = rng.choice([1, log_int(rng, 1, 64)])
        c["nodes_lo"] = rng.randint(0, c["nodes_hi"])
        c["half"] = rng.random() < 0.4
        c["q_heads"] = c["kv_heads"] * rng.choice([1, 2, 4, 5, 8])
        room = 32 * 32000 // c["requests"] * 128 // max(128, c["dim"])  # the cache's size, then the scores'
        room = min(room, (1 << 29) // (c["requests"] * c["nodes_hi"] * c["q_heads"]), 131000)
        c["ctx_hi"] = log_int(rng, 1, max(1, room))
        c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
    else:
        c["nodes_hi"] = log_int(rng, 4, 33)
        c["nodes_lo"] = rng.randint(3, c["nodes_hi"])
        c["accept_hi"] = rng.randint(0, (c["nodes_lo"] - 1) // 2 + 1)
        c["accept_lo"] = rng.randint(0, c["accept_hi"])
        c["ctx_hi"] = log_int(rng, 1, 9000)
        c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
        c["layers"] = log_int(rng, 1, 16)
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
    """Trees in order: a node's parent is an earlier node of its request, or -1."""
    return [-1 if j == 0 or rng.random() < 0.04 else rng.randrange(max(0, j - 8), j) for n in counts for j in range(n)]


def masks_of(parents, counts):
    """[T, 1] int64: node i sees node j of its request where bit j is set (itself and its ancestors)."""
    rows, at = [], 0
    for n in counts:
        bits = []
        for j in range(n):
            p = parents[at + j]
            bits.append((bits[p] if p >= 0 else 0) | (1 << j))
        rows += [b - 2 ** 64 if b >= 2 ** 63 else b for b in bits]
        at += n
    return torch.tensor(rows, dtype=torch.int64).reshape(-1, 1)


def lay_pages(rng, slots, counts, first, page):
    """A page table, int32 [B, most], over slots[r] cached tokens for each request: pages in drawn order.  Only pages that hold
    a slot at or behind first[r] get memory of their own where `first` is given (the step touches no other)."""
    most = max(1, max((-(-s // page) for s in slots), default=1))
    held = [[p for p in range(-(-s // page)) if first is None or (p + 1) * page > first[r]] for r, s in enumerate(slots)]
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

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device="cuda", dtype=torch.int64)

    def put(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device="cuda")

    def cache8(*shape):
        """Keys and values in one tensor [2, ...] and their scales: values of about 1, a few binades apart from block to block."""
        kv = torch.empty(2, *shape, device="cuda", dtype=ELEMENT)
        parts = kv.view(-1, *shape[-4:])
        for i in range(parts.shape[0]):
            parts[i] = (normal(*shape[-4:], dtype=torch.bfloat16) * 64).clamp(-LARGEST, LARGEST).to(ELEMENT)
        scale = torch.exp2(whole(-8, -5, 2, *shape[:-2], shape[-2] // c["block"]).float()).to(torch.bfloat16)
        s["kv"], s["kv_scale"] = kv, scale
        s["k_cache"], s["v_cache"] = kv[0], kv[1]
        s["k_scale"], s["v_scale"] = scale[0], scale[1]

    s = dict(case=c)
    if c["op"] == "plan":
        return prepare_plan(c, rng, s, put)
    if c["op"] == "copy":
        L, P, shape = c["layers"], 2 * c["copies"] + 3, (c["kv_heads"], c["page"], c["dim"])
        if c["bits"] == 8:
            cache8(L, P, *shape)
        else:
            s["k_cache"], s["v_cache"] = (normal(L, P, *shape, dtype=torch.bfloat16) for _ in range(2))
        order = list(range(P))
        rng.shuffle(order)
        n = c["copies"]
        # the last places are not in use
        s["copies"] = put([[order[i], order[n + i]] for i in range(n)] + [[-1, -1]] * 2)
        return s

    B = c["requests"]

    def shuffled(lo, hi):
        v = spread(lo, hi, B)
        rng.shuffle(v)
        return v

    counts, ctx = shuffled(c["nodes_lo"], c["nodes_hi"]), shuffled(c["ctx_lo"], c["ctx_hi"])
    T = sum(counts)
    s["cu_seqlens"], s["ctx_lens"] = put(prefix(counts)), put(ctx)
    s["tokens"], s["nodes_hi"] = T, c["nodes_hi"]
    dtype = torch.float16 if c.get("half") else torch.bfloat16
    first = None
    if c["op"] != "attention":  # memory for the pages that the call touches: from the block that it goes on with
        first = [a // c["block"] * c["block"] for a in ctx]
    table, pages = lay_pages(rng, [a + n for a, n in zip(ctx, counts)], counts, first, c["page"])
    s["page_table"] = table.cuda()
    Hk, D = c["kv_heads"], c["dim"]

    if c["op"] == "append":
        Hq = c["q_heads"]
        # one product of the layer gives queries, keys and values side by side
        qkv = normal(T, Hq + 2 * Hk, D, dtype=dtype) * 3
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        s["q_weight"] = (1 + 0.2 * normal(D)).to(dtype)
        s["k_weight"] = (1 + 0.2 * normal(D)).to(dtype)
        depth = [j for n in counts for j in range(n)]
        start = [ctx[r] for r, n in enumerate(counts) for _ in range(n)]
        s["positions"] = put([a + d for a, d in zip(start, depth)])
        # the angle for each position, in 2**-64 turns
        i = torch.arange(c["rotary"] // 2, dtype=torch.float64)
        s["rope"] = (ROPE_BASE ** (-2.0 * i / c["rotary"]) / (2 * math.pi) * 2.0 ** 64).to(torch.int64).cuda()
        cache8(pages, Hk, c["page"], D)
    elif c["op"] == "attention":
        s["q"] = normal(T, c["q_heads"], D, dtype=dtype) * 1.5
        s["tree_mask"] = masks_of(draw_parents(rng, counts), counts).cuda()
        cache8(pages, Hk, c["page"], D)
    else:
        accepted = shuffled(c["accept_lo"], c["accept_hi"])
        paths = []
        for n, a in zip(counts, accepted):
            # the sampled token is accepted first; a branch goes on behind its first sibling
            rest = sorted(rng.sample(range(2, n), max(0, a - 1)))
            paths.append(([0] + rest + [0] * c["accept_hi"])[:max(1, c["accept_hi"])])
        s["path"], s["accepted"] = put(paths), put(accepted)
        s["ids"] = whole(0, VOCAB, T)
        s["ngram_context"] = whole(0, VOCAB, B, c["ngram"] - 1)
        cache8(c["layers"], pages, Hk, c["page"], D)
    return s


def prepare_plan(c, rng, s, put):
    """Requests over pages in drawn order; some share the front of another's pages, as forked ones do."""
    B, N, page = c["requests"], c["rows"], c["page"]
    ctx = spread(c["ctx_lo"], c["ctx_hi"], B)
    rng.shuffle(ctx)
    most = -(-(c["ctx_hi"] + c["want_hi"]) // page)
    pages = sum(-(-n // page) for n in ctx) + c["spare"]
    order = list(range(pages))
    rng.shuffle(order)
    table, at = [], 0
    for r in range(B):
        held, shared = -(-ctx[r] // page), 0
        if r and rng.random() < 0.3:
            other = rng.randrange(r)
            shared = min(ctx[r], ctx[other]) // page  # whole pages
        table.append(table[other][:shared] if shared else [])
        table[r] += order[at:at + held - shared] + [-1] * (most - held)
        at += held - shared
    source, left = [], list(range(B))
    rng.shuffle(left)
    for _ in range(N):
        u = rng.random()
        if u < c["forked"]:
            source.append(rng.randrange(B))
        elif u < c["forked"] + c["ended"] or not left:
            source.append(-1)
        else:
            source.append(left.pop())
    want = spread(0, c["want_hi"], N)
    rng.shuffle(want)
    s["page_table"], s["ctx_lens"] = put(table), put(ctx)
    s["source"], s["want"] = put(source), put(want)
    s["pages"], s["limit"] = pages, pages - int(pages * c["shrink"])
    return s


# ------------------------------------------------------------------ the passes


def run(state):
    op = state["case"]["op"]
    if own:
        return OWN[op](state, state["case"])
    return PLAIN[op](state, state["case"])


def values(s):
    """What the 8-bit cache stands for: keys and values [2, ..., slots, dim]."""
    blocks = s["kv"].to(torch.bfloat16).unflatten(-2, (-1, s["case"]["block"]))
    return blocks.mul_(s["kv_scale"][..., None, None]).flatten(-3, -2)


def own_append(s, c):
    import layer_gram_embedding_gb300 as ple

    q = ple.ple_qk_norm_rope_fp8(s["q"], s["k"], s["v"], s["positions"], s["rope"], s["q_weight"], s["k_weight"], s["k_cache"],
                                 s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"], s["ctx_lens"], s["cu_seqlens"],
                                 eps=EPS, interleaved=c["interleaved"])
    return q, values(s)


def own_attention(s, c):
    import layer_gram_embedding_gb300 as ple

    return ple.ple_tree_attention_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"],
                                      s["ctx_lens"], s["cu_seqlens"], s["tree_mask"], return_lse=True)


def own_commit(s, c):
    import layer_gram_embedding_gb300 as ple

    context, lens = ple.ple_tree_commit_fp8(s["ids"], s["path"], s["accepted"], s["cu_seqlens"], s["ngram_context"],
                                            s["ctx_lens"], s["page_table"], s["k_cache"], s["v_cache"], s["k_scale"],
                                            s["v_scale"])
    return values(s), context, lens


def own_plan(s, c):
    import layer_gram_embedding_gb300 as ple

    return ple.ple_plan_pages(s["page_table"], s["ctx_lens"], s["source"], s["want"], s["pages"], c["page"], limit=s["limit"])


def own_copy(s, c):
    import layer_gram_embedding_gb300 as ple

    if c["bits"] == 8:
        ple.ple_copy_pages(s["copies"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        return values(s)
    ple.ple_copy_pages(s["copies"], s["k_cache"], s["v_cache"])
    return s["k_cache"], s["v_cache"]


OWN = dict(append=own_append, attention=own_attention, commit=own_commit, plan=own_plan, copy=own_copy)


def owners(s):
    """Each token's request, and its place in it."""
    cu = s["cu_seqlens"].to(torch.int64)
    t = torch.arange(s["tokens"], device=cu.device)
    req = torch.searchsorted(cu[1:], t, right=True)
    return req, t - cu[req], cu


def exponent_for(most):
    """The least exponent of two that takes values up to `most` to at most the largest element."""
    m, e = torch.frexp(most)
    e = torch.where(m > 0.875, e - 8, e - 9)  # 448 = 0.875 * 2**9
    return torch.where(most > 0, e, LEAST_EXPONENT).clamp(min=LEAST_EXPONENT)


def plain_append(s, c):
    R, D, size, page, dtype = c["rotary"], c["dim"], c["block"], c["page"], s["q"].dtype
    # whole turns of a far position are lost in 64 bits of a wrapping product, not in 32 of a float
    turn = (s["positions"].to(torch.int64)[:, None] * s["rope"]).double() * 2.0 ** -64
    cos = (turn * (2 * math.pi)).cos().float()[:, None]
    sin = (turn * (2 * math.pi)).sin().float()[:, None]

    def one(x, weight):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + EPS) * weight.float()
        if c["interleaved"]:
            a, b = x[..., 0:R:2], x[..., 1:R:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
        else:
            a, b = x[..., :R // 2], x[..., R // 2:R]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
        return torch.cat([turned, x[..., R:]], 2)

    req, local, cu = owners(s)
    slot = s["ctx_lens"].to(torch.int64)[req] + local
    # the blocks that tokens go to, one row a block: a request's blocks follow each other
    n, first = cu[1:] - cu[:-1], s["ctx_lens"].to(torch.int64)
    blocks = torch.where(n > 0, (first + n - 1) // size - first // size + 1, 0)
    start = blocks.cumsum(0) - blocks
    row = start[req] + slot // size - first[req] // size
    rows = c["requests"] * 2 + s["tokens"] // size  # room that no sizes on the device decide
    pages = s["page_table"].to(torch.int64)
    at = torch.zeros(rows, dtype=torch.int64, device=row.device)  # a block's place among the cache's
    at[row] = pages[req, slot // page] * (page // size) + slot % page // size
    old = torch.zeros(rows, dtype=torch.int64, device=row.device)  # tokens that it holds already
    old[row] = (first[req] - slot // size * size).clamp(0, size)
    used = torch.zeros(rows, dtype=torch.bool, device=row.device)
    used[row] = True
    place = torch.arange(size, device=row.device)
    P, H = s["k_cache"].shape[:2]
    for x, cache, scale in ((one(s["k"], s["k_weight"]), s["k_cache"], s["k_scale"]), (s["v"].float(), s["v_cache"], s["v_scale"])):
        most = torch.zeros(rows, H, device=row.device).index_reduce_(0, row, x.abs().amax(2), "amax")
        elements = cache.view(torch.uint8).view(P, H, -1, size, D).transpose(1, 2).reshape(-1, H, size, D)[at]
        before = scale.transpose(1, 2).reshape(-1, H)[at].float()
        after = torch.exp2(exponent_for(most).float())
        after = torch.where((old > 0)[:, None], torch.maximum(after, before), after)
        grown = (elements.view(ELEMENT).float() * (before / after)[..., None, None]).to(ELEMENT).view(torch.uint8)
        stays = ~((place < old[:, None])[:, None, :, None] & (after > before)[..., None, None])
        elements = torch.where(stays, elements, grown)
        new = (x / after[row][..., None]).to(ELEMENT).view(torch.uint8)
        elements[row, :, slot % size] = new
        p, b = at // (page // size), at % (page // size)
        # rows that no token goes to put back what is there, behind the last block's row
        p, b = torch.where(used, p, p[row[-1]]), torch.where(used, b, b[row[-1]])
        elements = torch.where(used[:, None, None, None], elements, elements[row[-1]])
        after = torch.where(used[:, None], after, after[row[-1]])
        cache.view(torch.uint8).view(P, H, -1, size, D)[p, :, b] = elements
        scale[p, :, b] = after.to(torch.bfloat16)
    return one(s["q"], s["q_weight"]).to(dtype), values(s)


def plain_attention(s, c):
    Hq, Hk, D = c["q_heads"], c["kv_heads"], c["dim"]
    B, n, G = c["requests"], s["nodes_hi"], c["q_heads"] // c["kv_heads"]
    req, local, cu = owners(s)
    S = s["page_table"].shape[1] * c["page"]
    pages = s["page_table"].to(torch.int64)

    def cached(x, scale):
        x = x.view(torch.uint8)[pages].view(ELEMENT).float().unflatten(3, (-1, c["block"]))
        x *= scale[pages].float()[..., None, None]
        return x.flatten(3, 4).permute(0, 2, 1, 3, 4).reshape(B, Hk, S, D)

    q = torch.zeros(B, n, Hk, G, D, device=cu.device)
    q[req, local] = s["q"].float().reshape(-1, Hk, G, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, Hk, n * G, D)
    # a slot is seen where it is of the context, or of a node in the mask
    place = torch.arange(S, device=cu.device) - s["ctx_lens"].to(torch.int64)[:, None]
    mask = torch.zeros(B, n, dtype=torch.int64, device=cu.device)
    mask[req, local] = s["tree_mask"][:, 0]
    bit = (mask[:, :, None] >> place.clamp(0, 63)[:, None]) & 1
    tree = (place[:, None] >= 0) & (place[:, None] < n) & (bit != 0)
    sees = ((place < 0)[:, None] | tree)[:, None, :, None].expand(B, Hk, n, G, S)
    score = (q @ cached(s["k_cache"], s["k_scale"]).transpose(2, 3)) * (1 / math.sqrt(D))
    score = score.masked_fill(~sees.reshape(B, Hk, n * G, S), -math.inf)
    top = score.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    weight = (score - top).exp()
    total = weight.sum(3, keepdim=True)
    out = (weight @ cached(s["v_cache"], s["v_scale"])) / torch.where(total == 0, 1.0, total)
    out = out.reshape(B, Hk, n, G, D).permute(0, 2, 1, 3, 4)[req, local]
    lse = (total.log() + top).reshape(B, Hk, n, G).permute(0, 2, 1, 3)[req, local]
    return out.reshape(-1, Hq, D).to(s["q"].dtype), lse.reshape(-1, Hq)


def plain_commit(s, c):
    N, page, size = c["ngram"], c["page"], c["block"]
    cu = s["cu_seqlens"].to(torch.int64)
    path, accepted = s["path"].to(torch.int64), s["accepted"].to(torch.int64)
    ctx, pages = s["ctx_lens"].to(torch.int64), s["page_table"].to(torch.int64)
    B, P = path.shape
    # the blocks from the one that holds slot ctx on: rows of slots, each with the slot that it comes from
    first, width = ctx // size * size, (P + 2 * size - 1) // size * size
    slot = first[:, None] + torch.arange(width, device=cu.device)
    j = slot - ctx[:, None]
    kept = (j >= 0) & (j < accepted[:, None])
    source = torch.where(kept, ctx[:, None] + path.gather(1, j.clamp(0, P - 1)), slot)
    live = j < accepted[:, None]
    live_block = live.view(B, -1, size).any(2)
    limit = pages.shape[1] * page - 1
    a, b = pages.gather(1, source.clamp(max=limit) // page), source % page
    x, y = pages.gather(1, slot.clamp(max=limit) // page), slot % page
    # blocks with nothing to keep write the first one's again
    some = live_block.any(1)
    for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        raw = cache.view(torch.uint8)
        scale_of = scale[:, a, :, b // size].float()  # [B, width, layers, heads]
        after = torch.where(live[..., None, None], scale_of, 0.0).unflatten(1, (-1, size)).amax(2)
        after_of = after.repeat_interleave(size, 1)
        element = raw[:, a, :, b]  # [B, width, layers, heads, dim]
        factor = torch.where(live[..., None, None], scale_of / after_of, 1.0)
        element = torch.where((factor == 1.0)[..., None], element,
                              (element.view(ELEMENT).float() * factor[..., None]).to(ELEMENT).view(torch.uint8))
        here = raw[:, x, :, y]
        element = torch.where(live[..., None, None, None], element, here)
        write = (live_block & some[:, None]).repeat_interleave(size, 1)
        raw[:, x[write], :, y[write]] = element[write]
        at = write.view(B, -1, size)[:, :, 0]
        scale[:, x[:, ::size][at], :, y[:, ::size][at] // size] = after[at].to(torch.bfloat16)
    # the last N - 1 ids of the context followed by the accepted ones
    ids = s["ids"][(cu[:-1, None] + path).clamp(max=s["tokens"] - 1)]
    line = torch.cat([s["ngram_context"], ids], 1)
    context = line.gather(1, accepted[:, None] + torch.arange(N - 1, device=cu.device))
    return values(s), context, (ctx + accepted).to(torch.int32)


def plain_plan(s, c):
    table, page, P, limit = s["page_table"].to(torch.int64), c["page"], s["pages"], s["limit"]
    source, want = s["source"].to(torch.int64), s["want"].to(torch.int64)
    N, M, dev = source.shape[0], table.shape[1], table.device
    ctx = torch.where(source >= 0, s["ctx_lens"].to(torch.int64)[source.clamp(min=0)], 0)
    held, need = (ctx + page - 1) // page, ((ctx + want + page - 1) // page).clamp(max=M)
    entry, row = torch.arange(M, device=dev), torch.arange(N, device=dev)[:, None]
    carried = entry < held[:, None]
    p = torch.where(carried, table[source.clamp(min=0)], P)  # P: none
    # a page that new tokens will be written to is one row's alone
    written = ((want > 0) & (ctx % page != 0))[:, None] & (entry == held[:, None] - 1)
    shared = torch.zeros(P + 1, dtype=torch.int64, device=dev)
    shared.index_add_(0, torch.where(written, P, p).flatten(), torch.ones(N * M, dtype=torch.int64, device=dev))
    writer = torch.full((P + 1,), N, dtype=torch.int64, device=dev)
    writer.scatter_reduce_(0, torch.where(written, p, P).flatten(), row.expand(N, M).flatten(), "amin")
    keeps = carried & (~written | ((shared[p] == 0) & (writer[p] == row)))
    used = (shared[:P] > 0) | (writer[:P] < N)
    number = torch.arange(P, device=dev)
    moves, free = used & (number >= limit), ~used & (number < limit)
    # free pages by rank: first to pages that move below the limit, then to the rows' new places in order
    rank = free.cumsum(0) - 1
    frees = torch.full((P + N * M + 1,), -1, dtype=torch.int64, device=dev)
    frees[torch.where(free, rank, P + N * M)] = number
    frees[P + N * M] = -1
    room, moving = free.sum(), moves.sum()
    goes = frees[(moves.cumsum(0) - 1).clamp(min=0)]
    goes = torch.where(moves & (goes >= 0), goes, number)
    new = ((entry < need[:, None]) & ~carried) | (carried & written & ~keeps)
    given = frees[(new.flatten().cumsum(0) - 1 + moving).clamp(0, P + N * M)].view(N, M)
    result = torch.where(new, given, torch.where(keeps, goes[p.clamp(max=P - 1)], -1))
    # what has to be copied: the pages that moved, then the doubled ones
    moved = goes != number
    doubled = carried & written & ~keeps & (given >= 0)
    C = N + P - limit
    copies = torch.full((C + 1, 2), -1, dtype=torch.int64, device=dev)
    copies[torch.where(moved, moved.cumsum(0) - 1, C)] = torch.stack([number, goes], 1)
    doubles = doubled.flatten()
    copies[torch.where(doubles, doubles.cumsum(0) - 1 + moved.sum(), C)] = torch.stack([p.flatten(), given.flatten()], 1)
    taken = (moving + new.sum()).clamp(max=room)
    counts = torch.stack([moved.sum() + doubles.sum(), used.sum() + taken - moved.sum(), moving + new.sum() - taken])
    return result.to(torch.int32), ctx.to(torch.int32), copies[:C].to(torch.int32), counts.to(torch.int32)


def plain_copy(s, c):
    src, dst = s["copies"][:c["copies"]].to(torch.int64).unbind(1)
    if c["bits"] == 8:
        for x in (s["k_cache"].view(torch.uint8), s["v_cache"].view(torch.uint8), s["k_scale"], s["v_scale"]):
            x[:, dst] = x[:, src]
        return values(s)
    for x in (s["k_cache"], s["v_cache"]):
        x[:, dst] = x[:, src]
    return s["k_cache"], s["v_cache"]


PLAIN = dict(append=plain_append, attention=plain_attention, commit=plain_commit, plan=plain_plan, copy=plain_copy)


# --------------------------------------------------------- the work and 64 bits


def work(case):
    c = case
    if c["op"] == "plan":
        B, N, page = c["requests"], c["rows"], c["page"]
        most = -(-(c["ctx_hi"] + c["want_hi"]) // page)
        # the entries that requests hold, read; the new table, written
        held = sum(-(-n // page) for n in spread(c["ctx_lo"], c["ctx_hi"], B))
        return dict(bytes=4 * (held + B + 2 * N + N * most + N), flops=0)
    Hk, D, block = c["kv_heads"], c["dim"], c["block"]
    if c["op"] == "copy":
        row = D * 2 if c["bits"] == 16 else D + 2 / block
        return dict(bytes=2 * 2 * c["copies"] * c["layers"] * Hk * c["page"] * row + 8 * c["copies"], flops=0)
    B = c["requests"]
    T = sum(spread(c["nodes_lo"], c["nodes_hi"], B))
    row = D + 2 / block  # a token's keys or values of a head with their share of a scale
    if c["op"] == "append":
        Hq = c["q_heads"]
        return dict(bytes=T * (Hq * D * 2 * 2 + 2 * Hk * (D * 2 + row)) + T * 4 + 8 * B + 4 * c["rotary"] + 4 * D,
                    flops=T * (Hq + Hk) * (4 * D + 3 * c["rotary"]) + T * Hk * D * 4)
    if c["op"] == "attention":
        Hq = c["q_heads"]
        # which tree meets which context is drawn: the products go by the means
        slots = T + sum(spread(c["ctx_lo"], c["ctx_hi"], B))
        return dict(bytes=slots * Hk * row * 2 + T * Hq * (D * 2 * 2 + 4) + 8 * T + 12 * B, flops=4 * D * Hq * T * slots / B)
    moved = sum(max(0, a - 1) for a in spread(c["accept_lo"], c["accept_hi"], B))
    return dict(bytes=moved * c["layers"] * Hk * row * 2 * 2 + B * (16 * (c["ngram"] - 1) + 16) + 8 * moved, flops=0)


def exact(case, seed):
    c = case
    if c["op"] == "plan":
        return None
    s = prepare(case, seed)
    if c["op"] == "copy":
        names = ("k_cache", "v_cache") if c["bits"] == 16 else ("kv",)
        out = [(s[x] if c["bits"] == 16 else values(s)).double() for x in names]
        for src, dst in s["copies"].tolist()[:c["copies"]]:
            for x in out:
                if c["bits"] == 16:
                    x[:, dst] = x[:, src]
                else:
                    x[:, :, dst] = x[:, :, src]
        return out if c["bits"] == 16 else out[0]
    cu, ctx, table = s["cu_seqlens"].tolist(), s["ctx_lens"].tolist(), s["page_table"].tolist()
    return dict(append=exact_append, attention=exact_attention, commit=exact_commit)[c["op"]](s, c, cu, ctx, table)


def nearest(x, scale):
    """x as the nearest element times scale, in 64 bits: elements have four significant bits down to 2**-6, and a spacing of 2**-9
    below; ties go to the even one."""
    y = x / scale
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * scale


def least_scale(most):
    """The least power of two that takes `most` into the elements' range, in 64 bits."""
    e = torch.ceil(torch.log2((most / LARGEST).clamp(min=2.0 ** (LEAST_EXPONENT - 1))))
    e = torch.where(most > LARGEST * torch.exp2(e), e + 1, e)
    e = torch.where(most <= LARGEST * torch.exp2(e - 1), e - 1, e)
    return torch.exp2(e.clamp(min=LEAST_EXPONENT))


def exact_append(s, c, cu, ctx, table):
    R, size, page = c["rotary"], c["block"], c["page"]
    i = torch.arange(R // 2, dtype=torch.float64)
    inv = (ROPE_BASE ** (-2.0 * i / R)).cuda()
    turn = torch.polar(torch.ones(s["tokens"], R // 2, dtype=torch.float64, device="cuda"), s["positions"].double()[:, None] * inv)

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

    held, scales = values(s).double(), s["kv_scale"].double()
    new = torch.stack([one(s["k"], s["k_weight"]), s["v"].double()])
    for r in range(c["requests"]):
        slot, end = ctx[r], ctx[r] + cu[r + 1] - cu[r]
        while slot < end:  # block by block
            first, upto = slot // size * size, min(end, (slot // size + 1) * size)
            p, at = table[r][slot // page], first % page
            x = new[:, cu[r] + slot - ctx[r]:cu[r] + upto - ctx[r]].transpose(1, 2)
            scale = least_scale(x.abs().amax((2, 3)))
            before = scales[:, p, :, at // size]
            if slot > first:
                scale = torch.maximum(scale, before)
                old = held[:, p, :, at:at + slot - first]
                held[:, p, :, at:at + slot - first] = nearest(old, scale[..., None, None])
            # what lies behind the new tokens keeps its elements, which stand for other values now
            rest = held[:, p, :, at + upto - first:at + size]
            rest *= (scale / before)[..., None, None]
            held[:, p, :, at + slot - first:at + upto - first] = nearest(x, scale[..., None, None])
            slot = upto
    return one(s["q"], s["q_weight"]), held


def exact_attention(s, c, cu, ctx, table):
    Hq, Hk, D, page = c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    if work(c)["flops"] > 6e11:
        return None
    out = torch.zeros(s["tokens"], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["tokens"], Hq, dtype=torch.float64, device="cuda")
    held = values(s)
    for r in range(c["requests"]):
        n, length = cu[r + 1] - cu[r], ctx[r] + cu[r + 1] - cu[r]
        if n == 0:
            continue
        pages = torch.tensor(table[r][:-(-length // page)], device="cuda")
        sees = torch.ones(n, length, dtype=torch.bool, device="cuda")
        bits = s["tree_mask"][cu[r]:cu[r + 1], 0].tolist()
        sees[:, ctx[r]:] = torch.tensor([[bool((row >> j) & 1) for j in range(n)] for row in bits], device="cuda")
        for h in range(Hq):  # head by head
            k, v = (held[x, pages, h // (Hq // Hk)].reshape(-1, D)[:length].double() for x in (0, 1))
            score = s["q"][cu[r]:cu[r + 1], h].double() @ k.T / math.sqrt(D)
            score[~sees] = -math.inf
            lse[cu[r]:cu[r + 1], h] = torch.logsumexp(score, 1)
            out[cu[r]:cu[r + 1], h] = torch.softmax(score, 1) @ v
    return out, lse


def exact_commit(s, c, cu, ctx, table):
    size, page = c["block"], c["page"]
    held, scales = values(s).double(), s["kv_scale"].double()
    accepted, paths = s["accepted"].tolist(), s["path"].tolist()
    for r in range(c["requests"]):
        end = ctx[r] + accepted[r]
        first = ctx[r] // size * size
        while first < end:  # block by block
            p, at = table[r][first // page], first % page
            before = scales[:, :, p, :, at // size].clone()
            after = torch.zeros_like(before)
            came = []
            for slot in range(first, min(end, first + size)):
                j = slot - ctx[r]
                o = ctx[r] + paths[r][j] if j >= 0 else slot
                came.append(held[:, :, table[r][o // page], :, o % page].clone())
                after = torch.maximum(after, scales[:, :, table[r][o // page], :, o % page // size])
            for i, x in enumerate(came):
                held[:, :, p, :, at + i] = nearest(x, after[..., None])
            # what lies behind keeps its elements, unless a later block takes it
            stale = held[:, :, p, :, at + len(came):at + size]
            stale *= (after / before)[..., None, None]
            scales[:, :, p, :, at // size] = after
            first += size
    return held, None, None
