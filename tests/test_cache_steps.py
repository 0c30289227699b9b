"""The operators on caches in 8 bits and on pages as a server runs them, on the
GPU: a plan, the copy of its pages, the append, the attention and the commit in
turn, each step against plain 64-bit host implementations; captured and
replayed; on other streams; and every argument in a wrong form."""

import numpy as np
import pytest
import torch

import cache_reference as ref8
import layer_gram_embedding_gb300 as ple
import tree_reference as ref
from test_cache_ops import (Cache8, check_append, check_attention, check_plan, read, same)
from test_tree_ops import U, check_rows, dev, host, rows
from test_tree_refusals import REFUSED, longer, other_dtype, strided

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = torch.device("cuda:0")
FP8 = torch.float8_e4m3fn
HQ, HK, D, PAGE, BLOCK, PAGES, LAYERS, MAX_PAGES = 8, 2, 64, 32, 16, 90, 2, 24


def take_over(cache, caches):
    """The device's caches as the host's."""
    cache.k, cache.v, cache.k_scale, cache.v_scale = (x.copy() for x in read(caches))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_requests_that_fork_and_end_step_by_step(dtype):
    rng = np.random.default_rng(61)
    cache = Cache8(rng, [1], PAGE, BLOCK, HK, D, layers=LAYERS, spare=PAGES - 1, odd=np.ones(1))
    caches = cache.device()
    table, ctx = np.full((1, MAX_PAGES), -1, np.int32), np.zeros(1, np.int32)
    rope, w = ple.ple_prepare_rope(D, 1e6), ref.inverse_frequencies(D, 1e6)
    qw, kw = rows(rng, (D,), dtype), rows(rng, (D,), dtype)
    steps = [  # source of each row, drafted nodes (the first step: a prompt), page limit
        ([-1], [75], None), ([0, 0, 0], [5, 1, 0], None), ([1, 0, 0, -1], [4, 7, 2, 40], None),
        ([3, 2, 1, 0, 0], [1, 1, 33, 1, 2], 40), ([4, 2], [64, 3], 30), ([1], [0], 8),
        ([0, 0], [1, 1], None),
    ]
    for source, counts, limit in steps:
        nxt, lens, copies, told = check_plan(table, ctx, source, counts, PAGES, PAGE, limit)
        assert int(told[2]) == 0
        before = read(caches)
        ple.ple_copy_pages(copies, *caches)
        after = read(caches)
        for a, b in zip(after, before):
            for x, y in copies.tolist():
                if x >= 0:
                    b[:, y] = a[:, x]
            assert same(a, b)
        table, ctx = nxt.cpu().numpy(), lens.cpu().numpy()
        cu, T = ref.prefix(counts), sum(counts)
        if T == 0:
            continue
        parent = ref.trees(rng, counts, reach=3)
        if len(counts) == 1:
            parent = np.arange(-1, T - 1).astype(np.int32)     # a prompt's rows are a chain
        positions, masks = ple.ple_build_tree_index(dev(parent), dev(cu), lens, 2)
        at, seen = positions.cpu().numpy(), masks.cpu().numpy()
        for layer in range(LAYERS):
            q, k, v = (rows(rng, (T, h, D), dtype, 2.0 ** layer) for h in (HQ, HK, HK))
            mine = [c[layer] for c in caches]
            before = read(mine)
            got = ple.ple_qk_norm_rope_fp8(q, k, v, positions, rope, qw, kw, *mine, nxt, lens,
                                           dev(cu))
            want, size = ref.norm_rope(host(q), host(qw), at, w, 1e-6, False, 1.0)
            check_rows(got, want, size, U[dtype], "q")
            want, size = ref.norm_rope(host(k), host(kw), at, w, 1e-6, False, 1.0)
            after = read(mine)
            check_append((after[0][0], after[2][0]), (before[0][0], before[2][0]), want,
                         2.0 ** -20 * size + 2.0 ** -40, table, ctx, cu, exact=False)
            check_append((after[1][0], after[3][0]), (before[1][0], before[3][0]), host(v),
                         np.zeros(v.shape), table, ctx, cu, exact=True)
            take_over(cache, mine)
            cache.table = table
            check_attention(got, cache, ctx, cu, seen, caches=mine, what=str(counts))
        # the longest branch of each tree is accepted
        path, accepted = np.zeros((len(counts), 80), np.int32), np.zeros(len(counts), np.int32)
        for r, n in enumerate(counts):
            lines = ref.ancestors(parent[cu[r]:cu[r + 1]])
            line = sorted(max(lines, key=len)) if n else []
            path[r, :len(line)], accepted[r] = line, len(line)
        ids = rng.integers(0, 99, T)
        before = read(caches)
        _, lens = ple.ple_tree_commit_fp8(dev(ids), dev(path), dev(accepted), dev(cu), None, lens,
                                          nxt, *caches)
        after = read(caches)
        for i in (0, 1):
            want, scales = ref8.commit(path, accepted, cu, ctx, table, before[i], before[i + 2])
            assert same(after[i], want) and same(after[i + 2], scales)
        ctx = lens.cpu().numpy()


def test_pages_that_move_change_no_answer():
    rng = np.random.default_rng(62)
    counts, ctx = [3, 20, 1], np.array([500, 77, 300], np.int32)
    cu = ref.prefix(counts)
    cache = Cache8(rng, [int(c) + n for c, n in zip(ctx, counts)], PAGE, BLOCK, HK, D, spare=60)
    for r, n in enumerate(counts):
        cache.fill(rng, r, 0, int(ctx[r]) + n)
    _, masks = ref.tree_index(ref.trees(rng, counts), cu, ctx, 1)
    q = rows(rng, (sum(counts), HQ, D), torch.bfloat16)
    caches = cache.device()
    want = ple.ple_tree_attention_fp8(q, *caches, dev(cache.table), dev(ctx), dev(cu), dev(masks))
    used = int((cache.table < 2 ** 30).sum())
    held = dev(ctx + np.array(counts, np.int32))      # the nodes' slots move with the rest
    nxt, lens, copies, told = ple.ple_plan_pages(
        dev(cache.table), held, dev(np.arange(3, dtype=np.int32)), dev(np.zeros(3, np.int32)),
        cache.k.shape[1], PAGE, used)
    assert told.tolist() == [int((copies[:, 0] >= 0).sum()), used, 0] and int(told[0]) > 0
    ple.ple_copy_pages(copies, *caches)
    assert int(nxt.max()) == used - 1 and torch.equal(lens, held)
    for c in caches:
        (c.view(torch.uint8) if c.dtype == FP8 else c)[used:] = 255     # given back
    got = ple.ple_tree_attention_fp8(q, *[c[:used] for c in caches], nxt, dev(ctx), dev(cu),
                                     dev(masks))
    assert torch.equal(got, want)


# ------------------------------------------------------------ graphs, streams


def make_step(seed, T=24, B=3):
    rng = np.random.default_rng(seed)
    counts, ctx = [T // B] * B, np.array([200, 33, 0], np.int32)[:B]
    cache = Cache8(rng, [200 + T] * B, PAGE, BLOCK, HK, D, odd=np.ones(1))
    for r in range(B):
        cache.fill(rng, r, 0, int(ctx[r]))
    parent = ref.trees(rng, counts)
    qkv = rows(rng, (T, HQ + 2 * HK, D), torch.bfloat16)
    kc, vc, ks, vs = cache.device()
    table = cache.table.copy()
    table[table >= 2 ** 30] = -1
    path = np.tile(np.arange(0, 6, 2, dtype=np.int32), (B, 1))
    return dict(q=qkv[:, :HQ], k=qkv[:, HQ:HQ + HK], v=qkv[:, HQ + HK:], kc=kc, vc=vc, ks=ks, vs=vs,
                table=dev(table), ctx=dev(ctx), cu=dev(ref.prefix(counts)), parent=dev(parent),
                w=rows(rng, (D,), torch.bfloat16), rope=ple.ple_prepare_rope(D),
                source=dev(np.array([0, 1, 1], np.int32)), want=dev(np.array(counts, np.int32)),
                ids=dev(rng.integers(0, 99, T)), context=dev(rng.integers(0, 99, (B, 2))),
                path=dev(path), accepted=dev(np.array([3, 0, 2], np.int32)))


def step(s):
    """Every operator in turn; what a step leaves behind."""
    pages = s["kc"].shape[0]
    caches = s["kc"], s["vc"], s["ks"], s["vs"]
    table, ctx, copies, told = ple.ple_plan_pages(s["table"], s["ctx"], s["source"], s["want"],
                                                  pages, PAGE)
    ple.ple_copy_pages(copies, *caches)
    positions, masks = ple.ple_build_tree_index(s["parent"], s["cu"], ctx, 1)
    q = ple.ple_qk_norm_rope_fp8(s["q"], s["k"], s["v"], positions, s["rope"], s["w"], s["w"],
                                 *caches, table, ctx, s["cu"])
    out, lse = ple.ple_tree_attention_fp8(q, *caches, table, ctx, s["cu"], masks, return_lse=True)
    nxt, lens = ple.ple_tree_commit_fp8(s["ids"], s["path"], s["accepted"], s["cu"], s["context"],
                                        ctx, table, *caches)
    return [table, ctx, copies, told, q, out, lse, nxt, lens]


def state(s):
    return [s[k].view(torch.uint8) if s[k].dtype == FP8 else s[k] for k in ("kc", "vc", "ks", "vs")]


def equal(a, b):
    """Bit for bit but for what a NaN carries: slots that nobody filled may be some."""
    return all(torch.equal(x.nan_to_num() if x.is_floating_point() else x,
                           y.nan_to_num() if y.is_floating_point() else y) for x, y in zip(a, b))


def test_a_captured_step_replays_as_it_runs():
    s, t = make_step(71), make_step(71)
    other = make_step(72)
    torch.cuda.synchronize()
    for x in (s, t):
        step(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(s)
    for keys in ((), ("q", "k", "v", "kc", "vc", "ks", "vs", "table", "parent"), ("ctx",)):
        for key in keys:
            if key == "ctx":
                for x in (s, t):
                    x["ctx"].copy_(dev(np.array([0, 190, 64], np.int32)))
            else:
                for x in (s, t):
                    x[key].copy_(other[key])
        for a, b in zip(state(s), state(t)):
            a.copy_(b)
        graph.replay()
        want = step(t)
        torch.cuda.synchronize()
        assert equal(captured, want) and equal(state(s), state(t))


def calls(s):
    """Each operator on a step's inputs, outputs its own: name, call(stream)."""
    positions, masks = ple.ple_build_tree_index(s["parent"], s["cu"], s["ctx"], 1)
    caches = s["kc"], s["vc"], s["ks"], s["vs"]
    nothing = torch.zeros_like(s["accepted"])
    tail = s["table"], s["ctx"], s["cu"]
    return {
        "append": lambda st: [ple.ple_qk_norm_rope_fp8(s["q"], s["k"], s["v"], positions, s["rope"],
                                                       s["w"], s["w"], *caches, *tail, stream=st)],
        "attention": lambda st: ple.ple_tree_attention_fp8(s["q"], *caches, *tail, masks,
                                                           return_lse=True, stream=st),
        # nothing is accepted: the caches stay as they are
        "commit": lambda st: ple.ple_tree_commit_fp8(s["ids"], s["path"], nothing, s["cu"],
                                                     s["context"], s["ctx"], s["table"], *caches,
                                                     stream=st),
        "plan": lambda st: ple.ple_plan_pages(s["table"], s["ctx"], s["source"], s["want"],
                                              s["kc"].shape[0], PAGE, stream=st),
    }


BUSY = 100_000_000  # clocks: some tens of ms


@pytest.mark.parametrize("name", ["append", "attention", "commit", "plan"])
def test_a_given_stream_waits_for_the_memory_it_is_given(name):
    s = make_step(73)
    call = calls(s)[name]
    want = [x.clone() for x in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of the outputs' sizes, freed while the current stream still writes them
    blocks = [torch.empty_like(x) for x in want]
    torch.cuda._sleep(BUSY)
    for x in blocks:
        x.fill_(1)
    del blocks, x
    got = call(side)
    assert not side.query()
    side.synchronize()
    assert torch.cuda.current_stream().query()   # it came after the fill
    assert equal(got, want)
    # and the other way round: freed while the side stream still writes them
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = call(side)
    taken = {x.data_ptr() for x in got}
    sizes = [(x.shape, x.dtype) for x in got]
    del got
    again = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in sizes]
    assert not side.query()
    assert not taken & {x.data_ptr() for x in again}
    torch.cuda.synchronize()


def test_calls_on_two_streams_share_no_workspace():
    rng = np.random.default_rng(74)
    for counts, ctx in (([2], [5001]), ([40], [3000])):
        cache = Cache8(rng, [ctx[0] + counts[0]], PAGE, BLOCK, HK, D)
        cache.fill(rng, 0, 0, ctx[0] + counts[0])
        cu, ctx = ref.prefix(counts), np.array(ctx, np.int32)
        _, masks = ref.tree_index(ref.trees(rng, counts), cu, ctx, 1)
        tail = (*cache.device(), dev(cache.table), dev(ctx), dev(cu), dev(masks))
        a = rows(rng, (sum(counts), HQ, D), torch.bfloat16)
        b = torch.flip(a, [0])
        want_a, want_b = (ple.ple_tree_attention_fp8(x, *tail) for x in (a, b))
        plan = (dev(cache.table), dev(ctx), dev(np.zeros(5, np.int32)),
                dev(np.full(5, 40, np.int32)), cache.k.shape[1] + 50, PAGE)
        want_p = [x.clone() for x in ple.ple_plan_pages(*plan)]
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(10):
            torch.cuda._sleep(BUSY // 20)
            got_a, p = ple.ple_tree_attention_fp8(a, *tail), ple.ple_plan_pages(*plan)
            got_b = ple.ple_tree_attention_fp8(b, *tail, stream=side)
            r = ple.ple_plan_pages(*plan, stream=side)
            torch.cuda.synchronize()
            assert torch.equal(got_a, want_a) and torch.equal(got_b, want_b)
            assert equal(p, want_p) and equal(r, want_p)


def test_the_current_stream_given_by_name_and_programmatic_launch():
    s = make_step(75)
    want = [x.clone() for x in step(s)]
    after = [x.clone() for x in state(s)]
    side = torch.cuda.Stream()
    for on in (True, False):
        t = make_step(75)
        torch.cuda.synchronize()
        old = ple.lib().ple_set_programmatic_launch(1 if on else 0)
        try:
            with torch.cuda.stream(side):
                got = step(t)
            side.synchronize()
        finally:
            ple.lib().ple_set_programmatic_launch(old)
        assert equal(got, want) and equal(state(t), after)


def test_empty_batches():
    s = make_step(76)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    caches = s["kc"], s["vc"], s["ks"], s["vs"]
    before = [x.clone() for x in state(s)]
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = ple.ple_qk_norm_rope_fp8(s["q"][:0], s["k"][:0], s["v"][:0], None, None, None, None,
                                 *caches, s["table"], s["ctx"], torch.zeros_like(s["cu"]))
    out, lse = ple.ple_tree_attention_fp8(q, *caches, s["table"], s["ctx"],
                                          torch.zeros_like(s["cu"]),
                                          torch.zeros((0, 1), dtype=torch.int64, device=DEV),
                                          return_lse=True)
    assert q.shape == out.shape == (0, HQ, D) and lse.shape == (0, HQ)
    ple.ple_tree_commit_fp8(s["ids"], s["path"][:0], none, zero, s["context"][:0], none,
                            s["table"][:0], *caches)
    nothing = ple.ple_tree_commit_fp8(s["ids"], s["path"][:, :0], s["accepted"], s["cu"], None,
                                      s["ctx"], s["table"], *caches)
    assert nothing[0] is None and torch.equal(nothing[1], s["ctx"])
    ple.ple_copy_pages(none.view(0, 2), *caches)
    assert equal(state(s), before)


# ------------------------------------------------------------------- refusals


def forms():
    s = make_step(81)
    T, B = s["q"].shape[0], 3

    def empty(*shape, dtype=torch.int32):
        return torch.zeros(shape, dtype=dtype, device=DEV)

    positions, masks = ple.ple_build_tree_index(s["parent"], s["cu"], s["ctx"], 1)
    caches = dict(k_cache=s["kc"], v_cache=s["vc"], k_scale=s["ks"], v_scale=s["vs"])
    paged = dict(caches, page_table=s["table"], ctx_lens=s["ctx"], cu_seqlens=s["cu"])
    append = dict(q=s["q"], k=s["k"], v=s["v"], positions=positions, rope=s["rope"],
                  q_weight=s["w"], k_weight=s["w"].clone(), **paged)
    attention = dict(q=s["q"], tree_mask=masks, **paged)
    commit = dict(input_ids=s["ids"], path=s["path"], accepted=torch.zeros_like(s["accepted"]),
                  ngram_context=s["context"], **paged)
    copies = dev(np.array([[0, 3], [-1, -1]], np.int32))
    return {
        "append": (ple.ple_qk_norm_rope_fp8, append),
        "append, outputs given": (ple.ple_qk_norm_rope_fp8, dict(
            append, q_out=empty(T, HQ, D, dtype=torch.bfloat16))),
        "attention": (ple.ple_tree_attention_fp8, attention),
        "attention, outputs given": (ple.ple_tree_attention_fp8, dict(
            attention, out=empty(T, HQ, D, dtype=torch.bfloat16),
            lse=empty(T, HQ, dtype=torch.float32),
            workspace=ple.ple_tree_attention_fp8_workspace(T, HQ, HK, D))),
        "commit": (ple.ple_tree_commit_fp8, commit),
        "commit, outputs given": (ple.ple_tree_commit_fp8, dict(
            commit, next_context=empty(B, 2, dtype=torch.int64), next_ctx_lens=empty(B))),
        "plan": (ple.ple_plan_pages, dict(
            page_table=s["table"], ctx_lens=s["ctx"], source=s["source"], want=s["want"],
            num_pages=s["kc"].shape[0], page_size=PAGE)),
        "copy": (ple.ple_copy_pages, dict(caches, copies=copies)),
    }


# sizes that a call takes from the argument itself, by form: (argument, dimension)
FREE = {
    "append": {("q", 1), ("page_table", 1)},
    "append, outputs given": {("page_table", 1)},
    "attention": {("page_table", 1), ("tree_mask", 1)},
    "attention, outputs given": {("page_table", 1), ("tree_mask", 1), ("workspace", 0)},
    "commit": {("input_ids", 0), ("path", 1), ("page_table", 1), ("ngram_context", 1)},
    "commit, outputs given": {("input_ids", 0), ("path", 1), ("page_table", 1)},
    "plan": {("page_table", 1)},
    "copy": {("copies", 0)},
}


def wider(t):
    """The same values with a stride of 2 in the last dimension."""
    if t.dtype != FP8:
        return strided(t)
    wide = torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=torch.uint8, device=t.device)
    wide[..., ::2] = t.view(torch.uint8)
    return wide.view(FP8)[..., ::2]


def one_longer(t, dim):
    return longer(t.view(torch.uint8), dim).view(FP8) if t.dtype == FP8 else longer(t, dim)


@pytest.mark.parametrize("name", list(FREE))
def test_every_argument_is_looked_at(name):
    fn, good = forms()[name]
    fn(**good)
    for key, t in good.items():
        if not isinstance(t, torch.Tensor):
            continue
        bad = {"dtype": t.view(torch.uint8) if t.dtype == FP8 else other_dtype(t),
               "host": t.cpu(), "stride": wider(t)}
        if name == "attention" and key == "q":
            del bad["dtype"]      # either goes with such a cache
        for dim in range(t.dim()):
            if (key, dim) not in FREE.get(name, ()):
                bad[f"longer in dimension {dim}"] = one_longer(t, dim)
        for what, wrong in bad.items():
            try:
                fn(**dict(good, **{key: wrong}))
            except REFUSED:
                continue
            pytest.fail(f"{key}: {what} was taken")


def test_other_refusals():
    f = forms()
    append, attention, commit, copy = (f[n][1] for n in ("append", "attention", "commit", "copy"))
    plan = f["plan"][1]
    cases = [
        (ple.ple_qk_norm_rope_fp8, dict(append, positions=None), "positions"),
        (ple.ple_tree_attention_fp8, dict(attention, workspace=torch.empty(
            16, dtype=torch.uint8, device=DEV)), ""),
        (ple.ple_tree_attention_fp8, dict(attention, scale=float("inf")), ""),
        (ple.ple_tree_commit_fp8, dict(commit, next_ctx_lens=commit["ctx_lens"]), "overlap"),
        (ple.ple_plan_pages, dict(plan, limit=-1), "limit"),
        (ple.ple_plan_pages, dict(plan, limit=10 ** 6), "limit"),
        (ple.ple_plan_pages, dict(plan, num_pages=0), ""),
        (ple.ple_plan_pages, dict(plan, num_pages=2 ** 31), ""),
        (ple.ple_plan_pages, dict(plan, page_size=0), ""),
        (ple.ple_plan_pages, dict(plan, page_size=2 ** 31), ""),
        (ple.ple_plan_pages, dict(plan, source=plan["source"][:0], want=plan["want"][:0]), "row"),
        (ple.ple_copy_pages, dict(copy, k_scale=None), "scales"),
        (ple.ple_copy_pages, dict(copy, k_scale=None, v_scale=None), "scales"),
    ]
    # a block of three pages' parts, of a page that holds no whole block, and none at all
    for key in ("k_scale", "v_scale"):
        assert append[key].shape[2] == 2
    odd = torch.ones((append["k_cache"].shape[0], HK, 3), dtype=torch.bfloat16, device=DEV)
    none = odd[:, :, :0]
    many = torch.ones((append["k_cache"].shape[0], HK, 4), dtype=torch.bfloat16, device=DEV)
    for bad in (odd, none, many):
        for name in ("append", "attention", "commit", "copy"):
            cases.append((f[name][0], dict(f[name][1], k_scale=bad, v_scale=bad), "scale"))
    for fn, kw, match in cases:
        with pytest.raises(REFUSED, match=match):
            fn(**kw)
    torch.cuda.synchronize()
