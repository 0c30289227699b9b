"""Tree operators on a given stream: what a call allocates comes from the
current stream's memory, which work queued there may still be using, so the
given stream waits for it; and nothing is handed out again before the given
stream is done.  A call that allocates nothing leaves the streams alone."""

import numpy as np
import pytest
import torch

import layer_gram_embedding_gb300 as ple
from test_tree_ops import attention_inputs, dev, make_step, step

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BUSY = 100_000_000  # clocks: some tens of ms


def same(a, b):
    return all(torch.equal(x.nan_to_num() if x.is_floating_point() else x,
                           y.nan_to_num() if y.is_floating_point() else y) for x, y in zip(a, b))


def calls(s):
    """Each operator on a step's inputs, outputs its own: name, call(stream)."""
    positions, masks = ple.ple_build_tree_index(s["parent"], s["cu"], s["ctx"], 1)
    nothing = torch.zeros_like(s["accepted"])
    paged = dict(k_cache=s["kc"], v_cache=s["vc"], page_table=s["table"], ctx_lens=s["ctx"],
                 cu_seqlens=s["cu"])
    return {
        "index": lambda st: ple.ple_build_tree_index(s["parent"], s["cu"], s["ctx"], 1, stream=st),
        "row ids": lambda st: [ple.ple_tree_row_ids(s["ids"], s["parent"], s["cu"], s["context"],
                                                    s["M"], s["vocab"], s["off"], 3, 2, 7,
                                                    stream=st)],
        "rope": lambda st: [ple.ple_prepare_rope(128, stream=st)],
        "norm": lambda st: [ple.ple_qk_norm_rope(s["q"], s["k"], s["v"], positions, s["rope"],
                                                 s["qw"], s["kw"], stream=st, **paged)],
        "norm alone": lambda st: ple.ple_qk_norm_rope(s["q"], s["k"], None, positions, s["rope"],
                                                      stream=st),
        "attention": lambda st: ple.ple_tree_attention(s["q"], s["kc"], s["vc"], s["table"],
                                                       s["ctx"], s["cu"], masks, return_lse=True,
                                                       stream=st),
        # nothing is accepted: the caches stay as they are
        "commit": lambda st: ple.ple_tree_commit(s["ids"], s["path"], nothing, s["cu"],
                                                 s["context"], s["ctx"], s["table"], s["kc"],
                                                 s["vc"], stream=st),
    }


@pytest.mark.parametrize("name", ["index", "row ids", "rope", "norm", "norm alone", "attention",
                                  "commit"])
def test_a_given_stream_waits_for_the_memory_it_is_given(name):
    s = make_step(51)
    step(s)
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
    assert same(got, want)
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


def test_attention_calls_on_two_streams_share_no_workspace():
    # a call on the current stream frees its workspace on return, its kernels still waiting to run
    rng = np.random.default_rng(52)
    for counts, ctx, Hq, Hk, D, page in (([20], [3001], 8, 2, 64, 16), ([3], [5000], 4, 2, 128, 20)):
        q, cache, ctx, cu, masks = attention_inputs(rng, counts, ctx, Hq, Hk, D, page,
                                                    torch.bfloat16)
        tail = (cache.k, cache.v, dev(cache.table), dev(ctx), dev(cu), dev(masks))
        a, b = q, torch.flip(q, [0])
        want_a, want_b = ple.ple_tree_attention(a, *tail), ple.ple_tree_attention(b, *tail)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(10):
            torch.cuda._sleep(BUSY // 20)
            got_a = ple.ple_tree_attention(a, *tail)
            got_b = ple.ple_tree_attention(b, *tail, stream=side)
            torch.cuda.synchronize()
            assert torch.equal(got_a, want_a) and torch.equal(got_b, want_b)


def test_a_call_that_allocates_nothing_does_not_wait():
    rng = np.random.default_rng(53)
    q, cache, ctx, cu, masks = attention_inputs(rng, [20], [301], 8, 2, 64, 16, torch.bfloat16)
    call = (q, cache.k, cache.v, dev(cache.table), dev(ctx), dev(cu), dev(masks))
    want = ple.ple_tree_attention(*call)
    out, workspace = torch.empty_like(q), ple.ple_tree_attention_workspace(20, 8, 2, 64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    ple.ple_tree_attention(*call, out=out, workspace=workspace, stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_the_current_stream_given_by_name():
    s = make_step(54)
    want = [x.clone() for x in step(s)]
    side = torch.cuda.Stream()
    t = make_step(54)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for name, call in calls(t).items():
            call(side)
        got = step(t)
    side.synchronize()
    assert same(got, want)


def test_a_given_stream_inside_a_capture():
    s = make_step(55)
    positions, masks = ple.ple_build_tree_index(s["parent"], s["cu"], s["ctx"], 1)
    call = (s["q"], s["kc"].nan_to_num(), s["vc"].nan_to_num(), s["table"], s["ctx"], s["cu"], masks)
    want = ple.ple_tree_attention(*call)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        got = ple.ple_tree_attention(*call, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
