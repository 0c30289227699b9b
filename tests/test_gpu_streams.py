"""The hash's calls on a given stream: what they allocate comes from the
current stream's memory, so the given stream waits for the work queued there,
and nothing is handed out again before the given stream is done."""

import numpy as np
import pytest
import torch

import layer_gram_embedding_gb300 as ple
import oracle
import workloads as wl

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BUSY = 100_000_000  # clocks: some tens of ms


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


def calls():
    b = wl.prefill_512()
    cu, ids, ctx = dev(b.cu_seqlens), dev(b.ids), dev(b.ngram_context)
    M, vocab, off = dev(b.layer_multipliers), dev(b.vocab_sizes), dev(b.offsets)
    req, local = (dev(x) for x in oracle.token_index(b.cu_seqlens, b.num_requests, b.num_tokens,
                                                     False))
    B, T, N, hpn = b.num_requests, b.num_tokens, b.ngram_size, b.heads_per_ngram
    L, H = b.layer_multipliers.reshape(-1, N).shape[0], b.vocab_sizes.shape[-1]
    rows = ple.ple_row_ids(ids, req, local, ctx, M, vocab, off, N, hpn, b.boundary_id)
    table = torch.ones((L, int(rows.max()) + 1, 8), dtype=torch.bfloat16, device="cuda")
    x, v = dev(np.arange(-500, 500)), dev(np.full(1000, 7))
    plan = ple.ple_shard_plan(b.cu_seqlens, B, T, 2, 1)
    return {
        "index": lambda st: ple.ple_build_token_index(cu, B, T, False, stream=st),
        "row ids": lambda st: [ple.ple_row_ids(ids, req, local, ctx, M, vocab, off, N, hpn,
                                               b.boundary_id, stream=st)],
        "heads": lambda st: [ple.ple_prepare_heads(vocab, off, stream=st)],
        "embed": lambda st: [ple.ple_row_embed(ids, req, local, ctx, M, vocab, off, N, hpn,
                                               b.boundary_id, table, stream=st)],
        "shard": lambda st: ple.ple_shard_inputs(ids, cu, ctx, plan, stream=st),
        "validate": lambda st: [ple.ple_validate_index(cu, B, T, False, local, local, stream=st)],
        "floor mod": lambda st: ple.ple_selftest_floor_mod(x, v, stream=st),
    }


@pytest.mark.parametrize("name", ["index", "row ids", "heads", "embed", "shard", "validate",
                                  "floor mod"])
def test_a_given_stream_waits_for_the_memory_it_is_given(name):
    call = calls()[name]
    want = [x.clone() for x in call(None)]
    if name == "validate":
        assert int(want[0]) < 512   # a local index for a request one: the call finds the first such token
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    blocks = [torch.empty_like(x) for x in want]
    torch.cuda._sleep(BUSY)
    for x in blocks:
        x.fill_(1)
    del blocks, x
    got = call(side)
    assert not side.query()
    side.synchronize()
    assert torch.cuda.current_stream().query()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    # freed while the side stream still writes them
    own = slice(1, None) if name == "shard" else slice(None)   # the ids are a view of the batch's
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = call(side)[own]
    taken = {x.data_ptr() for x in got}
    sizes = [(x.shape, x.dtype) for x in got]
    del got
    again = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in sizes]
    assert not side.query()
    assert not taken & {x.data_ptr() for x in again}
    torch.cuda.synchronize()


def test_given_outputs_make_no_stream_wait():
    b = wl.prefill_512()
    cu = dev(b.cu_seqlens)
    req, local = (torch.empty(b.num_tokens, dtype=torch.int32, device="cuda") for _ in range(2))
    want = oracle.token_index(b.cu_seqlens, b.num_requests, b.num_tokens, False)
    ple.ple_build_token_index(cu, b.num_requests, b.num_tokens, False, req=req, local=local)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    ple.ple_build_token_index(cu, b.num_requests, b.num_tokens, False, req=req, local=local,
                              stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert np.array_equal(req.cpu().numpy(), want[0])
    assert np.array_equal(local.cpu().numpy(), want[1])
