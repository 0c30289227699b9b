"""The commit's outputs may share no byte with what it reads, or with each
other: a request's blocks read while another of them writes.  The C ABI says so
without a GPU; the binding names the pair."""

import itertools

import pytest
import torch

import layer_gram_embedding_gb300 as ple
from layer_gram_embedding_gb300 import build
from test_tree_abi import FIELDS, GOOD

# distinct addresses for the arguments of GOOD's sizes, far apart
NAMES = ["input_ids", "path", "accepted", "cu_seqlens", "ngram_context", "next_context", "ctx_lens",
         "next_ctx_lens", "page_table", "k_cache", "v_cache"]
AT = {name: 0x100000 * (i + 1) for i, name in enumerate(NAMES)}
B, T, P, C, MAX_PAGES = 2, 5, 3, 2, 4
BYTES = dict(input_ids=8 * T, path=4 * B * P, accepted=4 * B, cu_seqlens=4 * (B + 1),
             ngram_context=8 * B * C, next_context=8 * B * C, ctx_lens=4 * B, next_ctx_lens=4 * B,
             page_table=4 * B * MAX_PAGES)
PAIRS = [(out, other) for out in ("next_context", "next_ctx_lens") for other in BYTES
         if other != out]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ple.lib()


def call(lib, **kw):
    packer, fields = FIELDS["ple_tree_commit"]
    values = dict(GOOD["ple_tree_commit"], **AT)
    values.update(kw)
    return lib.ple_tree_commit(packer.pack(*(values[f] for f in fields)), None)


@pytest.mark.parametrize("out,other", PAIRS)
def test_c_abi_refuses_every_overlap(lib, out, other):
    step = 8 if out == "next_context" else 4
    for shift in (0, BYTES[other] - step, step - BYTES[out]):
        if (AT[other] + shift) % step == 0:
            assert call(lib, **{out: AT[other] + shift}) == ple.PLE_ERR_SIZE, shift


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are no memory")
def test_c_abi_takes_neighbours(lib):
    # past the checks: without a device the launch is what fails
    assert call(lib) == ple.PLE_ERR_CUDA
    for out, other in PAIRS:
        for at in (AT[other] + BYTES[other], AT[other] - BYTES[out]):
            if at % (8 if out == "next_context" else 4) == 0:
                assert call(lib, **{out: at}) == ple.PLE_ERR_CUDA, (out, other)
    # what is not read without a carried context may lie anywhere
    assert call(lib, ngram_context=0, next_context=AT["ctx_lens"],
                next_ctx_lens=AT["input_ids"]) == ple.PLE_ERR_CUDA


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
def test_binding_names_the_pair():
    from test_tree_ops import make_step

    s = make_step(61)
    given = dict(input_ids=s["ids"], path=s["path"], accepted=s["accepted"], cu_seqlens=s["cu"],
                 ngram_context=s["context"], ctx_lens=s["ctx"], page_table=s["table"])
    cases = {"next_ctx_lens": (torch.int32, given["ctx_lens"].shape),
             "next_context": (torch.int64, given["ngram_context"].shape)}
    for (out, (dtype, shape)), other in itertools.product(cases.items(), given):
        u = given[other]
        n = max(1, shape.numel() * (8 if dtype == torch.int64 else 4) + u.numel() * u.element_size())
        space = torch.zeros((n + 15) // 8 * 8, dtype=torch.uint8, device="cuda")
        # the argument at the start of the space, the output over its last element
        a = space[:u.numel() * u.element_size()].view(u.dtype).view(u.shape)
        a.copy_(u)
        last = (a.numel() - 1) * a.element_size() // 8 * 8
        b = space[last:last + shape.numel() * (8 if dtype == torch.int64 else 4)].view(dtype)
        with pytest.raises(ValueError, match=f"{out} must not overlap {other}"):
            ple.ple_tree_commit(**dict(given, **{other: a, out: b.view(shape)}), k_cache=s["kc"],
                                v_cache=s["vc"])
    for out, other in (("next_ctx_lens", "ctx_lens"), ("next_context", "ngram_context")):
        with pytest.raises(ValueError, match=f"{out} must not overlap {other}"):
            ple.ple_tree_commit(**given, k_cache=s["kc"], v_cache=s["vc"], **{out: given[other]})
    space = torch.zeros(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="next_context must not overlap next_ctx_lens"):
        ple.ple_tree_commit(**given, k_cache=s["kc"], v_cache=s["vc"],
                            next_context=space[:48].view(torch.int64).view(3, 2),
                            next_ctx_lens=space[44:56].view(torch.int32))
