"""A step that keeps no node at all: a path of no columns."""

import numpy as np
import pytest
import torch

import layer_gram_embedding_gb300 as ple
from layer_gram_embedding_gb300 import build
from test_tree_abi import FIELDS, GOOD
from test_tree_commit_overlap import AT


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ple.lib()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are no memory")
@pytest.mark.parametrize("path_len,path,status", [
    (0, 0, ple.PLE_ERR_CUDA),          # past the checks: without a device the launch is what fails
    (0, AT["path"], ple.PLE_ERR_SIZE), (1, 0, ple.PLE_ERR_NULL), (-1, 0, ple.PLE_ERR_SIZE)])
def test_host_checks(lib, path_len, path, status):
    packer, fields = FIELDS["ple_tree_commit"]
    values = dict(GOOD["ple_tree_commit"], **AT)
    values.update(path_len=path_len, path=path)
    assert lib.ple_tree_commit(packer.pack(*(values[f] for f in fields)), None) == status


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
@pytest.mark.parametrize("kind", [np.int32, np.int64])
def test_nothing_is_kept(kind):
    from test_tree_ops import Cache, dev

    rng = np.random.default_rng(71)
    cache = Cache(rng, [26, 9, 3], 16, 2, 64, torch.bfloat16, layers=2)
    for r, n in enumerate((26, 9, 3)):
        cache.fill(rng, r, 0, n)
    old = cache.k.clone(), cache.v.clone()
    ids, context = rng.integers(0, 1000, 8).astype(kind), rng.integers(0, 1000, (3, 4)).astype(kind)
    ctx = np.array([20, 8, 2], np.int32)
    wide = torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    for path in (torch.zeros((3, 0), dtype=torch.int32, device="cuda"), wide[:, :0].contiguous()):
        nxt, lens = ple.ple_tree_commit(dev(ids), path, dev(np.array([3, 0, 1], np.int32)),
                                        dev(np.array([0, 6, 7, 8], np.int32)), dev(context),
                                        dev(ctx), dev(cache.table), cache.k, cache.v)
        assert np.array_equal(nxt.cpu().numpy(), context)
        assert np.array_equal(lens.cpu().numpy(), ctx)
        for now, before in zip((cache.k, cache.v), old):
            assert torch.equal(now.nan_to_num(), before.nan_to_num())
