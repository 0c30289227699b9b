"""The binding's memo of workspace sizes: a query that failed is asked again."""

import contextlib
import types

import torch

from layer_gram_embedding_gb300 import tree


def test_a_failed_query_is_not_kept(monkeypatch):
    answers = [-1, 4096, 77]
    asked = []

    def query(*sizes):
        asked.append(sizes)
        return answers.pop(0)

    monkeypatch.setattr(tree, "lib",
                        lambda: types.SimpleNamespace(ple_tree_attention_workspace=query))
    monkeypatch.setattr(tree, "_workspace_sizes", {})
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    assert tree._workspace_size(5, 8, 2, 64, 0) == 0        # the device could not be asked
    assert tree._workspace_size(5, 8, 2, 64, 0) == 4096     # now it could
    assert tree._workspace_size(5, 8, 2, 64, 0) == 4096     # and is not asked again
    assert tree._workspace_size(6, 8, 2, 64, 0) == 77
    assert asked == [(5, 8, 2, 64)] * 2 + [(6, 8, 2, 64)]


def test_the_memo_is_bounded(monkeypatch):
    monkeypatch.setattr(tree, "lib", lambda: types.SimpleNamespace(
        ple_tree_attention_workspace=lambda T, *rest: T))
    monkeypatch.setattr(tree, "_workspace_sizes", {})
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    for T in range(10000):
        assert tree._workspace_size(T, 8, 2, 64, 0) == T
        assert len(tree._workspace_sizes) <= 4096
