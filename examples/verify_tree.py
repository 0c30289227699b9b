"""A decoding loop that drafts trees of tokens and verifies each in one pass.

A small model with per-layer n-gram embeddings and random weights serves a few
requests.  A cheap drafter proposes a tree of tokens behind each request's last
one; one pass of the model checks all of them:

  ple_build_tree_index   positions and ancestor masks of the trees
  ple_tree_row_ids       the n-gram row ids of every node, along its branch
  ple_qk_norm_rope       norms, rotation and the append to the paged cache
  ple_tree_attention     the nodes over the cache and their own branch
  ple_tree_commit        the accepted branches kept, the next step's state

A prompt is a tree that is a chain, and plain decoding a tree of one node.

  python examples/verify_tree.py
"""

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import layer_gram_embedding_gb300 as ple  # noqa: E402

VOCAB, BOUNDARY = 1000, 7
LAYERS, HIDDEN, Q_HEADS, KV_HEADS, HEAD_DIM = 2, 256, 8, 2, 64
NGRAM, HEADS_PER_NGRAM, PAGE = 3, 2, 16


def rms(x):
    return x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype)


class Model:
    def __init__(self, device, seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def draw(*shape, size):
            return (torch.randn(*shape, generator=gen, device=device) * size).to(torch.bfloat16)

        heads = (NGRAM - 1) * HEADS_PER_NGRAM
        width = (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM
        self.embed = draw(VOCAB, HIDDEN, size=1.0)
        self.qkv = draw(LAYERS, HIDDEN, width, size=HIDDEN ** -0.5)
        self.out = draw(LAYERS, Q_HEADS * HEAD_DIM, HIDDEN, size=0.3 * HIDDEN ** -0.5)
        self.q_weight = 1 + draw(LAYERS, HEAD_DIM, size=0.1)
        self.k_weight = 1 + draw(LAYERS, HEAD_DIM, size=0.1)
        self.head = draw(HIDDEN, VOCAB, size=HIDDEN ** -0.5)
        self.multipliers = torch.randint(-2 ** 62, 2 ** 62, (LAYERS, NGRAM), generator=gen,
                                         device=device) * 2 + 1
        self.vocab_sizes = torch.tensor([[997, 991, 983, 977]] * LAYERS, device=device)
        self.offsets = self.vocab_sizes.cumsum(1) - self.vocab_sizes
        self.tables = draw(LAYERS, int(self.vocab_sizes[0].sum()), HIDDEN, size=0.1)
        # set up once for these parameters
        self.heads = ple.ple_prepare_heads(self.vocab_sizes, self.offsets)
        self.rope = ple.ple_prepare_rope(HEAD_DIM, device=device)
        assert heads == self.vocab_sizes.shape[1]

    def forward(self, ids, parent, cu_seqlens, mask_words, state):
        """Logits [T, VOCAB] of the nodes; their keys and values are appended."""
        positions, mask = ple.ple_build_tree_index(parent, cu_seqlens, state.ctx_lens, mask_words)
        rows = ple.ple_tree_row_ids(ids, parent, cu_seqlens, state.ngram_context,
                                    self.multipliers, self.vocab_sizes, self.offsets, NGRAM,
                                    HEADS_PER_NGRAM, BOUNDARY, heads=self.heads)
        x = self.embed[ids]
        for layer in range(LAYERS):
            x = x + self.tables[layer][rows[layer]].sum(1)
            qkv = (rms(x) @ self.qkv[layer]).reshape(len(ids), -1, HEAD_DIM)
            q, k, v = qkv.split([Q_HEADS, KV_HEADS, KV_HEADS], 1)
            q = ple.ple_qk_norm_rope(q, k, v, positions, self.rope, self.q_weight[layer],
                                     self.k_weight[layer], k_cache=state.k_cache[layer],
                                     v_cache=state.v_cache[layer], page_table=state.page_table,
                                     ctx_lens=state.ctx_lens, cu_seqlens=cu_seqlens)
            seen = ple.ple_tree_attention(q, state.k_cache[layer], state.v_cache[layer],
                                          state.page_table, state.ctx_lens, cu_seqlens, mask)
            x = x + seen.flatten(1) @ self.out[layer]
        return (rms(x) @ self.head).float()

    def draft(self, token):
        """The drafter's two best guesses of what follows each token: the model without its layers."""
        return (rms(self.embed[token]) @ self.head).float().topk(2, -1).indices


class State:
    """What is kept between steps: the paged caches of every layer, cached lengths and the carried contexts."""

    def __init__(self, requests, capacity, device):
        pages = math.ceil(capacity / PAGE)
        shape = (LAYERS, requests * pages, KV_HEADS, PAGE, HEAD_DIM)
        self.k_cache = torch.zeros(shape, dtype=torch.bfloat16, device=device)
        self.v_cache = torch.zeros_like(self.k_cache)
        order = torch.randperm(requests * pages, generator=torch.Generator().manual_seed(1))
        self.page_table = order.reshape(requests, pages).to(torch.int32).to(device)
        self.ctx_lens = torch.zeros(requests, dtype=torch.int32, device=device)
        self.ngram_context = torch.full((requests, NGRAM - 1), BOUNDARY, device=device)

    def commit(self, ids, paths, cu_seqlens):
        longest = max(1, max(map(len, paths)))
        device = ids.device
        path = torch.tensor([p + [0] * (longest - len(p)) for p in paths], dtype=torch.int32,
                            device=device)
        accepted = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=device)
        self.ngram_context, self.ctx_lens = ple.ple_tree_commit(
            ids, path, accepted, cu_seqlens, self.ngram_context, self.ctx_lens, self.page_table,
            self.k_cache, self.v_cache)


def pack(trees, device):
    """Trees [(ids, parents)] as the calls take them."""
    counts = [len(ids) for ids, _ in trees]
    cu = torch.tensor([0] + counts, dtype=torch.int64).cumsum(0).to(torch.int32).to(device)
    ids = torch.tensor([t for i, _ in trees for t in i], device=device)
    parent = torch.tensor([p for _, ps in trees for p in ps], dtype=torch.int32, device=device)
    return ids, parent, cu, (max(counts) + 63) // 64


def chains(token_lists):
    return [(ids, list(range(-1, len(ids) - 1))) for ids in token_lists]


def drafted(model, roots, depth):
    """A tree behind each root: the two best guesses, and behind each of them the same again."""
    trees = []
    for root in roots:
        ids, parents, level = [root], [-1], [0]
        for _ in range(depth):
            guesses = model.draft(torch.tensor([ids[j] for j in level],
                                               device=model.embed.device)).tolist()
            new = []
            for j, pair in zip(level, guesses):
                for token in pair:
                    ids.append(token)
                    parents.append(j)
                    new.append(len(ids) - 1)
            level = new
        trees.append((ids, parents))
    return trees


def accept(trees, chosen):
    """The accepted branch of each tree: from the root on, the child that the model itself chose."""
    paths, at = [], 0
    for ids, parents in trees:
        path = [0]
        while True:
            want = chosen[at + path[-1]]
            child = [j for j, p in enumerate(parents) if p == path[-1] and ids[j] == want]
            if not child:
                break
            path.append(child[0])
        paths.append(path)
        at += len(ids)
    return paths


def generate(model, prompts, steps, depth):
    """Tokens of every request with the logits that chose them, and the number of accepted drafts."""
    device = model.embed.device
    capacity = max(map(len, prompts)) + steps * (depth + 1) + 2 ** (depth + 1)
    state = State(len(prompts), capacity, device)
    trees = chains(prompts)
    tokens, scores, drafts = [[] for _ in prompts], [[] for _ in prompts], 0
    for step in range(steps + 1):
        ids, parent, cu, words = pack(trees, device)
        logits = model.forward(ids, parent, cu, words, state)
        chosen = logits.argmax(-1).tolist()
        # a prompt is kept whole; of a drafted tree the branch that the model agrees with
        paths = [list(range(len(p))) for p in prompts] if step == 0 else accept(trees, chosen)
        state.commit(ids, paths, cu)
        roots, starts = [], cu.tolist()
        for r, path in enumerate(paths):
            answers = path[-1:] if step == 0 else path
            tokens[r] += [chosen[starts[r] + j] for j in answers]
            scores[r] += [logits[starts[r] + j] for j in answers]
            drafts += 0 if step == 0 else len(path) - 1
            roots.append(tokens[r][-1])
        trees = drafted(model, roots, depth)
    return tokens, scores, drafts


def forced(model, prompt, tokens):
    """The logits of plain decoding, one node a step, along given tokens."""
    device = model.embed.device
    state = State(1, len(prompt) + len(tokens) + 1, device)
    out = []
    for ids in [prompt] + [[t] for t in tokens]:
        packed, parent, cu, words = pack(chains([ids]), device)
        out.append(model.forward(packed, parent, cu, words, state)[-1])
        state.commit(packed, [list(range(len(ids)))], cu)
    return out


def main(steps=12, depth=3):
    device = torch.device("cuda")
    model = Model(device)
    gen = torch.Generator().manual_seed(5)
    prompts = [torch.randint(0, VOCAB, (n,), generator=gen).tolist() for n in (5, 70, 33)]
    tokens, scores, drafts = generate(model, prompts, steps, depth)
    count = sum(map(len, tokens))
    print(f"{count} tokens for {len(prompts)} requests in {steps + 1} passes, {drafts} of them "
          f"drafted")
    worst = 0.0
    for r, prompt in enumerate(prompts):
        for a, b in zip(scores[r], forced(model, prompt, tokens[r][:-1])):
            worst = max(worst, float((a - b).abs().max()))
    print(f"logits of the verified trees against plain decoding: at most {worst:.3f} apart")
    return count, drafts, worst


if __name__ == "__main__":
    main()
