"""Speculative decoding over a paged cache, every cache operation on the GPU.

A toy decoder with random weights: token embeddings, layers of attention (no
feed-forward), an output projection.  A step gives each sequence room for a
tree of drafts (kv_resize), writes the drafts' keys and values into its pages,
runs all drafts through the layers (tree_attention), accepts the longest path
of drafts that the model itself would have chosen, keeps that path's keys and
values (kv_compact) and finally branches or drops sequences as a beam search
would (kv_fork).  No page list, length or mask goes through the host.

    python examples/tree_decode.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from copy_reduce_dst_gb300 import tb  # noqa: E402

LAYERS, HEADS, CACHE_HEADS, DIM, VOCABULARY = 2, 8, 2, 64, 50
WIDTH = HEADS * DIM
PAGE, SLOTS, TABLE, PAGES = 16, 4, 16, 80
PARENTS = (-1, -1, 0, 0, 1, 2, 2, 5)  # the draft tree: two first tokens, one path four deep


class Cache:
    """The state of the paged cache: pools, page table, pages held, lengths, counts."""

    def __init__(self):
        shape = (LAYERS, PAGES, PAGE, CACHE_HEADS, DIM)
        self.k, self.v = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        ints = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((SLOTS, TABLE), -1, **ints)
        self.held, self.lens = torch.zeros(SLOTS, **ints), torch.zeros(SLOTS, **ints)
        self.refs, self.status = torch.zeros(PAGES, **ints), torch.zeros(1, **ints)
        self.slot_status = torch.zeros(SLOTS, **ints)
        self.describe()

    def describe(self):
        self.c = tb.kv_cache(self.k, self.v, self.table, self.held, self.lens, self.refs)


class Decoder:
    def __init__(self, ctx, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weights(*shape, scale):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()

        self.ctx, self.cache = ctx, Cache()
        self.embed = weights(VOCABULARY, WIDTH, scale=1.0)
        self.qkv = weights(LAYERS, WIDTH, (HEADS + 2 * CACHE_HEADS) * DIM, scale=WIDTH ** -0.5)
        self.head = weights(WIDTH, VOCABULARY, scale=WIDTH ** -0.5).float()
        self.proj = weights(LAYERS, WIDTH, WIDTH, scale=WIDTH ** -0.5)
        self.workspace = torch.empty(ctx.tree_attention_workspace(self.cache.c, HEADS), dtype=torch.uint8,
                                     device="cuda")

    def forward(self, tokens, mask):
        """Logits [slots, n, vocabulary] of n tokens for each slot, placed after
        its committed ones; mask [slots * n, words] says what they see of one another."""
        cache, n = self.cache, tokens.shape[1]
        self.ctx.kv_resize(cache.c, cache.lens + n, cache.status)
        at = cache.lens[:, None] + torch.arange(n, device="cuda")
        page, place = cache.table.gather(1, at // PAGE).long(), at % PAGE
        q_start = torch.arange(SLOTS + 1, dtype=torch.int32, device="cuda") * n
        x = self.embed[tokens].float()
        for layer in range(LAYERS):
            y = torch.nn.functional.layer_norm(x, (WIDTH,)).bfloat16() @ self.qkv[layer]
            q, k, v = y.view(SLOTS, n, -1, DIM).split((HEADS, CACHE_HEADS, CACHE_HEADS), 2)
            cache.k[layer, page, place], cache.v[layer, page, place] = k, v
            q = q.reshape(SLOTS * n, HEADS, DIM)
            out = torch.empty_like(q)
            self.ctx.tree_attention(cache.c, layer, q, q_start, mask, out, self.workspace)
            x = x + (out.view(SLOTS, n, WIDTH) @ self.proj[layer]).float()
        return torch.nn.functional.layer_norm(x, (WIDTH,)) @ self.head

    def prompt(self, tokens):
        """Commits a prompt [slots, n]; the next token of each slot."""
        n = tokens.shape[1]
        chain = torch.tensor(tb.tree_mask([i - 1 for i in range(n)]), dtype=torch.int32, device="cuda")
        logits = self.forward(tokens, chain.repeat(SLOTS, 1))
        self.cache.lens += n
        return logits[:, -1].argmax(-1)

    def step(self, first, drafts):
        """One speculative step: `first` [slots] is the token already chosen, drafts
        [slots, len(PARENTS)] guesses for those after it.  Commits `first` and the
        drafts that agree with the model; returns (tokens [slots, depth], how many
        of them are real, the next token)."""
        cache, n = self.cache, len(PARENTS) + 1
        # The chosen token is the tree's root; the drafts hang below it.
        tree = [-1] + [p + 1 for p in PARENTS]
        mask = torch.tensor(tb.tree_mask(tree), dtype=torch.int32, device="cuda")
        tokens = torch.cat([first[:, None], drafts], 1)
        choice = self.forward(tokens, mask.repeat(SLOTS, 1)).argmax(-1)  # the token after each node
        # A node is accepted if its parent is and the model chose it there.
        depth = [0] * n
        accepted = torch.ones(SLOTS, n, dtype=torch.bool, device="cuda")
        for i in range(1, n):
            depth[i] = depth[tree[i]] + 1
            accepted[:, i] = accepted[:, tree[i]] & (tokens[:, i] == choice[:, tree[i]])
        depth = torch.tensor(depth, device="cuda")
        last = torch.where(accepted, depth, -1).argmax(1)  # the deepest accepted node, the first such
        path = torch.zeros(SLOTS, n, dtype=torch.int32, device="cuda")  # nodes by depth
        node, parents = last, torch.tensor([0] + tree[1:], device="cuda")
        for _ in range(n):
            path.scatter_(1, depth[node][:, None], node[:, None].to(torch.int32))
            node = parents[node]
        count = (depth[last] + 1).to(torch.int32)
        self.ctx.kv_compact(cache.c, cache.lens.clone(), path, count, cache.slot_status)
        every = torch.arange(SLOTS, device="cuda")
        return tokens.gather(1, path.long()), count, choice[every, last]

    def fork(self, parents):
        """Slot s goes on as slot parents[s]; a negative parent empties it."""
        cache = self.cache
        out = [torch.empty_like(t) for t in (cache.table, cache.held, cache.lens)]
        self.ctx.kv_fork(cache.c, torch.tensor(parents, dtype=torch.int32, device="cuda"), *out, cache.status)
        cache.table, cache.held, cache.lens = out
        cache.describe()


def main(steps=6, seed=0):
    """Decodes a few steps with drafts that are partly right; the tokens of each slot."""
    torch.manual_seed(seed)
    with tb.Context(0) as ctx:
        model = Decoder(ctx, seed)
        prompt = torch.randint(0, VOCABULARY, (1, 21), device="cuda").repeat(SLOTS, 1)
        prompt[:, -1] = torch.arange(SLOTS, device="cuda")
        texts = [row.tolist() for row in prompt]
        first = model.prompt(prompt)
        for step in range(steps):
            # Few tokens to choose from, so that some guesses hit.
            drafts = torch.randint(0, VOCABULARY, (SLOTS, len(PARENTS)), device="cuda")
            if step % 2:  # what a good drafter would propose: the model's own choices
                drafts = oracle_drafts(model, texts, first)
            tokens, count, first = model.step(first, drafts)
            for s, (row, n) in enumerate(zip(tokens.tolist(), count.tolist())):
                texts[s] += row[:n]
            if step == 2:  # slot 1 is dropped for a second copy of slot 0
                model.fork([0, 0, 2, 3])
                texts[1], first[1] = list(texts[0]), first[0]
        torch.cuda.synchronize()
        assert int(model.cache.status) == 0 and not model.cache.slot_status.any()
        assert model.cache.lens.tolist() == [len(t) for t in texts]
        return model, texts, first.tolist()


def oracle_drafts(model, texts, first):
    """Drafts along the tree's deepest path as the model would choose them, by plain greedy decoding."""
    drafts = torch.zeros(SLOTS, len(PARENTS), dtype=torch.long, device="cuda")
    for s in range(SLOTS):
        text = texts[s] + [int(first[s])]
        for node in (0, 2, 5, 7):
            text.append(int(plain_logits(model, text)[-1].argmax()))
            drafts[s, node] = text[-1]
    return drafts


def plain_logits(model, text):
    """The decoder without a cache: one sequence, plain torch operations."""
    x = model.embed[torch.tensor(text, device="cuda")].float()
    n = len(text)
    hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
    for layer in range(LAYERS):
        y = torch.nn.functional.layer_norm(x, (WIDTH,)).bfloat16() @ model.qkv[layer]
        q, k, v = y.view(n, -1, DIM).split((HEADS, CACHE_HEADS, CACHE_HEADS), 1)
        k, v = (t.repeat_interleave(HEADS // CACHE_HEADS, 1).float() for t in (k, v))
        scores = torch.einsum("qhd,khd->hqk", q.float(), k) * DIM ** -0.5
        weights = scores.masked_fill(hidden, float("-inf")).softmax(-1)
        out = torch.einsum("hqk,khd->qhd", weights, v).bfloat16()
        x = x + (out.reshape(n, WIDTH) @ model.proj[layer]).float()
    return torch.nn.functional.layer_norm(x, (WIDTH,)) @ model.head


if __name__ == "__main__":
    model, texts, following = main()
    for s, text in enumerate(texts):
        print(f"slot {s}: {len(text)} tokens, the last {text[-8:]}, next {following[s]}")
