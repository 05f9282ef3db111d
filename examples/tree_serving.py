"""Serving with trees of drafted tokens over one paged cache.

A small transformer with rotated keys and random weights; its first layer drafts.  Each step of a sequence:

    draft           the drafter grows a tree from the last token, level by level: of all nodes of a level
                    its most likely continuations become the next level (up to `width` of them)
    append          cache_append_rotated: the tree's keys at slots behind the context, rotated by context +
                    depth; the queries rotated with them
    target          tree_attention: one pass over all nodes, each sees the context and its ancestors
    draw            filtered_sample: the target's token after every node
    accept          tree_accept: the path that those tokens take through the tree
    keep            cache_keep: the path's keys and values to the front of the tree's slots
    trim            cache_fork: the pages behind them leave, room for the next tree comes

The emitted tokens follow the target's distribution whatever the drafter proposes: at temperature 0 they are
those of plain greedy decoding.

    python examples/tree_serving.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from draft_verify_acceptance_gb300 import decode, tree  # noqa: E402


class Transformer:
    """Pre-norm decoder with rotated queries and keys and random weights; its keys and values live in layers
    first .. first + layers - 1 of the cache."""

    def __init__(self, vocab, width, layers, Hq, H, D, dtype, seed, first=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        w = lambda *s: (torch.randn(s, generator=g) * s[0] ** -0.5).to(device, dtype)  # noqa: E731
        self.Hq, self.H, self.D, self.first = Hq, H, D, first
        self.embed = w(vocab, width) * vocab ** 0.5
        self.layers = [(w(width, (Hq + 2 * H) * D), w(Hq * D, width), w(width, 2 * width), w(2 * width, width))
                       for _ in range(layers)]
        self.head = w(width, vocab) * 3
        self.inv_freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().to(device)

    def first_layers(self, layers, first):
        """A drafter: the first layers of this model, with keys and values of their own."""
        m = object.__new__(Transformer)
        m.__dict__.update(self.__dict__, layers=self.layers[:layers], first=first)
        return m

    @staticmethod
    def norm(h):
        return torch.nn.functional.rms_norm(h, h.shape[-1:])

    def forward(self, tokens, attend):
        """Logits [B, n, vocab] of tokens [B, n]; ``attend(layer, q, k, v)`` appends and attends."""
        h = self.embed[tokens.long()]
        for i, (qkv, out, up, down) in enumerate(self.layers):
            x = self.norm(h) @ qkv
            q, k, v = (x[..., a * self.D:b * self.D].unflatten(-1, (b - a, self.D))
                       for a, b in ((0, self.Hq), (self.Hq, self.Hq + self.H), (self.Hq + self.H, self.Hq + 2 * self.H)))
            h = h + attend(self.first + i, q, k, v).flatten(2) @ out
            h = h + torch.relu(self.norm(h) @ up) @ down
        return self.norm(h) @ self.head


class Server:
    """Sequences over one cache of `layers` layers, and the trees behind them."""

    def __init__(self, layers, pages, page_size, H, D, max_pages, dtype, device="cuda"):
        shape = (layers, pages, page_size, H, D)
        self.k, self.v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
        self.table = torch.full((1, max_pages), -1, dtype=torch.int32, device=device)
        self.lengths = torch.zeros(1, dtype=torch.int32, device=device)

    def fork(self, parents, keep, room):
        r = decode.cache_fork(self.k, self.v, self.table, self.lengths, parents, keep, room, debug=True)
        if int(r.status):
            raise RuntimeError(f"cache_fork: status {int(r.status)}")
        self.table, self.lengths = r.page_table, r.lengths

    def run(self, model, tokens, parents, depth, rows=slice(None)):
        """The model's logits at the nodes of trees [B, n] behind the sequences `rows`, whose lengths stay."""
        n = tokens.shape[1]
        table, context = self.table[rows], self.lengths[rows]
        lengths = context + n
        positions = (context[:, None] + depth).to(torch.int32).contiguous()

        def attend(layer, q, k, v):
            q = tree.cache_append_rotated(k, v, self.k[layer], self.v[layer], table, lengths, model.inv_freq, q, positions)
            return tree.tree_attention(q, self.k[layer], self.v[layer], table, lengths, parents)

        return model.forward(tokens, attend)


def grow(server, drafter, root, levels, width):
    """The drafter's trees below roots [B]: tokens and parents [B, N], depths [N] (the same number of nodes a level
    for every sequence).  Each pass runs the tree as it is; the last level is not run."""
    B = root.shape[0]
    tokens = root[:, None]
    parents = torch.full((B, 1), -1, dtype=torch.int32, device=root.device)
    depth, score, level = [0], torch.zeros((B, 1), device=root.device), slice(0, 1)
    for d in range(1, levels + 1):
        logits = server.run(drafter, tokens, parents.contiguous(), torch.tensor(depth, device=root.device))[:, level]
        best, token = torch.log_softmax(logits.float(), -1).topk(width, -1)  # of every node of the level
        best = (best + score[:, :, None]).flatten(1)
        score, which = best.topk(min(width, best.shape[1]), -1)
        which = which.sort(-1).values  # nodes in the order of their parents
        score = best.gather(1, which)
        parents = torch.cat((parents, (which // width + level.start).to(torch.int32)), 1)
        tokens = torch.cat((tokens, token.flatten(1).gather(1, which).to(torch.int32)), 1)
        level = slice(level.stop, tokens.shape[1])
        depth += [d] * (level.stop - level.start)
    return tokens.contiguous(), parents.contiguous(), torch.tensor(depth, device=root.device)


def serve(prompts, *, levels=4, width=4, steps=8, temperature=0.0, top_k=None, top_p=None, vocab=2048, dtype=torch.bfloat16, seed=0,
          pages=1024, page_size=16, target=None, drafter=None):
    """Continues each prompt (a list of tokens) and returns the lists of new tokens, with the mean number of
    drafted tokens accepted a step."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(seed)
    H, D = 2, 64
    target = target or Transformer(vocab, 256, 3, 8, H, D, dtype, seed, first=1)
    drafter = drafter or target.first_layers(1, 0)
    N = 1 + levels * width
    longest = max(map(len, prompts)) + (steps + 1) * (levels + 1) + N
    s = Server(4, pages, page_size, H, D, -(-longest // page_size), dtype)

    # prompts, all but their last token: chains, in both models
    B = len(prompts)
    s.fork(i32([-1] * B), i32([0] * B), max(map(len, prompts)))
    for b, p in enumerate(prompts):
        for a in range(0, len(p) - 1, tree.MAX_NODES):  # a tree has no more nodes
            part = i32([p[a:min(a + tree.MAX_NODES, len(p) - 1)]])
            n = part.shape[1]
            chain = torch.arange(-1, n - 1, dtype=torch.int32, device="cuda")
            for m in (drafter, target):
                s.run(m, part, chain, torch.arange(n, device="cuda"), slice(b, b + 1))
            s.lengths[b] += n

    last, done, accepted = i32([p[-1] for p in prompts]), [[] for _ in prompts], 0
    for _ in range(steps):
        s.fork(torch.arange(B, dtype=torch.int32, device="cuda"), s.lengths, N)
        tokens, parents, depth = grow(s, drafter, last, levels, width)
        if drafter is not target:  # the drafter's last level into its cache, for what is accepted of it
            s.run(drafter, tokens, parents, depth)
        logits = s.run(target, tokens, parents, depth).contiguous()
        drawn = decode.filtered_sample(logits, torch.rand(logits.shape[:2], generator=g, device="cuda"), temperature, top_k=top_k,
                                       top_p=top_p).tokens
        r = tree.tree_accept(tokens, parents, drawn)
        s.lengths = tree.cache_keep(s.k, s.v, s.table, s.lengths + tokens.shape[1], r.path)
        last = r.out_tokens.gather(1, r.accepted_len.long()[:, None])[:, 0].contiguous()
        for d, n, out in zip(done, r.accepted_len.tolist(), r.out_tokens.tolist()):
            d += out[:n + 1]
            accepted += n
    return done, accepted / (steps * B)


def main():
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 2048, (n,), generator=g).tolist() for n in (1, 17, 100, 431)]
    done, rate = serve(prompts)
    for b, tokens in enumerate(done):
        print(f"prompt {b}: {len(tokens)} tokens: {tokens[:8]} ...")
    print(f"{rate:.2f} drafted tokens accepted a step")


if __name__ == "__main__":
    main()
