"""Best-of-N serving with speculative decoding over one paged cache.

The first layer of a small transformer with random weights drafts for the whole of it.  Every operator of the
framework's decode side runs as a server would use it:

    prompts         cache_append and paged_attention over their tokens, once per prompt
    best of N       cache_fork: N continuations share the prompt's pages
    draft           K times one token: append, attention, filtered_sample, whose filtered
                    rows are the drafter's distributions
    target          one pass over the K drafted tokens and the one before them, its rows
                    filtered alike
    verify          accepted tokens and the one drawn after them
    trim            cache_fork: what was rejected leaves, room for the next step comes
    reject          rejection_cut on mean log-probabilities every few steps; the prompts'
                    worst continuations end (cache_fork) and the pool is compacted

Both models' layers lie in one cache tensor, so one page table and one fork serve both.

    python examples/speculative_serving.py
"""
import copy
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from draft_verify_acceptance_gb300 import binding, decode  # noqa: E402


class Transformer:
    """Pre-norm decoder with random weights; its keys and values live in layers
    first .. first + layers - 1 of the cache."""

    def __init__(self, vocab, width, layers, first, Hq, H, D, dtype, seed, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        w = lambda *s: (torch.randn(s, generator=g) * s[0] ** -0.5).to(device, dtype)  # noqa: E731
        self.Hq, self.H, self.D, self.first = Hq, H, D, first
        self.embed = w(vocab, width) * vocab ** 0.5
        self.place = w(4096, width) * 4096 ** 0.5 * 0.5
        self.layers = [(w(width, (Hq + 2 * H) * D), w(Hq * D, width), w(width, 2 * width), w(2 * width, width))
                       for _ in range(layers)]
        self.head = w(width, vocab) * 3

    def first_layers(self, layers, first):
        """A drafter: the first layers of this model, with keys and values of their own."""
        m = copy.copy(self)
        m.layers, m.first = self.layers[:layers], first
        return m

    @staticmethod
    def norm(h):
        return torch.nn.functional.rms_norm(h, h.shape[-1:])

    def forward(self, tokens, attend):
        """Logits [B, n, vocab] of tokens [B, n]; ``attend(layer, q, k, v)`` is the attention
        over the cache, and without a layer gives the tokens' positions."""
        B, n = tokens.shape
        h = self.embed[tokens.long()] + self.place[attend(None, None, None, None)]
        for i, (qkv, out, up, down) in enumerate(self.layers):
            x = self.norm(h) @ qkv
            q, k, v = (x[..., a * self.D:b * self.D].unflatten(-1, (b - a, self.D))
                       for a, b in ((0, self.Hq), (self.Hq, self.Hq + self.H), (self.Hq + self.H, self.Hq + 2 * self.H)))
            h = h + attend(self.first + i, q, k, v).flatten(2) @ out
            h = h + torch.relu(self.norm(h) @ up) @ down
        return self.norm(h) @ self.head


class Cache:
    """The paged cache of both models and the sequences in it."""

    def __init__(self, layers, pages, page_size, H, D, max_pages, dtype, device="cuda"):
        shape = (layers, pages, page_size, H, D)
        self.k, self.v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
        self.table = torch.full((1, max_pages), -1, dtype=torch.int32, device=device)
        self.lengths = torch.zeros(1, dtype=torch.int32, device=device)
        self.free = pages

    def fork(self, parents, keep, room):
        r = decode.cache_fork(self.k, self.v, self.table, self.lengths, parents, keep, room, debug=True)
        if int(r.status):
            raise RuntimeError(f"cache_fork: status {int(r.status)}")  # DATA_CACHE_FULL: no pages left
        self.table, self.lengths, self.free = r.page_table, r.lengths, int(r.n_free)

    def compact(self):
        self.table = decode.cache_compact(self.k, self.v, self.table).page_table

    def run(self, model, tokens, rows=slice(None)):
        """Appends tokens [B, n] to the sequences `rows` and returns the model's logits.  The sequences'
        lengths are the caller's to advance: draft and target pass over the same positions."""
        B, n = tokens.shape
        table, lengths = self.table[rows], self.lengths[rows] + n

        def attend(layer, q, k, v):
            if layer is None:
                return lengths[:, None] - n + torch.arange(n, device=tokens.device)
            decode.cache_append(k, v, self.k[layer], self.v[layer], table, lengths)
            return decode.paged_attention(q, self.k[layer], self.v[layer], table, lengths)

        return model.forward(tokens, attend)


def serve(prompts, *, N=4, K=3, steps=8, cut_every=4, alpha=0.5, temperature=0.9, top_k=50, top_p=0.95, vocab=4096,
          dtype=torch.bfloat16, seed=0, pages=2048, page_size=16, drafter=None, target=None):
    """Continues each prompt (a list of tokens) N times and returns a list of (prompt index, tokens, mean
    log-probability), with the share of drafted tokens that were accepted."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    H, D = 2, 64
    target = target or Transformer(vocab, 256, 2, 1, 8, H, D, dtype, seed)
    drafter = drafter or target.first_layers(1, 0)
    longest = max(map(len, prompts)) + steps * (K + 1) + K + 2
    cache = Cache(3, pages, page_size, H, D, -(-longest // page_size), dtype)
    setting = dict(temperature=temperature, top_k=top_k, top_p=top_p)
    verify_at = temperature or 1.0  # rows filtered at temperature 0 hold one token

    # prompts, all but their last token, in both models
    G = len(prompts)
    cache.fork(i32([-1] * G), i32([0] * G), max(map(len, prompts)))
    for b, p in enumerate(prompts):
        if len(p) > 1:
            for m in (drafter, target):
                cache.run(m, i32([p[:-1]]), slice(b, b + 1))
    cache.lengths += i32([len(p) - 1 for p in prompts])

    origin = [b for b in range(G) for _ in range(N)]
    last = i32([prompts[b][-1] for b in origin])
    done, logp = [[] for _ in origin], [0.0] * len(origin)
    cache.fork(i32(origin), cache.lengths[origin].contiguous(), K + 1)
    accepted = drafted = 0
    for step in range(steps):
        B, start = len(origin), cache.lengths.clone()
        x, rows = [last], []
        for i in range(K + 1):  # the last pass only caches the last drafted token
            logits = cache.run(drafter, x[-1][:, None])[:, 0]
            cache.lengths += 1
            if i < K:
                r = decode.filtered_sample(logits, draw(B), return_filtered=True, **setting)
                x.append(r.tokens)
                rows.append(r.filtered)
        cache.lengths.copy_(start)
        tokens = torch.stack(x, 1)
        r = decode.filtered_sample(cache.run(target, tokens).contiguous(), draw(B, K + 1), return_filtered=True, **setting)
        n, out = binding.verify(r.filtered, torch.stack(rows, 1), tokens[:, 1:].contiguous(), draw(B, K + 1), verify_at)
        # what the tokens' probabilities were among those that the target keeps
        p = torch.log_softmax(r.filtered.float() / verify_at, -1).gather(2, out.clamp(min=0).long()[..., None])[..., 0]
        last = out.gather(1, n.long()[:, None])[:, 0].contiguous()
        cache.lengths.copy_(start + K + 1)
        cache.fork(torch.arange(B, dtype=torch.int32, device="cuda"), start + 1 + n, K + 1)
        for b, (m, o, q) in enumerate(zip(n.tolist(), out.tolist(), p.tolist())):
            done[b] += o[:m + 1]
            logp[b] += sum(q[:m + 1])
            accepted, drafted = accepted + m, drafted + K
        if cut_every and (step + 1) % cut_every == 0 and step + 1 < steps:
            # each prompt keeps its better continuations (all have the same number left)
            scores = torch.tensor([s / len(d) for s, d in zip(logp, done)], device="cuda").view(G, -1)
            _, left, index = binding.rejection_cut(scores, alpha)
            per = scores.shape[1]
            most = min(left.tolist())
            kept = [b * per + i for b, row in enumerate(index.tolist()) for i in row[:most]]
            cache.fork(i32(kept), cache.lengths[kept].contiguous(), K + 1)
            cache.compact()
            origin, done, logp = ([v[i] for i in kept] for v in (origin, done, logp))
            last = last[kept].contiguous()
    return [(b, d, s / len(d)) for b, d, s in zip(origin, done, logp)], accepted / drafted


def main():
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 4096, (n,), generator=g).tolist() for n in (1, 17, 100, 431)]
    results, rate = serve(prompts)
    for b, tokens, score in results:
        print(f"prompt {b}: {len(tokens)} tokens, mean log-probability {score:.2f}: {tokens[:8]} ...")
    print(f"{100 * rate:.0f}% of the drafted tokens accepted")


if __name__ == "__main__":
    main()
