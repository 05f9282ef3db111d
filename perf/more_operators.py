"""The operators of speculation over trees of drafted tokens, as cases that can be timed and compared.

Four operators, one module of the package (``draft_verify_acceptance_gb300.tree``):

  attention   queries of a tree's N nodes over a paged key-value cache: each sees the context, its ancestors and itself
  append      new tokens' keys rotated by their positions and written into their pages with the values; queries rotated
  accept      the walk from a tree's root along the children that the target's tokens name
  keep        the accepted nodes' keys and values moved to the front of the tree's slots, all layers

A tree's node i is the token at slot lengths - N + i of its sequence; parents [B, N] hold each node's parent (a lower index),
-1 for a child of the context, -2 for no node at all.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the package's calls.
``run`` returns every output of a pass, the updated pools among them.
"""
import math

import torch

own = False

DEV = "cuda"


# ---- the cases ------------------------------------------------------------------------------------

def listed():
    return [
        # four small trees over short sequences in a small test model, fp32: latency counts
        {"name": "attention_tiny_f32", "op": "attention", "dtype": "f32", "B": 4, "N": 13, "Hq": 4, "Hkv": 2, "D": 64, "S": 16,
         "len_min": 13, "len_max": 190, "branch": 3, "pad": False},
        # one user's verify step, 59 drafted tokens and the root: eight items of 240 rows to share out
        {"name": "attention_one_bf16", "op": "attention", "dtype": "bf16", "B": 1, "N": 60, "Hq": 32, "Hkv": 8, "D": 128, "S": 16,
         "len_min": 2111, "len_max": 2111, "branch": 6, "pad": False},
        # a served batch with small trees: 64 rows a cache head, the cache's bytes bound
        {"name": "attention_batch_bf16", "op": "attention", "dtype": "bf16", "B": 64, "N": 16, "Hq": 32, "Hkv": 8, "D": 128, "S": 16,
         "len_min": 400, "len_max": 4000, "branch": 4, "pad": True},
        # half the batch with four times the nodes: 256 rows a cache head, products as long as the bytes
        {"name": "attention_wide_bf16", "op": "attention", "dtype": "bf16", "B": 32, "N": 64, "Hq": 32, "Hkv": 8, "D": 128, "S": 16,
         "len_min": 400, "len_max": 4000, "branch": 8, "pad": True},
        # two very long sequences: the work has to be split over the length
        {"name": "attention_long_bf16", "op": "attention", "dtype": "bf16", "B": 2, "N": 26, "Hq": 32, "Hkv": 8, "D": 128, "S": 64,
         "len_min": 60001, "len_max": 131072, "branch": 4, "pad": False},
        # one sequence's small tree in a small test model, pairs side by side
        {"name": "append_tiny_f32", "op": "append", "dtype": "f32", "B": 1, "n_min": 13, "n_max": 13, "Hq": 4, "Hkv": 2, "D": 64, "S": 16,
         "rot": 64, "before_max": 170, "branch": 3, "interleaved": True, "far": 0},
        # one layer's new tokens of the served batch's trees, at their depths
        {"name": "append_trees_bf16", "op": "append", "dtype": "bf16", "B": 64, "n_min": 16, "n_max": 16, "Hq": 32, "Hkv": 8, "D": 128,
         "S": 16, "rot": 128, "before_max": 4000, "branch": 4, "interleaved": False, "far": 0},
        # one layer of a batch of prompts of ragged length behind far contexts, at their places in the cache
        {"name": "append_prompts_bf16", "op": "append", "dtype": "bf16", "B": 12, "n_min": 301, "n_max": 7001, "Hq": 32, "Hkv": 8, "D": 128,
         "S": 16, "rot": 128, "before_max": 333, "branch": 0, "interleaved": False, "far": 900000},
        # the small test model's trees
        {"name": "accept_tiny", "op": "accept", "B": 4, "N": 13, "branch": 3, "pad": False, "hit": 0.7},
        # a best-of-N batch's trees
        {"name": "accept_batch", "op": "accept", "B": 512, "N": 64, "branch": 8, "pad": True, "hit": 0.8},
        # the accepted nodes of one user's tree in a small model of four layers
        {"name": "keep_one_f32", "op": "keep", "dtype": "f32", "B": 1, "N": 13, "L": 4, "Hkv": 2, "D": 64, "S": 16, "len_min": 100,
         "len_max": 190, "branch": 3, "hit": 0.8},
        # the served batch's accepted nodes, sixteen layers
        {"name": "keep_batch_bf16", "op": "keep", "dtype": "bf16", "B": 64, "N": 64, "L": 16, "Hkv": 8, "D": 128, "S": 16, "len_min": 70,
         "len_max": 160, "branch": 4, "hit": 0.9},
    ]


def _span(rng, lo, hi):
    """An integer between lo and hi, spread over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attention", "attention", "attention", "attention", "append", "append", "accept", "keep"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op == "attention":
        hkv = rng.choice((1, 2, 4, 8))
        g = rng.choice((1, 2, 3, 4, 5, 7, 8))
        d = rng.choice((64, 128, 128))
        n = _span(rng, 1, 200)
        b = _span(rng, 1, 64)
        # bounded by the largest listed case's bytes and arithmetic (fp32: a fifth of it)
        most = min(131072, int(0.7e9 / (b * hkv * d * (8 if dtype == "f32" else 4))),
                   int((1.4e10 if dtype == "f32" else 7e10) / (4 * b * n * hkv * g * d)))
        most = max(most, n + 1)
        hi = max(n, _span(rng, min(64, most), most))
        return {"op": op, "dtype": dtype, "B": b, "N": n, "Hq": hkv * g, "Hkv": hkv, "D": d, "S": rng.choice((8, 16, 16, 32, 64, 128)),
                "len_min": max(n, int(hi * rng.uniform(0.05, 1.0))), "len_max": hi, "branch": rng.randint(1, 9),
                "pad": rng.choice((True, False))}
    if op == "append":
        b = _span(rng, 1, 128)
        tree = rng.choice((True, False))
        n = _span(rng, 1, 200 if tree else min(7000, 40000 // b))
        d = rng.choice((64, 128))
        hkv = rng.choice((1, 2, 4, 8))
        return {"op": op, "dtype": dtype, "B": b, "n_min": n if tree else rng.randint(0, n), "n_max": n, "Hq": hkv * rng.choice((1, 3, 4)),
                "Hkv": hkv, "D": d, "S": rng.choice((8, 16, 32, 64)), "rot": rng.choice((d, d, d // 2)),
                "before_max": _span(rng, 1, 4000 if b < 32 else 500), "branch": rng.randint(1, 9) if tree else 0,
                "interleaved": rng.choice((True, False)), "far": rng.choice((0, 0, 100000, 1000000))}
    if op == "accept":
        return {"op": op, "B": _span(rng, 1, 512), "N": _span(rng, 1, 64), "branch": rng.randint(1, 9), "pad": rng.choice((True, False)),
                "hit": rng.uniform(0.2, 0.98)}
    n = _span(rng, 1, 64)
    return {"op": op, "dtype": dtype, "B": _span(rng, 1, 64), "N": n, "L": rng.choice((1, 2, 4, 8)), "Hkv": rng.choice((1, 2, 8)),
            "D": rng.choice((64, 128)), "S": rng.choice((8, 16, 32)), "len_min": n, "len_max": n + _span(rng, 1, 96),
            "branch": rng.randint(1, 9), "hit": rng.uniform(0.3, 0.98)}


# ---- inputs ---------------------------------------------------------------------------------------

def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _pages(n, S):
    return (n + S - 1) // S


def _tables(pages, M, P, g):
    """A page table [B, M] of distinct random pages, `pages` [B] (host list) of them used a row, -1 beyond."""
    ids = torch.randperm(P, generator=g, device=DEV)[:sum(pages)].to(torch.int32)
    count = torch.tensor(pages, device=DEV)
    used = torch.arange(M, device=DEV)[None] < count[:, None]
    table = torch.full((len(pages), M), -1, dtype=torch.int32, device=DEV)
    table.masked_scatter_(used, ids)
    return table


def _lens(lo, hi, n, seed):
    v = torch.randint(lo, hi + 1, (n,), generator=torch.Generator().manual_seed(seed)).tolist()
    v[-1] = hi
    return v


def _trees(B, N, branch, pad, g):
    """Parents [B, N]: levels of `branch` nodes behind the root, each below one of the level before, more often below its
    first ones, the first below the first; with `pad`, up to a third of the last nodes of a sequence are none."""
    i = torch.arange(N, device=DEV)[None]
    start = 1 + ((i - 1).div(branch, rounding_mode="floor") - 1) * branch  # of the level before
    which = (torch.rand((B, N), generator=g, device=DEV).square() * branch).long() * ((i - 1) % branch > 0)
    parents = torch.where(i <= branch, i.clamp(max=1) - 1, start + which)
    if pad:
        count = N - (torch.rand((B, 1), generator=g, device=DEV) * (N / 3)).long()
        parents = torch.where(i < count, parents, -2)
    return parents.to(torch.int32)


def _tokens(parents, hit, g):
    """Drafted tokens, and the target's token after each node: one of its children's with probability `hit`."""
    B, N = parents.shape
    tokens = torch.randint(0, 128256, (B, N), generator=g, device=DEV)
    drawn = torch.randint(0, 128256, (B, N), generator=g, device=DEV)
    child = torch.full((B, N + 1), N, device=DEV)
    at = torch.where(parents >= 0, parents.long(), N)
    child.scatter_reduce_(1, at, torch.arange(N, device=DEV).expand(B, N), "amin")  # (the first has the deepest line below it)
    child = child[:, :N]
    named = (child < N) & (torch.rand((B, N), generator=g, device=DEV) < hit)
    drawn = torch.where(named, torch.gather(tokens, 1, child.clamp(max=N - 1)), drawn)
    return tokens.to(torch.int32), drawn.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, B = case["op"], case["B"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    state = {"case": dict(case)}
    if op == "accept":
        parents = _trees(B, case["N"], case["branch"], case["pad"], g)
        tokens, drawn = _tokens(parents, case["hit"], g)
        return state | {"parents": parents, "tokens": tokens, "drawn": drawn}
    dt, H, D, S = _type(case), case["Hkv"], case["D"], case["S"]
    pool = lambda *shape: torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dt)  # noqa: E731
    if op == "append":
        n = _lens(case["n_min"], case["n_max"], B, 1)  # the same tokens in all for every seed, in another order
        n = [n[i] for i in torch.randperm(B, generator=torch.Generator().manual_seed(seed)).tolist()]
        before = torch.randint(0, case["before_max"] + 1, (B,), generator=torch.Generator().manual_seed(seed + 1)).tolist()
        lens = [a + b for a, b in zip(n, before)]
        pages = [_pages(a, S) for a in lens]
        P = B * _pages(case["n_max"] + case["before_max"], S) + 5  # a pool for the longest
        starts = [0]
        for a in n:
            starts.append(starts[-1] + a)
        T, Hq = starts[-1], case["Hq"]
        qkv = pool(T, (Hq + 2 * H) * D)  # a fused projection's rows
        q, k, v = qkv.split([Hq * D, H * D, H * D], 1)
        F = case["rot"] // 2
        state |= {"q": q.unflatten(1, (Hq, D)), "k_new": k.unflatten(1, (H, D)), "v_new": v.unflatten(1, (H, D)),
                  "k": pool(P, S, H, D), "v": pool(P, S, H, D), "table": _tables(pages, max(pages) + 1, P, g), "lengths": i32(lens),
                  "starts": i32(starts), "inv_freq": (500000.0 ** (-torch.arange(F, dtype=torch.float64) / F)).float().to(DEV),
                  "positions": None}
        if case["branch"]:  # trees: behind the context by the node's depth
            parents = _trees(B, case["n_max"], case["branch"], False, g)
            depth = ancestors(parents).sum(-1) - 1
            state["positions"] = (depth + i32(before)[:, None] + case["far"]).reshape(-1).to(torch.int32)
        elif case["far"]:  # behind a context that another cache holds
            at = torch.cat([torch.arange(b, b + a) for a, b in zip(n, before)]) + case["far"]
            state["positions"] = at.to(DEV, torch.int32)
        return state
    N = case["N"]
    lens = _lens(max(N, case["len_min"]), case["len_max"], B, seed)
    pages = [_pages(n, S) for n in lens]
    P, M = B * max(pages) + 3, max(pages) + 2
    if op == "attention":
        q = (torch.randn((B, N, case["Hq"], D), generator=g, device=DEV) * 2).to(dt)
        return state | {"q": q, "k": pool(P, S, H, D), "v": pool(P, S, H, D), "table": _tables(pages, M, P, g), "lengths": i32(lens),
                        "parents": _trees(B, N, case["branch"], case["pad"], g)}
    L = case["L"]
    parents = _trees(B, N, case["branch"], False, g)
    tokens, drawn = _tokens(parents, case["hit"], g)
    return state | {"k": pool(L, P, S, H, D), "v": pool(L, P, S, H, D), "table": _tables(pages, M, P, g), "lengths": i32(lens),
                    "path": plain_accept(tokens, parents, drawn)["path"]}


# ---- the plain forms ------------------------------------------------------------------------------

def ancestors(parents):
    """[B, N, N] truth values: is j an ancestor of i, or i itself; all false where node i is none."""
    B, N = parents.shape
    p = parents.long()
    step = torch.zeros((B, N, N + 1), device=p.device)
    i = torch.arange(N, device=p.device).expand(B, N)
    step.scatter_(2, i[..., None], 1.0)
    step.scatter_(2, torch.where(p >= 0, p, N)[..., None], 1.0)
    reach = step[:, :, :N]
    for _ in range(max(1, N.bit_length())):  # paths of doubled length
        reach = (torch.matmul(reach, reach) > 0).float()
    none = (p < -1).float()
    lost = torch.matmul(reach, none[..., None])[..., 0] > 0  # a node below none is none
    return (reach > 0) & ~lost[..., None]


def plain_attention(q, k, v, table, lengths, parents):
    B, N, Hq, D = q.shape
    S, H = k.shape[1], k.shape[2]
    n = int(table.shape[1])
    ids = table.clamp(min=0).long()
    kd = k[ids].reshape(B, n * S, H, D).float()
    vd = v[ids].reshape(B, n * S, H, D).float()
    qd = q.float().reshape(B, N, H, Hq // H, D)
    scores = torch.einsum("bqhgd,bthd->bhgqt", qd, kd) * (1.0 / math.sqrt(D))
    t = torch.arange(n * S, device=q.device)
    node = t[None] - (lengths.long()[:, None] - N)  # [B, T]: which node of the tree a token is
    inside = torch.gather(ancestors(parents), 2, node.clamp(0, N - 1)[:, None].expand(B, N, n * S))
    seen = torch.where((node < 0)[:, None], (parents >= -1)[..., None], inside & (node < N)[:, None])
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    m = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(scores - m)
    z = e.sum(-1, keepdim=True)
    o = torch.einsum("bhgqt,bthd->bqhgd", e / z.clamp(min=1e-38), vd).reshape(B, N, Hq, D)
    lse = (m + torch.log(z))[..., 0].permute(0, 3, 1, 2).reshape(B, N, Hq)
    return {"out": o.to(q.dtype), "lse": lse}


def rotated(x, cos, sin, interleaved):
    """Rows x [T, heads, D] with their first 2 F dimensions turned by cos, sin [T, F]."""
    F = cos.shape[1]
    a = x.float()
    c, s = cos[:, None], sin[:, None]
    if interleaved:
        u, w = a[..., 0:2 * F:2], a[..., 1:2 * F:2]
        turned = torch.stack((u * c - w * s, w * c + u * s), -1).flatten(-2)
    else:
        u, w = a[..., :F], a[..., F:2 * F]
        turned = torch.cat((u * c - w * s, w * c + u * s), -1)
    return torch.cat((turned, a[..., 2 * F:]), -1).to(x.dtype)


def plain_append(q, k_new, v_new, k, v, table, lengths, starts, inv_freq, positions, interleaved):
    T, S = k_new.shape[0], k.shape[1]
    row = torch.arange(T, device=k.device)
    b = (row[:, None] >= starts[None, 1:].long()).sum(1)
    at = lengths.long()[b] - (starts.long()[b + 1] - row)
    slot = table.long()[b, at // S] * S + at % S
    angle = (at if positions is None else positions).double()[:, None] * inv_freq.double()[None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    k.view(-1, *k.shape[2:]).index_copy_(0, slot, rotated(k_new, cos, sin, interleaved))
    v.view(-1, *v.shape[2:]).index_copy_(0, slot, v_new)
    return {"q": rotated(q, cos, sin, interleaved), "k": k, "v": v}


def plain_accept(tokens, parents, drawn):
    B, N = tokens.shape
    p = parents.long()
    i = torch.arange(N, device=p.device)
    named = (p >= 0) & (tokens == torch.gather(drawn, 1, p.clamp(min=0)))  # the target's token after the parent
    twin = (p[:, :, None] == p[:, None]) & (tokens[:, :, None] == tokens[:, None]) & (i[None, None] < i[None, :, None])
    good = (named & ~(twin & named[:, None]).any(-1)) | ((i[None] == 0) & (p == -1))
    above = ancestors(parents)
    on = above[:, i, i] & (good[:, None] | ~above).all(-1)
    order = torch.sort(torch.where(on, i[None], N), 1).values
    path = torch.where(order < N, order, -1)
    out = torch.where(order < N, torch.gather(drawn, 1, order.clamp(max=N - 1)).long(), -1)
    return {"accepted_len": (on.sum(1) - 1).to(torch.int32), "out_tokens": out.to(torch.int32), "path": path.to(torch.int32)}


def plain_keep(k, v, table, lengths, path):
    B, N = path.shape
    S = k.shape[2]
    base = (lengths.long() - N)[:, None]
    j = torch.arange(N, device=k.device)[None].expand(B, N)
    b = torch.arange(B, device=k.device)[:, None].expand(B, N)
    kept = path >= 0
    at, to = (base + path)[kept].long(), (base + j)[kept]
    b = b[kept]
    page, place, dpage, dplace = table.long()[b, at // S], at % S, table.long()[b, to // S], to % S
    k[:, dpage, dplace] = k[:, page, place]
    v[:, dpage, dplace] = v[:, page, place]
    return {"lengths": (base[:, 0] + kept.sum(1)).to(torch.int32), "k": k, "v": v}


# ---- one pass -------------------------------------------------------------------------------------

def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        if op == "attention":
            return plain_attention(s["q"], s["k"], s["v"], s["table"], s["lengths"], s["parents"])
        if op == "append":
            return plain_append(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lengths"], s["starts"], s["inv_freq"],
                                s["positions"], case["interleaved"])
        if op == "accept":
            return plain_accept(s["tokens"], s["parents"], s["drawn"])
        return plain_keep(s["k"], s["v"], s["table"], s["lengths"], s["path"])
    from draft_verify_acceptance_gb300 import tree
    if op == "attention":
        out, lse = tree.tree_attention(s["q"], s["k"], s["v"], s["table"], s["lengths"], s["parents"], return_lse=True)
        return {"out": out, "lse": lse}
    if op == "append":
        q = tree.cache_append_rotated(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lengths"], s["inv_freq"], q=s["q"],
                                      positions=s["positions"], starts=s["starts"], interleaved=case["interleaved"])
        return {"q": q, "k": s["k"], "v": s["v"]}
    if op == "accept":
        r = tree.tree_accept(s["tokens"], s["parents"], s["drawn"])
        return {"accepted_len": r.accepted_len, "out_tokens": r.out_tokens, "path": r.path}
    lengths = tree.cache_keep(s["k"], s["v"], s["table"], s["lengths"], s["path"])
    return {"lengths": lengths, "k": s["k"], "v": s["v"]}


# ---- what a pass cannot do without ----------------------------------------------------------------

def work(case):
    op, B = case["op"], case["B"]
    if op == "accept":
        return {"bytes": 4 * B * (5 * case["N"] + 1), "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    row = case["Hkv"] * case["D"] * e
    if op == "append":
        new = B * (case["n_min"] + case["n_max"]) / 2
        return {"bytes": new * (4 * row + 2 * case["Hq"] * case["D"] * e + 4), "flops": 3 * new * (case["Hq"] + case["Hkv"]) * case["rot"]}
    N = case["N"]
    if op == "attention":
        tokens = B * (max(N, case["len_min"]) + case["len_max"]) / 2
        q = B * N * case["Hq"] * case["D"]
        return {"bytes": 2 * tokens * row + 2 * q * e + q / case["D"] * 4, "flops": 4 * tokens * N * case["Hq"] * case["D"]}
    # of a walk that goes on with probability `hit` while there are levels: the root and, mostly, its first child stay
    levels = -(-(N - 1) // case["branch"])
    moved = B * max(0.0, sum(case["hit"] ** (j + 1) for j in range(1, levels))) if case["branch"] > 1 else 0
    return {"bytes": 4 * case["L"] * moved * row + 4 * B * (N + 2), "flops": 0}


# ---- the same from the definitions, in 64 bits ----------------------------------------------------

def exact_attention(s):
    """Sequence by sequence, head by head, in float64; a node's ancestors by following its parents."""
    q, k, v, table = s["q"], s["k"], s["v"], s["table"].long()
    B, N, Hq, D = q.shape
    S, H = k.shape[1], k.shape[2]
    G = Hq // H
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device=q.device)
    parents = s["parents"].tolist()
    for b, n in enumerate(s["lengths"].tolist()):
        sees = torch.zeros((N, n), dtype=torch.bool)
        for i in range(N):
            line, a = [], i
            while a >= 0:
                line.append(n - N + a)
                a = parents[b][a]
            if a == -1:  # the line ends at the context
                sees[i, :n - N] = True
                sees[i, line] = True
        some = sees.any(1)
        sees, some = sees.to(q.device), some.to(q.device)
        pages = table[b, :-(-n // S)]
        for h in range(H):
            kb, vb = k[pages, :, h].reshape(-1, D)[:n].double(), v[pages, :, h].reshape(-1, D)[:n].double()
            x = q[b, :, h * G:(h + 1) * G].double() @ kb.T / math.sqrt(D)  # [N, G, n]
            x = x.masked_fill(~sees[:, None], -math.inf)
            lse[b, :, h * G:(h + 1) * G] = torch.where(some[:, None], torch.logsumexp(x, -1), -math.inf)
            p = torch.where(some[:, None, None], torch.softmax(x, -1), 0.0)
            out[b, :, h * G:(h + 1) * G] = p @ vb
    return {"out": out, "lse": lse}


def exact_append(s, case):
    """Turned as complex numbers of 64-bit parts; the keys land token by token of each sequence."""
    k = s["k"].double()
    S, D, F = k.shape[1], k.shape[3], case["rot"] // 2
    starts, lens = s["starts"].tolist(), s["lengths"].tolist()
    count = [b - a for a, b in zip(starts, starts[1:])]
    at = torch.cat([torch.arange(n - c, n) for n, c in zip(lens, count)]).to(k.device)
    seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(count)).to(k.device)
    where = at if s["positions"] is None else s["positions"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=k.device), where.double()[:, None] * s["inv_freq"].double())[:, None]

    def full(x):
        x = x.double()
        r = x.clone()
        one, two = (slice(0, 2 * F, 2), slice(1, 2 * F, 2)) if case["interleaved"] else (slice(0, F), slice(F, 2 * F))
        z = torch.complex(x[..., one], x[..., two]) * turn
        r[..., one], r[..., two] = z.real, z.imag
        return r

    k[s["table"].long()[seq, at // S], at % S] = full(s["k_new"])
    return {"q": full(s["q"]), "k": k, "v": None}


def exact(case, seed):
    """The computed outputs in 64 bits; accept and keep choose and move values and compute none."""
    if case["op"] == "attention":
        if 4 * case["B"] * case["len_max"] * case["N"] * case["Hq"] * case["D"] > 4e11:
            return None
        return exact_attention(prepare(case, seed))
    if case["op"] == "append":
        return exact_append(prepare(case, seed), case)
    return None
