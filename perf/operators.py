"""The decode-side operators around the verify step, as cases that can be timed and compared.

Five operators, one module of the package (``draft_verify_acceptance_gb300.decode``):

  attention   queries of the newest Q tokens of each sequence over a paged key-value cache
  append      the newest tokens' keys and values written into their pages
  fork        the next step's sequences from the current ones: shared, trimmed, forked, freed and
              newly reserved pages, partly filled shared pages copied
  compact     live pages moved to the front of the pool, page table rewritten
  sample      temperature, top-k, min-p and top-p from given uniforms

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the package's calls.
``run`` returns every output of a pass, the updated pools among them.
"""
import math

import torch

own = False

DEV = "cuda"
LOG2E = 1.4426950216293335  # log2(e) rounded to 32 bits
# 2^f on [-1/2, 1/2], relative error below 2e-7 in 32-bit arithmetic (constant term 1); part of the
# sampler's definition: see sample_weights
POLY = (0.6931470036506653, 0.24022242426872253, 0.05550733581185341, 0.009671513922512531,
        0.0013264728477224708)
# request settings of a mixed batch: temperature, top-k (0: off), top-p (1: off), min-p (0: off)
SETTINGS = ((1.0, 0, 1.0, 0.0), (0.7, 50, 0.95, 0.0), (0.8, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05),
            (0.6, 20, 0.8, 0.02), (0.0, 0, 1.0, 0.0), (1.2, 400, 1.0, 0.0), (0.9, 0, 0.6, 0.01))


# ---- the cases ------------------------------------------------------------------------------------

def listed():
    return [
        # a verify step's attention in a small test model, fp32: four short sequences, latency counts
        {"name": "attention_tiny_f32", "op": "attention", "dtype": "f32", "B": 4, "Q": 5, "Hq": 4, "Hkv": 2,
         "D": 64, "S": 16, "len_min": 5, "len_max": 190},
        # the target's verify step of a served batch: K = 5 drafted tokens and the one before them
        {"name": "attention_verify_bf16", "op": "attention", "dtype": "bf16", "B": 64, "Q": 6, "Hq": 32, "Hkv": 8,
         "D": 128, "S": 16, "len_min": 400, "len_max": 4000},
        # one new token each for three very long sequences: the work has to be split over the length
        {"name": "attention_long_bf16", "op": "attention", "dtype": "bf16", "B": 3, "Q": 1, "Hq": 32, "Hkv": 8,
         "D": 128, "S": 64, "len_min": 60001, "len_max": 131072},
        # one layer's keys and values of a verify step
        {"name": "append_step_bf16", "op": "append", "dtype": "bf16", "B": 64, "n_min": 6, "n_max": 6, "Hkv": 8,
         "D": 128, "S": 16, "before_max": 4000},
        # one layer's keys and values of a batch of prompts of ragged length
        {"name": "append_prompts_bf16", "op": "append", "dtype": "bf16", "B": 12, "n_min": 301, "n_max": 7001,
         "Hkv": 8, "D": 128, "S": 16, "before_max": 333},
        # the end of a verify step: the rejected tokens leave the cache, room for the next step is reserved
        {"name": "fork_commit_bf16", "op": "fork", "dtype": "bf16", "G": 64, "N": 1, "L": 2, "Hkv": 8, "D": 128,
         "S": 16, "len_min": 40, "len_max": 1000, "drop": 5, "room": 6},
        # best-of-N: eight prompts become 64 sequences each, pages shared up to the last, partly filled one
        {"name": "fork_best_of_n_bf16", "op": "fork", "dtype": "bf16", "G": 8, "N": 64, "L": 4, "Hkv": 8, "D": 128,
         "S": 32, "len_min": 300, "len_max": 8000, "drop": 0, "room": 33},
        # a small test model's pool after some sequences ended
        {"name": "compact_tiny_f32", "op": "compact", "dtype": "f32", "B": 7, "L": 1, "Hkv": 2, "D": 64, "S": 16,
         "P": 97, "live": 0.45},
        # a server's pool after a rejection cut dropped half of its sequences
        {"name": "compact_pool_bf16", "op": "compact", "dtype": "bf16", "B": 48, "L": 4, "Hkv": 8, "D": 128, "S": 16,
         "P": 4096, "live": 0.5},
        # four rows of a small test vocabulary: latency counts
        {"name": "sample_tiny_f32", "op": "sample", "dtype": "f32", "R": 4, "V": 1000, "std": 3.0, "zipf": 0.0,
         "settings": 2, "filtered": False},
        # the verify batch's target rows, each request with settings of its own, filtered rows for the verifier
        {"name": "sample_mixed_bf16", "op": "sample", "dtype": "bf16", "R": 384, "V": 128256, "std": 4.0,
         "zipf": 1.1, "settings": -1, "filtered": True},
        # the best-of-N batch's drafter rows, top-p alone
        {"name": "sample_top_p_bf16", "op": "sample", "dtype": "bf16", "R": 4096, "V": 32000, "std": 3.0, "zipf": 0.0,
         "settings": 2, "filtered": False},
    ]


def _span(rng, lo, hi):
    """An integer between lo and hi, spread over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attention", "attention", "attention", "sample", "sample", "sample", "append", "fork", "compact"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op == "attention":
        hkv = rng.choice((1, 2, 4, 8))
        g = rng.choice((1, 2, 3, 4, 5, 7, 8))
        d = rng.choice((64, 128, 128))
        q = rng.choice((1, 1, 1, 2, 4, 5, 6, 9, 17))
        b = _span(rng, 1, 128)
        rows = q * g
        # bounded by the largest listed case's bytes, and for long drafts by its arithmetic
        most = min(131072, int(1.2e9 / (b * hkv * d * 4 * (4 if dtype == "f32" else 1))), int(3e11 / (b * hkv * rows * d * 4)))
        hi = max(q, _span(rng, min(64, max(1, most)), max(64, most)))
        return {"op": op, "dtype": dtype, "B": b, "Q": q, "Hq": hkv * g, "Hkv": hkv, "D": d,
                "S": rng.choice((8, 16, 16, 32, 64, 128)), "len_min": max(1, int(hi * rng.uniform(0.05, 1.0))), "len_max": hi}
    if op == "append":
        b = _span(rng, 1, 128)
        n = _span(rng, 1, min(8192, 42000 // b))
        return {"op": op, "dtype": dtype, "B": b, "n_min": rng.randint(0, n), "n_max": n, "Hkv": rng.choice((1, 2, 4, 8)),
                "D": rng.choice((64, 128)), "S": rng.choice((8, 16, 32, 64)), "before_max": _span(rng, 1, 4000 if b < 64 else 500)}
    if op == "fork":
        g = _span(rng, 1, 64)
        n = _span(rng, 1, max(1, 512 // g))
        hi = _span(rng, 20, min(8000, 64000 // g))
        return {"op": op, "dtype": dtype, "G": g, "N": n, "L": rng.choice((1, 2, 4)), "Hkv": rng.choice((1, 2, 8)),
                "D": rng.choice((64, 128)), "S": rng.choice((8, 16, 32)), "len_min": max(8, hi // 9), "len_max": hi,
                "drop": rng.randint(0, 7), "room": rng.choice((0, 1, 5, 17, 33))}
    if op == "compact":
        return {"op": op, "dtype": dtype, "B": _span(rng, 1, 64), "L": rng.choice((1, 2, 4)), "Hkv": rng.choice((1, 2, 8)),
                "D": rng.choice((64, 128)), "S": rng.choice((8, 16)), "P": _span(rng, 33, 4001 if dtype == "bf16" else 2000),
                "live": rng.uniform(0.1, 0.95)}
    whole = rng.choice((1, 8, 8))  # odd vocabularies too
    v = _span(rng, 500, 152064) // whole * whole
    r = _span(rng, 1, min(4096, 49_000_000 // v))
    return {"op": op, "dtype": dtype, "R": r, "V": v, "std": rng.uniform(2.0, 5.0), "zipf": rng.choice((0.0, 1.1)),
            "settings": rng.randint(-1, len(SETTINGS) - 1), "filtered": rng.choice((True, False))}


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


def _lens(lo, hi, n, seed, exact_max):
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(lo, hi + 1, (n,), generator=g).tolist()
    if exact_max:
        v[-1] = hi
    return v


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt, op = _type(case), case["op"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    state = {"case": dict(case)}
    if op == "sample":
        R, V = case["R"], case["V"]
        x = torch.randn((R, V), generator=g, device=DEV) * case["std"]
        if case["zipf"]:
            x -= case["zipf"] * torch.log(torch.arange(1, V + 1, dtype=torch.float32, device=DEV))
        which = [case["settings"]] * R if case["settings"] >= 0 else [i % len(SETTINGS) for i in range(R)]
        rows = [SETTINGS[i] for i in which]
        state |= {"logits": x.to(dt), "uniforms": torch.rand(R, generator=g, device=DEV),
                  "temperature": torch.tensor([r[0] for r in rows], device=DEV), "top_k": i32([r[1] for r in rows]),
                  "top_p": torch.tensor([r[2] for r in rows], device=DEV), "min_p": torch.tensor([r[3] for r in rows], device=DEV)}
        return state
    H, D, S = case["Hkv"], case["D"], case["S"]
    pool = lambda *shape: torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dt)  # noqa: E731
    if op == "attention":
        B, Q = case["B"], case["Q"]
        lens = _lens(max(1, case["len_min"]), case["len_max"], B, seed, True)
        pages = [_pages(n, S) for n in lens]
        P = sum(pages) + 3
        M = max(pages) + 2
        state |= {"q": (torch.randn((B, Q, case["Hq"], D), generator=g, device=DEV) * 2).to(dt),
                  "k": pool(P, S, H, D), "v": pool(P, S, H, D), "table": _tables(pages, M, P, g), "lengths": i32(lens)}
        return state
    if op == "append":
        B = case["B"]
        n = _lens(case["n_min"], case["n_max"], B, seed, True)
        lens = [a + b for a, b in zip(n, _lens(0, case["before_max"], B, seed + 1, False))]
        pages = [_pages(a, S) for a in lens]
        P = B * _pages(case["n_max"] + case["before_max"], S) + 5  # a pool for the longest
        starts = [0]
        for a in n:
            starts.append(starts[-1] + a)
        state |= {"k_new": pool(starts[-1], H, D), "v_new": pool(starts[-1], H, D), "k": pool(P, S, H, D), "v": pool(P, S, H, D),
                  "table": _tables(pages, max(pages) + 1, P, g), "lengths": i32(lens), "starts": i32(starts)}
        return state
    L = case["L"]
    if op == "fork":
        G, N = case["G"], case["N"]
        lens = _lens(case["len_min"], case["len_max"], G, seed, True)
        pages = [_pages(n, S) for n in lens]
        room = case["room"]
        drop = _lens(0, case["drop"], G * N, seed + 1, False)
        parents = [c // N for c in range(G * N)]
        keep = [lens[p] - d for p, d in zip(parents, drop)]
        M = _pages(case["len_max"] + room, S) + 1
        P = G * _pages(case["len_max"], S) + G * N * (_pages(room, S) + 1) + 9
        state |= {"k": pool(L, P, S, H, D), "v": pool(L, P, S, H, D), "table": _tables(pages, M, P, g), "lengths": i32(lens),
                  "parents": i32(parents), "keep": i32(keep)}
        return state
    if op == "compact":
        B, P = case["B"], case["P"]
        total = max(1, int(P * case["live"]))
        base = _lens(1, 100, B, seed, False)
        M = max(8, 4 * total // B)
        pages = [min(M, total * a // sum(base)) for a in base]
        state |= {"k": pool(L, P, S, H, D), "v": pool(L, P, S, H, D), "table": _tables(pages, M, P, g)}
        if B > 2:  # two sequences share their first pages, as after a fork
            n = min(pages[0], pages[1]) // 2
            state["table"][1, :n] = state["table"][0, :n]
        return state
    raise ValueError(op)


# ---- the plain forms ------------------------------------------------------------------------------

def plain_attention(q, k, v, table, lengths):
    B, Q, Hq, D = q.shape
    S, H = k.shape[1], k.shape[2]
    n = _pages(int(table.shape[1]) * S, S)
    ids = table.clamp(min=0).long()
    kd = k[ids].reshape(B, n * S, H, D).float()
    vd = v[ids].reshape(B, n * S, H, D).float()
    qd = q.float().reshape(B, Q, H, Hq // H, D)
    scores = torch.einsum("bqhgd,bthd->bhgqt", qd, kd) * (1.0 / math.sqrt(D))
    t = torch.arange(n * S, device=q.device)
    last = lengths.long()[:, None] - Q + torch.arange(Q, device=q.device)[None]  # each query's own position
    seen = t[None, None] <= last[:, :, None]
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    m = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(scores - m)
    z = e.sum(-1, keepdim=True)
    o = torch.einsum("bhgqt,bthd->bqhgd", e / z.clamp(min=1e-38), vd).reshape(B, Q, Hq, D)
    lse = (m + torch.log(z))[..., 0].permute(0, 3, 1, 2).reshape(B, Q, Hq)
    return {"out": o.to(q.dtype), "lse": lse}


def plain_append(k_new, v_new, k, v, table, lengths, starts):
    T, S = k_new.shape[0], k.shape[1]
    row = torch.arange(T, device=k.device)
    b = (row[:, None] >= starts[None, 1:].long()).sum(1)
    at = lengths.long()[b] - (starts.long()[b + 1] - row)
    slot = table.long()[b, at // S] * S + at % S
    k.view(-1, *k.shape[2:]).index_copy_(0, slot, k_new)
    v.view(-1, *v.shape[2:]).index_copy_(0, slot, v_new)
    return {"k": k, "v": v}


def plain_fork(k, v, table, lengths, parents, keep, room):
    L, P, S = k.shape[:3]
    B2, M = parents.shape[0], table.shape[1]
    dev = k.device
    keep = keep.long()
    full, tail, need = (keep // S)[:, None], (keep % S)[:, None], ((keep + room + S - 1) // S)[:, None]
    j = torch.arange(M, device=dev)[None].expand(B2, M)
    src = table.long()[parents.long()]
    at = src.clamp(min=0)
    isfull, istail = j < full, (j == full) & (tail > 0)
    refs = torch.zeros(P, dtype=torch.long, device=dev).scatter_add_(0, at.reshape(-1), isfull.long().reshape(-1))
    c = torch.arange(B2, device=dev)[:, None].expand(B2, M)
    first = torch.full((P,), B2, device=dev).scatter_reduce_(0, at.reshape(-1), torch.where(istail, c, B2).reshape(-1), "amin")
    stays = istail & (refs[at] == 0) & (first[at] == c)
    refs = refs.scatter_add(0, at.reshape(-1), stays.long().reshape(-1))
    fresh = (j < need) & ~isfull & ~stays
    free = refs == 0
    ids = torch.arange(P, device=dev)
    order = torch.full((P + 1,), -1, device=dev).scatter_(0, torch.where(free, torch.cumsum(free, 0) - 1, P), ids)
    order[P] = -1
    rank = (torch.cumsum(fresh.reshape(-1), 0) - 1).reshape(B2, M)
    page = order[torch.where(fresh, rank, P).clamp(max=P)]
    new = torch.where(isfull | stays, src, torch.where(fresh, page, -1))
    refs = refs.scatter_add(0, page.clamp(min=0).reshape(-1), (fresh & (page >= 0)).long().reshape(-1))
    left = refs == 0
    free_pages = torch.full((P + 1,), -1, device=dev).scatter_(0, torch.where(left, torch.cumsum(left, 0) - 1, P), ids)[:P]
    free_pages = torch.where(ids < left.sum(), free_pages, -1)
    copied = (istail & fresh).nonzero(as_tuple=True)
    a, d, n = src[copied], new[copied], tail[copied[0], 0]
    keepers = (torch.arange(S, device=dev)[None] < n[:, None])[None, :, :, None, None]
    k[:, d] = torch.where(keepers, k[:, a], k[:, d])
    v[:, d] = torch.where(keepers, v[:, a], v[:, d])
    i = lambda x: x.to(torch.int32)  # noqa: E731
    return {"table": i(new), "lengths": i(keep), "ref_counts": i(refs), "free_pages": i(free_pages), "n_free": i(left.sum().reshape(1)), "k": k, "v": v}


def plain_compact(k, v, table):
    P = k.shape[1]
    dev = k.device
    at = table.long().clamp(min=0).reshape(-1)
    used = (table >= 0).reshape(-1)
    refs = torch.zeros(P, dtype=torch.long, device=dev).scatter_add_(0, at, used.long())
    ids = torch.arange(P, device=dev)
    live = refs > 0
    n = live.sum()
    a = (live & (ids >= n)).nonzero()[:, 0]
    d = (~live & (ids < n)).nonzero()[:, 0]
    to = ids.clone()
    to[a] = d
    k[:, d] = k[:, a]
    v[:, d] = v[:, a]
    new = torch.where(used, to[at], -1).reshape(table.shape)
    moved = torch.zeros(P, dtype=torch.long, device=dev).scatter_(0, torch.where(live, to, P - 1), refs) if P else refs
    moved = torch.where(ids < n, moved, 0)
    return {"table": new.to(torch.int32), "ref_counts": moved.to(torch.int32), "n_live": n.reshape(1).to(torch.int32), "k": k, "v": v}


def sample_weights(x, temperature):
    """The sampler's integer weights: w = round(2^40 * 2^t) of t = (x - max) * (log2(e) / T), every step rounded to 32 bits.

    The definition is in single roundings of named operations so that sums, cuts and draws are exact integers, the same in
    any order and on any machine."""
    M = x.amax(-1, keepdim=True)
    s = torch.div(torch.full_like(temperature, LOG2E), temperature)[:, None]
    t = ((x - M) * s).clamp(min=-64.0)
    n = torch.round(t)
    f = t - n
    p = torch.full_like(f, POLY[4])
    p = p * f + POLY[3]
    p = p * f + POLY[2]
    p = p * f + POLY[1]
    p = p * f + POLY[0]
    p = p * f + 1.0
    scale = ((n.to(torch.int32) + (40 + 127)) << 23).view(torch.float32)
    return torch.round(p * scale).to(torch.int64)


def scaled_floor(u, S):
    """floor(u * S) exactly, for 32-bit u in [0, 1) and whole S below 2^62."""
    m, e = torch.frexp(u)
    m, sh = (m * 16777216.0).to(torch.int64), (24 - e).to(torch.int64)  # u = m * 2^-sh, sh >= 24
    a, low = m * (S >> 32), m * (S & 0xffffffff)
    a, low = a + (low >> 32), low & 0xffffffff
    small = (a << (32 - sh).clamp(0, 8)) | (low >> sh.clamp(24, 32))
    return torch.where(sh < 32, small, a >> (sh - 32).clamp(0, 63))


def plain_sample(logits, uniforms, temperature, top_k, top_p, min_p, filtered):
    R, V = logits.shape
    x = logits.float() + 0.0
    greedy = temperature == 0
    w = sample_weights(x, torch.where(greedy, 1.0, temperature))
    value, order = torch.sort(x, dim=-1, descending=True, stable=True)
    ws = torch.gather(w, 1, order)
    k = torch.where(greedy, 1, torch.where((top_k <= 0) | (top_k > V), V, top_k))
    least = torch.round(min_p.clamp(0.0, 1.0) * 1099511627776.0).to(torch.int64)
    base = (torch.arange(V, device=x.device)[None] < k[:, None]) & (ws >= least[:, None])
    ws = torch.where(base, ws, 0)
    total = ws.sum(-1)
    need = torch.where(top_p >= 1.0, total, scaled_floor(top_p.clamp(0.0, 0.99999994), total).clamp(min=1))
    run = torch.cumsum(ws, -1)
    kept = base & (run - ws < need[:, None]) & (ws > 0)
    chosen = torch.zeros_like(kept).scatter_(1, order, kept)
    w = torch.where(chosen, w, 0)
    c = torch.cumsum(w, -1)
    theta = scaled_floor(uniforms, c[:, -1])
    token = (c <= theta[:, None]).sum(-1)
    p = torch.gather(w, 1, token[:, None])[:, 0].float() / c[:, -1].float()
    out = {"tokens": token.to(torch.int32), "p": p, "n_kept": chosen.sum(-1).to(torch.int32)}
    if filtered:
        out["filtered"] = torch.where(chosen, logits, torch.full_like(logits, -math.inf))
    return out


# ---- one pass -------------------------------------------------------------------------------------

def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        if op == "attention":
            return plain_attention(s["q"], s["k"], s["v"], s["table"], s["lengths"])
        if op == "append":
            return plain_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lengths"], s["starts"])
        if op == "fork":
            return plain_fork(s["k"], s["v"], s["table"], s["lengths"], s["parents"], s["keep"], case["room"])
        if op == "compact":
            return plain_compact(s["k"], s["v"], s["table"])
        return plain_sample(s["logits"], s["uniforms"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], case["filtered"])
    from draft_verify_acceptance_gb300 import decode
    if op == "attention":
        out, lse = decode.paged_attention(s["q"], s["k"], s["v"], s["table"], s["lengths"], return_lse=True)
        return {"out": out, "lse": lse}
    if op == "append":
        decode.cache_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lengths"], starts=s["starts"])
        return {"k": s["k"], "v": s["v"]}
    if op == "fork":
        r = decode.cache_fork(s["k"], s["v"], s["table"], s["lengths"], s["parents"], s["keep"], room=case["room"])
        return {"table": r.page_table, "lengths": r.lengths, "ref_counts": r.ref_counts, "free_pages": r.free_pages,
                "n_free": r.n_free, "k": s["k"], "v": s["v"]}
    if op == "compact":
        r = decode.cache_compact(s["k"], s["v"], s["table"])
        return {"table": r.page_table, "ref_counts": r.ref_counts, "n_live": r.n_live, "k": s["k"], "v": s["v"]}
    r = decode.filtered_sample(s["logits"], s["uniforms"], s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                               min_p=s["min_p"], return_filtered=case["filtered"])
    out = {"tokens": r.tokens, "p": r.p, "n_kept": r.n_kept}
    if case["filtered"]:
        out["filtered"] = r.filtered
    return out


# ---- what a pass cannot do without ----------------------------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "sample":
        n = case["R"] * case["V"]
        return {"bytes": n * e * (2 if case["filtered"] else 1) + case["R"] * 32, "flops": 0}
    row = case["Hkv"] * case["D"] * e
    if op == "attention":
        tokens = case["B"] * (max(1, case["len_min"]) + case["len_max"]) / 2
        q = case["B"] * case["Q"] * case["Hq"] * case["D"]
        return {"bytes": 2 * tokens * row + 2 * q * e + q / case["D"] * 4,
                "flops": 4 * tokens * case["Q"] * case["Hq"] * case["D"]}
    if op == "append":
        return {"bytes": 4 * case["B"] * (case["n_min"] + case["n_max"]) / 2 * row, "flops": 0}
    S, L = case["S"], case["L"]
    if op == "fork":
        C = case["G"] * case["N"]
        copies = C - case["G"] if case["drop"] == 0 else max(0, C - case["G"])
        avg = (case["len_min"] + case["len_max"]) / 2
        plan = 4 * (C * 2 * avg / S + 2 * C)
        # each source page's half-filled tail read once, each copy written
        return {"bytes": plan + 2 * L * (copies + (case["G"] if case["N"] > 1 else 0)) * (S / 2) * row, "flops": 0}
    live = case["P"] * case["live"]
    return {"bytes": 2 * 2 * L * live * (1 - case["live"]) * S * row + 8 * live, "flops": 0}


# ---- the same from the definitions, in 64 bits ----------------------------------------------------

def exact_attention(s):
    """Sequence by sequence, head by head, in float64: gather the context, soften the scores, weigh the values."""
    q, k, v, table = s["q"], s["k"], s["v"], s["table"].long()
    B, Q, Hq, D = q.shape
    S, H = k.shape[1], k.shape[2]
    out = torch.zeros((B, Q, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((B, Q, Hq), -math.inf, dtype=torch.float64, device=q.device)
    for b, n in enumerate(s["lengths"].tolist()):
        pages = table[b, :-(-n // S)]
        for h in range(H):
            kb, vb = k[pages, :, h].reshape(-1, D)[:n].double(), v[pages, :, h].reshape(-1, D)[:n].double()
            heads = slice(h * (Hq // H), (h + 1) * (Hq // H))
            for i in range(Q):
                end = n - Q + i + 1
                if end > 0:
                    x = q[b, i, heads].double() @ kb[:end].T / math.sqrt(D)
                    lse[b, i, heads] = torch.logsumexp(x, -1)
                    out[b, i, heads] = torch.softmax(x, -1) @ vb[:end]
    return {"out": out, "lse": lse}


def exact_sample(s, case):
    """Row by row with numpy's integers: the weights by their definition, then the cuts and the draw without rounding; p is the
    true softmax of the row over the kept tokens, in float64."""
    import numpy as np
    f = np.float32
    R, V = s["logits"].shape
    tokens, ps, counts = np.zeros(R, np.int32), np.zeros(R), np.zeros(R, np.int32)
    filtered = np.full((R, V), -np.inf) if case["filtered"] else None
    X = s["logits"].float().cpu().numpy()
    par = [s[n].cpu().numpy() for n in ("uniforms", "temperature", "top_k", "top_p", "min_p")]
    for r in range(R):
        x, (u, T, k, p, m) = X[r] + f(0), (a[r] for a in par)
        if T == 0:
            T, k = f(1), 1
        t = np.maximum((x - x.max()) * (f(LOG2E) / f(T)), f(-64))
        n = np.rint(t)
        y = t - n
        g = f(POLY[4])
        for c in (POLY[3], POLY[2], POLY[1], POLY[0], 1.0):
            g = g * y + f(c)
        w = np.rint(np.ldexp(g.astype(np.float64), n.astype(np.int64) + 40)).astype(np.int64)
        if 0 < k < V:  # only the best k can be kept: the k-th value, then its ties by index
            kth = np.partition(x, V - k)[V - k]
            cand = np.flatnonzero(x >= kth)
        else:
            cand = np.arange(V)
        cand = cand[np.argsort(-x[cand], kind="stable")]
        if 0 < k < V:
            cand = cand[:k]
        cand = cand[w[cand] >= int(np.rint(np.float64(min(max(m, 0), 1)) * 2.0 ** 40))]
        cand = cand[w[cand] > 0]
        run = np.cumsum(w[cand])
        if p < 1 and len(cand):
            need = max(1, int(f(max(p, 0)).as_integer_ratio()[0]) * int(run[-1]) // f(max(p, 0)).as_integer_ratio()[1])
            cand = cand[:int(np.searchsorted(run, need, "left")) + 1]
        cand.sort()
        c = np.cumsum(w[cand])
        a, d = f(u).as_integer_ratio()
        j = cand[int(np.searchsorted(c, a * int(c[-1]) // d, "right"))]
        true = np.exp((x[cand].astype(np.float64) - np.float64(x.max())) / np.float64(T))
        tokens[r], counts[r] = j, len(cand)
        ps[r] = np.exp((np.float64(x[j]) - np.float64(x.max())) / np.float64(T)) / true.sum()
        if filtered is not None:
            filtered[r, cand] = X[r, cand]
    out = {"tokens": tokens, "p": ps, "n_kept": counts}
    if filtered is not None:
        out["filtered"] = filtered
    return out


def exact(case, seed):
    """The computed outputs in 64 bits; the cache operators move values and compute none."""
    if case["op"] == "attention":
        if case["B"] * case["Q"] * case["Hkv"] > 12000 or case["B"] * case["len_max"] * case["Q"] * case["Hq"] > 2e8:
            return None
        return exact_attention(prepare(case, seed))
    if case["op"] == "sample":
        return exact_sample(prepare(case, seed), case) if case["R"] * case["V"] <= 140_000_000 else None
    return None
