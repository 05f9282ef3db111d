"""Plain 64-bit references of the decode-side operators, from their definitions (numpy, loops)."""
import numpy as np

POLY = (0.6931470036506653, 0.24022242426872253, 0.05550733581185341, 0.009671513922512531,
        0.0013264728477224708)


def attention(q, k, v, table, lengths, scale):
    """q [B, Q, Hq, D], k / v [P, S, H, D], all float64.  Returns out, lse, and the bounds' ingredients:
    sum_t p |v| per output and max_t scale * sum_d |q||k| per row."""
    B, Q, Hq, D = q.shape
    P, S, H, _ = k.shape
    out, lse = np.zeros((B, Q, Hq, D)), np.full((B, Q, Hq), -np.inf)
    mag, spread = np.zeros((B, Q, Hq, D)), np.zeros((B, Q, Hq))
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * S)
        pages = table[b, :-(-n // S)]
        ok = np.repeat((pages >= 0) & (pages < P), S)[:n]
        ids = np.clip(pages, 0, P - 1)
        for h in range(Hq):
            kb = k[ids][:, :, h // (Hq // H)].reshape(-1, D)[:n]
            vb = v[ids][:, :, h // (Hq // H)].reshape(-1, D)[:n]
            for i in range(Q):
                end = max(0, min(n, n - Q + i + 1))
                see = np.flatnonzero(ok[:end])
                if not len(see):
                    continue
                x = kb[see] @ q[b, i, h] * scale
                m = x.max()
                e = np.exp(x - m)
                z = e.sum()
                out[b, i, h] = (e / z) @ vb[see]
                lse[b, i, h] = m + np.log(z)
                mag[b, i, h] = (e / z) @ np.abs(vb[see])
                spread[b, i, h] = (np.abs(kb[see]) @ np.abs(q[b, i, h])).max() * abs(scale)
    return out, lse, mag, spread


def fork(table, lengths, parents, keep, room, P, S):
    """Returns (new_table, new_lengths, refs, free, copies); copies: (from, to, tokens)."""
    B, M = table.shape
    C = len(parents)
    kids = []
    for c in range(C):
        p, n = int(parents[c]), int(keep[c])
        if not (0 <= p < B and 0 <= n <= min(int(lengths[p]), M * S)):
            p, n = -1, 0
        kids.append((p, n))
    valid = lambda x: 0 <= x < P  # noqa: E731
    full, first = {}, {}
    for c, (p, n) in enumerate(kids):
        for j in range(n // S):
            if valid(table[p, j]):
                full[table[p, j]] = full.get(table[p, j], 0) + 1
        if n % S and valid(table[p, n // S]):
            first.setdefault(table[p, n // S], c)
    stays = {page: c for page, c in first.items() if page not in full}
    refs = np.zeros(P, np.int64)
    for page, n in full.items():
        refs[page] = n
    for page in stays:
        refs[page] = 1
    free = [p for p in range(P) if refs[p] == 0]
    new, copies = np.full((C, M), -1), []
    for c, (p, n) in enumerate(kids):
        need = min(M, -(-(n + room) // S))
        for j in range(need):
            if j < n // S:
                new[c, j] = table[p, j] if valid(table[p, j]) else -1
            elif j == n // S and n % S and stays.get(table[p, j]) == c:
                new[c, j] = table[p, j]
            elif free:
                new[c, j] = free.pop(0)
                refs[new[c, j]] += 1
                if j == n // S and n % S and valid(table[p, j]):
                    copies.append((int(table[p, j]), int(new[c, j]), n % S))
    return new, np.array([n for _, n in kids]), refs, free, copies


def compact(table, P):
    used = sorted({int(x) for x in table.ravel() if 0 <= x < P})
    n = len(used)
    holes = [p for p in range(n) if p not in set(used)]
    moves = dict(zip([p for p in used if p >= n], holes))
    new = np.array([[moves.get(int(x), int(x)) if 0 <= x < P else -1 for x in row] for row in table]).reshape(table.shape)
    refs = np.bincount(new[new >= 0].ravel(), minlength=P)
    return new, refs, n, moves


def weights(x, T):
    f = np.float32
    t = np.maximum((x - x.max()) * (f(1.4426950216293335) / f(T)), f(-64))
    n = np.rint(t)
    y = t - n
    g = f(POLY[4])
    for c in (POLY[3], POLY[2], POLY[1], POLY[0], 1.0):
        g = g * y + f(c)
    return np.rint(np.ldexp(g.astype(np.float64), n.astype(np.int64) + 40)).astype(np.int64)


def sample_row(x, u, T=1.0, k=0, top_p=1.0, min_p=0.0):
    """(token, p, kept token indices) of one row of float32 logits."""
    x = x.astype(np.float32) + np.float32(0)
    V = len(x)
    if T == 0:
        T, k = 1.0, 1
    with np.errstate(invalid="ignore"):
        w = weights(x, T)
    order = np.argsort(-x, kind="stable")
    if 0 < k < V:
        order = order[:k]
    m = np.float32(min(max(min_p, 0.0), 1.0))
    order = order[w[order] >= max(1, int(np.rint(np.float64(m) * 2.0 ** 40)))]
    run = np.cumsum(w[order])
    if top_p < 1:
        a, d = np.float32(max(top_p, 0.0)).as_integer_ratio()
        need = max(1, a * int(run[-1]) // d)
        order = order[:int(np.searchsorted(run, need, "left")) + 1]
    kept = np.sort(order)
    c = np.cumsum(w[kept])
    a, d = np.float32(u).as_integer_ratio()
    j = int(kept[int(np.searchsorted(c, a * int(c[-1]) // d, "right"))])
    z = np.exp((x[kept].astype(np.float64) - np.float64(x.max())) / np.float64(np.float32(T)))
    return j, float(np.exp((np.float64(x[j]) - np.float64(x.max())) / np.float64(np.float32(T))) / z.sum()), kept
