"""Plain 64-bit references of the tree operators, from their definitions (numpy, loops)."""
import numpy as np


def line(parents, i):
    """Node i and its ancestors, or None when it is no node."""
    out = []
    while True:
        out.append(i)
        p = int(parents[i])
        if p == -1:
            return out
        if p < 0 or p >= i:
            return None
        i = p


def attention(q, k, v, table, lengths, parents, scale):
    """q [B, N, Hq, D], k / v [P, S, H, D], all float64; parents [B, N].  Returns out, lse, and the bounds'
    ingredients: sum_t p |v| per output and max_t scale * sum_d |q||k| per row."""
    B, N, Hq, D = q.shape
    P, S, H, _ = k.shape
    out, lse = np.zeros((B, N, Hq, D)), np.full((B, N, Hq), -np.inf)
    mag, spread = np.zeros((B, N, Hq, D)), np.zeros((B, N, Hq))
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * S)
        pages = table[b, :-(-n // S)]
        ok = np.repeat((pages >= 0) & (pages < P), S)[:n]
        ids = np.clip(pages, 0, P - 1)
        base = n - N
        for h in range(H):
            kb, vb = k[ids][:, :, h].reshape(-1, D)[:n], v[ids][:, :, h].reshape(-1, D)[:n]
            for i in range(N):
                up = line(parents[b], i)
                if up is None or base + i < 0:
                    continue
                see = [t for t in range(max(base, 0)) if ok[t]] + sorted(base + a for a in up if base + a >= 0 and ok[base + a])
                if not see:
                    continue
                ks, vs = kb[see], vb[see]
                for hq in range(h * (Hq // H), (h + 1) * (Hq // H)):
                    x = ks @ q[b, i, hq] * scale
                    m = x.max()
                    e = np.exp(x - m)
                    z = e.sum()
                    out[b, i, hq] = (e / z) @ vs
                    lse[b, i, hq] = m + np.log(z)
                    mag[b, i, hq] = (e / z) @ np.abs(vs)
                    spread[b, i, hq] = (np.abs(ks) @ np.abs(q[b, i, hq])).max() * abs(scale)
    return out, lse, mag, spread


def turns(position, f):
    """The fraction of a turn that position * f radians makes, exactly: for angles that a double loses."""
    def arctan_inv(x):  # arctan(1 / x) * 2^400
        term, total, n = (1 << 400) // x, 0, 1
        while term:
            total += term // n if n % 4 == 1 else -(term // n)
            term //= x * x
            n += 2
        return total
    one_turn = 8 * (4 * arctan_inv(5) - arctan_inv(239))  # 2 pi * 2^400 (Machin)
    num, den = float(f).as_integer_ratio()
    return ((position * num << 800) // (den * one_turn) % (1 << 400)) / (1 << 400)


def rotate(x, position, inv_freq, interleaved):
    """Heads x [..., D] of one token, and the bound's ingredient |x| + |y| of each pair."""
    F = len(inv_freq)
    a = float(position) * inv_freq.astype(np.float64)
    one, two = (slice(0, 2 * F, 2), slice(1, 2 * F, 2)) if interleaved else (slice(0, F), slice(F, 2 * F))
    out, mag = x.copy(), np.zeros_like(x)
    u, w = x[..., one], x[..., two]
    out[..., one], out[..., two] = u * np.cos(a) - w * np.sin(a), w * np.cos(a) + u * np.sin(a)
    mag[..., one] = mag[..., two] = np.abs(u) + np.abs(w)
    return out, mag


def accept(tokens, parents, drawn):
    B, N = tokens.shape
    n, out, path = np.full(B, -1), np.full((B, N), -1), np.full((B, N), -1)
    for b in range(B):
        if N == 0 or parents[b, 0] != -1:
            continue
        node, j = 0, 0
        while node is not None:
            path[b, j], out[b, j] = node, drawn[b, node]
            j += 1
            node = next((i for i in range(node + 1, N) if parents[b, i] == node and tokens[b, i] == drawn[b, node]), None)
        n[b] = j - 1
    return n, out, path


def keep(table, lengths, path, P, S):
    """(new lengths, moves): moves as ((page, place), (page, place)) in order, from and to."""
    B, N = path.shape
    new, moves = np.zeros(B, np.int64), []
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * S)
        kept = []
        for p in path[b]:
            if p < 0 or p >= N or (kept and p <= kept[-1]):
                break
            kept.append(int(p))
        base = n - N
        if kept and base < 0:
            new[b] = n
            continue
        new[b] = max(base + len(kept), 0)
        for j, p in enumerate(kept):
            a, d = base + p, base + j
            if a != d and 0 <= table[b, a // S] < P and 0 <= table[b, d // S] < P:
                moves.append(((table[b, a // S], a % S), (table[b, d // S], d % S)))
    return new, moves
