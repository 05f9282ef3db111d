"""The tree operators against plain 64-bit references, at the sizes and masks where they can go wrong.

Tolerances.  Attention as in test_gpu_decode: a score is a sum of D products in fp32, off by at most (D + 8) 2^-24
sum|q||k| scale, which moves a weight by that relative amount (twice: numerator and sum); weights, scaling and
joining add less than 2^-18 of sum p|v|; a bf16 output is rounded once, by at most 2^-8 of itself.  lse is off by the score's
error plus 2^-20 of its own size.  Rotation: sine and cosine are within 2^-23, the angle within 2^-28 radians, the two
products and the sum round by 2^-24 of |x| + |y| each: 2^-21.5 (|x| + |y|), and a bf16 result half a step more, 2^-8 of
itself.  Everything else is whole numbers or copies and must be equal.
"""
import math

import numpy as np
import pytest
import torch

import tree_reference as ref

pytestmark = pytest.mark.gpu
BOTH = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def tree():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    from draft_verify_acceptance_gb300 import tree
    return tree


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def f64(t):
    return t.double().cpu().numpy()


def make_cache(lens, S, H, D, dtype, seed, layers=None, spare=3, extra_cols=2):
    g = gen(seed)
    pages = [-(-n // S) for n in lens]
    P, M = sum(pages) + spare, max(pages + [0]) + extra_cols
    shape = (P, S, H, D) if layers is None else (layers, P, S, H, D)
    k = torch.randn(shape, generator=g, device="cuda").to(dtype)
    v = torch.randn(shape, generator=g, device="cuda").to(dtype)
    ids = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), M), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = ids[at:at + n]
        at += n
    return k, v, table, i32(lens)


def make_trees(B, N, seed, kind="mixed"):
    """Parents [B, N] on the host: chains, stars, random trees, forests and padded ones in turn."""
    r = np.random.RandomState(seed)
    p = np.full((B, N), -1, np.int32)
    for b in range(B):
        what = ("random", "chain", "star", "forest", "padded")[b % 5] if kind == "mixed" else kind
        for i in range(1, N):
            p[b, i] = {"random": r.randint(max(0, i - 9), i), "chain": i - 1, "star": 0, "forest": r.randint(-1, i),
                       "padded": r.randint(0, i) if r.rand() < 0.9 else -2 - r.randint(5)}[what]
        if what == "padded" and N > 2:
            p[b, N - N // 3:] = -2
    return p


def check_attention(out, lse, q, k, v, table, lengths, parents, scale=None):
    D = q.shape[-1]
    scale = 1 / math.sqrt(D) if scale is None else scale
    o, l, mag, spread = ref.attention(f64(q), f64(k), f64(v), table.cpu().numpy(), lengths.cpu().numpy(),
                                      np.broadcast_to(parents.cpu().numpy(), q.shape[:2]), scale)
    score = (D + 8) * 2.0 ** -24 * spread
    tol = mag * (2 * score[..., None] + 2.0 ** -18) + 1e-30
    if q.dtype == torch.bfloat16:
        tol += 2.0 ** -8 * np.abs(o)
    err = np.abs(f64(out) - o)
    assert (err <= tol).all(), (err - tol).max()
    if lse is not None:
        got = f64(lse)
        empty = np.isinf(l)
        assert np.array_equal(np.isinf(got), empty)
        e = np.abs(got[~empty] - l[~empty])
        assert (e <= score[~empty] + 2.0 ** -20 * (1 + np.abs(l[~empty]))).all(), e.max()


# ---- attention ----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("B,N,Hq,H,D,S,lens", [
    (1, 1, 1, 1, 64, 16, [1]),                       # a root and nothing else
    (3, 1, 4, 1, 128, 1, [1, 0, 5]),                 # an empty sequence, pages of one token
    (5, 7, 8, 2, 64, 16, [7, 16, 17, 23, 300]),
    (5, 5, 6, 2, 128, 5, [3, 5, 77, 6, 1]),          # nodes before the sequence's start
    (2, 13, 7, 1, 64, 48, [13, 129]),                # odd group, page not a power of two
    (5, 33, 16, 2, 128, 8, [33, 97, 64, 513, 40]),   # 264 rows a cache head
    (5, 16, 8, 2, 128, 16, [16, 80, 333, 1000, 127]),  # 64 rows
    (5, 31, 8, 2, 128, 16, [31, 80, 333, 159, 128]),   # 124 rows
    (5, 40, 8, 2, 128, 16, [40, 104, 103, 333, 168]),  # 160 rows
    (5, 64, 8, 2, 128, 32, [64, 128, 191, 333, 65]),   # 256 rows
    (2, 200, 4, 2, 64, 16, [200, 777]),              # 400 rows
    (2, 256, 3, 1, 128, 64, [256, 1000]),            # the largest tree, 768 rows
    (5, 65, 2, 1, 64, 16, [400, 65, 66, 128, 129]),
    (40, 6, 12, 4, 128, 32, list(range(6, 46))),
    (1, 26, 8, 8, 128, 128, [6001]),                 # one sequence, cut over many blocks
    (2, 9, 32, 4, 128, 16, [2000, 31]),
    (3, 20, 32, 8, 64, 16, [1500, 20, 700]),
])
def test_attention(tree, dtype, B, N, Hq, H, D, S, lens):
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=B * 1000 + N)
    q = (torch.randn((B, N, Hq, D), generator=gen(5), device="cuda") * 2).to(dtype)
    parents = i32(make_trees(B, N, N + B).tolist())
    out, lse, status = tree.tree_attention(q, k, v, table, lengths, parents, return_lse=True, debug=True)
    assert int(status) == 0
    check_attention(out, lse, q, k, v, table, lengths, parents)
    again, lse2 = tree.tree_attention(q, k, v, table, lengths, parents, return_lse=True)
    assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("B,N,Hq,H,D", [(400, 7, 32, 8, 64), (350, 40, 16, 4, 64), (330, 9, 20, 5, 128)])
def test_attention_of_many_short_sequences(tree, B, N, Hq, H, D):
    """Blocks that take ten and more items each, of one tile or two, whole and cut, empty sequences among them."""
    r = np.random.RandomState(B)
    lens = [int(n) for n in r.randint(0, N + 70, B)]
    k, v, table, lengths = make_cache(lens, 16, H, D, torch.bfloat16, seed=B)
    q = (torch.randn((B, N, Hq, D), generator=gen(5), device="cuda") * 2).to(torch.bfloat16)
    parents = i32(make_trees(B, N, N).tolist())
    out, lse, status = tree.tree_attention(q, k, v, table, lengths, parents, return_lse=True, debug=True)
    assert int(status) == 0
    part = slice(B % 7, None, 11)
    check_attention(out[part], lse[part], q[part], k, v, table[part], lengths[part], parents[part])
    for _ in range(3):
        assert torch.equal(tree.tree_attention(q, k, v, table, lengths, parents), out)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("N,G,D", [(3, 4, 128), (13, 4, 64), (16, 8, 128), (30, 4, 128), (60, 4, 128), (33, 3, 64)])
def test_a_chain_is_paged_attention(tree, dtype, N, G, D):
    """Nodes one below the other see what a verify step's queries see."""
    from draft_verify_acceptance_gb300 import decode
    lens, S, H = [N, N + 5, 50 + N, 777, 3], 16, 2
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=N)
    q = torch.randn((len(lens), N, H * G, D), generator=gen(1), device="cuda").to(dtype)
    chain = torch.arange(-1, N - 1, dtype=torch.int32, device="cuda")
    out, lse = tree.tree_attention(q, k, v, table, lengths, chain, return_lse=True)
    check_attention(out, lse, q, k, v, table, lengths, chain)
    want, wl = decode.paged_attention(q, k, v, table, lengths, return_lse=True)
    step = 2.0 ** -7 if dtype == torch.bfloat16 else 2.0 ** -17  # (both are within half of it of the formula)
    assert ((out.double() - want.double()).abs() <= step * want.double().abs() + 2.0 ** -16).all()
    assert torch.equal(torch.isinf(lse), torch.isinf(wl))


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("N,G,D", [(2, 4, 128), (6, 4, 64), (12, 8, 128), (17, 3, 64), (40, 4, 128), (70, 4, 64)])
def test_unseen_tokens_do_not_matter(tree, dtype, N, G, D):
    """NaN and infinities where a node does not look: behind the sequence, in unused pages, and at every other branch."""
    lens, S, H = [N, 50 + N, 333], 16, 2
    B = len(lens)
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=3)
    q = torch.randn((B, N, H * G, D), generator=gen(1), device="cuda").to(dtype)
    p = make_trees(B, N, 7, "random")
    parents = i32(p.tolist())
    clean, lse = tree.tree_attention(q, k, v, table, lengths, parents, return_lse=True)
    used = torch.zeros(k.shape[:2], dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        used[table[b, t // S].long(), t % S] = True
    for bad in (math.nan, math.inf, -math.inf):
        k2, v2 = k.clone(), v.clone()
        k2[~used], v2[~used] = bad, bad
        got, l2 = tree.tree_attention(q, k2, v2, table, lengths, parents, return_lse=True)
        assert torch.equal(got, clean) and torch.equal(l2, lse)
        for node in sorted({0, N // 2, N - 1}):  # this node's token is bad: who does not see it does not change
            for which in ((True, True), (False, True), (True, False)):
                k2, v2 = k.clone(), v.clone()
                for b, n in enumerate(lens):
                    t = n - N + node
                    if which[0]:
                        k2[table[b, t // S].long(), t % S] = bad
                    if which[1]:
                        v2[table[b, t // S].long(), t % S] = bad
                got = tree.tree_attention(q, k2, v2, table, lengths, parents)
                for b in range(B):
                    for i in range(N):
                        if node in ref.line(p[b], i):
                            if which[1] and not which[0]:
                                assert not torch.isfinite(got[b, i]).any(), (bad, node, b, i)
                        else:
                            assert torch.equal(got[b, i], clean[b, i]), (bad, node, which, b, i)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("N,G", [(5, 2), (20, 4), (50, 4)])
def test_a_bad_context_value_reaches_every_node(tree, dtype, N, G):
    lens, S, H, D = [N + 200], 16, 1, 128
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=4)
    v[table[0, 2].long(), 3, 0, 7] = math.inf
    q = torch.randn((1, N, G, D), generator=gen(1), device="cuda").to(dtype)
    p = make_trees(1, N, 3, "random")
    p[0, -1] = -2
    out = tree.tree_attention(q, k, v, table, lengths, i32(p.tolist()))
    assert not torch.isfinite(out[0, :-1, :, 7]).any()
    assert torch.isfinite(out[0, :-1, :, :7]).all() and torch.isfinite(out[0, :-1, :, 8:]).all()
    assert (out[0, -1] == 0).all()


@pytest.mark.parametrize("dtype,N,G,D", [
    (torch.bfloat16, 9, 4, 128), (torch.bfloat16, 30, 4, 64), (torch.bfloat16, 16, 8, 128),  # one row tile
    (torch.bfloat16, 40, 4, 128), (torch.bfloat16, 64, 4, 64), (torch.bfloat16, 33, 8, 64),  # two, the last of eight rows of 264
    (torch.bfloat16, 6, 4, 128), (torch.bfloat16, 11, 2, 64),                                # up to 24 rows
    (torch.float32, 5, 4, 128), (torch.float32, 13, 4, 64), (torch.float32, 30, 2, 128)])
def test_values_that_are_not_finite_in_a_cut_item(tree, dtype, N, G, D):
    """One long sequence, cut over many blocks (more tiles than any kernel leaves whole; the lengths move the cuts and the
    tree over them).  NaN queries and keys make the rows that see them NaN, values that are not finite make their
    dimension not finite, wherever among the parts they lie; all else keeps its bits."""
    S, H = 16, 2
    p = make_trees(1, N, N, "random")
    p[0, N - 1] = -2  # one that is none
    up = [set(ref.line(p[0], i) or ()) for i in range(N)]
    parents = i32(p.tolist())
    for tiles in range(18, 30):
        n = 64 * tiles + (1, N // 2, 63)[tiles % 3]
        k, v, table, lengths = make_cache([n], S, H, D, dtype, seed=tiles)
        q = torch.randn((1, N, H * G, D), generator=gen(1), device="cuda").to(dtype)
        call = lambda q, k, v: tree.tree_attention(q, k, v, table, lengths, parents, return_lse=True)  # noqa: E731
        clean, lse = call(q, k, v)
        assert torch.isfinite(clean).all() and torch.isfinite(lse[0, :-1]).all()
        q2 = q.clone()
        q2[0, N - 2, G + 1, 3] = math.nan  # of cache head 1
        out, l2 = call(q2, k, v)
        assert torch.isnan(out[0, N - 2, G + 1]).all() and torch.isnan(l2[0, N - 2, G + 1])
        out[0, N - 2, G + 1], l2[0, N - 2, G + 1] = clean[0, N - 2, G + 1], lse[0, N - 2, G + 1]
        assert torch.equal(out, clean) and torch.equal(l2, lse)
        spots = [0, 700 + 13 * tiles, n - N - 1] + [n - N + i for i in sorted({0, 1, N // 2, N - 2, N - 1})]
        for j, t in enumerate(spots):
            node = t - (n - N)
            sees = [i for i in range(N - 1) if node < 0 or node in up[i]]
            place = (table[0, t // S].long(), t % S, 1)
            h = slice(G, 2 * G)

            def others(out, l2, d=slice(None), with_lse=True):  # put back, all is as it was
                out, l2 = out.clone(), l2.clone()
                for i in sees:
                    out[0, i, h, d] = clean[0, i, h, d]
                    l2[0, i, h] = lse[0, i, h] if with_lse else l2[0, i, h]
                assert torch.equal(out, clean) and torch.equal(l2, lse), (n, t, j)
            k2 = k.clone()
            k2[(*place, 7)] = math.nan
            out, l2 = call(q, k2, v)
            assert all(torch.isnan(out[0, i, h]).all() and torch.isnan(l2[0, i, h]).all() for i in sees), (n, t)
            others(out, l2)
            k2[(*place, 7)] = math.inf  # scores of +inf (NaN) or -inf (a weight of 0), by the query's sign
            out, l2 = call(q, k2, v)
            for i in sees:
                over = q[0, i, h, 7] > 0
                assert torch.isnan(out[0, i, h][over]).all() and torch.isnan(l2[0, i, h][over]).all(), (n, t, i)
                if dtype == torch.bfloat16:  # (fp32 operands are two parts, infinity's second one NaN: all of these rows are)
                    assert torch.isfinite(out[0, i, h][~over]).all() and torch.isfinite(l2[0, i, h][~over]).all(), (n, t, i)
                    assert (l2[0, i, h][~over] <= lse[0, i, h][~over] + 1e-5).all()
            others(out, l2)
            for bad in (math.nan, math.inf, -math.inf):
                v2 = v.clone()
                v2[(*place, D - 3)] = bad
                out, l2 = call(q, k, v2)
                assert all((~torch.isfinite(out[0, i, h, D - 3])).all() for i in sees), (n, t, bad)
                others(out, l2, D - 3, False)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("N,G,H,D,lens", [
    (9, 4, 2, 128, [512, 9, 100]), (30, 4, 8, 64, [30, 511, 65, 0, 300, 128] * 3), (16, 8, 1, 128, [5, 449]),
    (40, 4, 2, 128, [512, 40, 104]), (60, 4, 8, 128, [60, 512, 333, 7, 190] * 3), (33, 8, 2, 64, [33, 97, 512]),
    (5, 4, 2, 64, [5, 512, 77]), (13, 4, 2, 64, [13, 190, 100, 50])])
def test_short_sequences_under_a_table_with_room_for_long_ones(tree, dtype, N, G, H, D, lens):
    """A server's table has room for its longest context: that no item is cut is then known from the lengths alone.  The results
    are those of a table that has no more room than these sequences need (bf16: bit for bit)."""
    k, v, tight, lengths = make_cache(lens, 16, H, D, dtype, seed=N, extra_cols=0)
    q = torch.randn((len(lens), N, H * G, D), generator=gen(5), device="cuda").to(dtype)
    parents = i32(make_trees(len(lens), N, N).tolist())
    want, wl = tree.tree_attention(q, k, v, tight, lengths, parents, return_lse=True)
    check_attention(want, wl, q, k, v, tight, lengths, parents)
    roomy = torch.full((len(lens), 4096 // 16), -1, dtype=torch.int32, device="cuda")
    roomy[:, :tight.shape[1]] = tight
    out, lse, status = tree.tree_attention(q, k, v, roomy, lengths, parents, return_lse=True, debug=True)
    assert int(status) == 0
    check_attention(out, lse, q, k, v, roomy, lengths, parents)
    if dtype == torch.bfloat16:
        assert torch.equal(out, want) and torch.equal(lse, wl)
    for _ in range(3):
        again, l2 = tree.tree_attention(q, k, v, roomy, lengths, parents, return_lse=True)
        assert torch.equal(again, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("N", [4, 40])
def test_large_scores_and_far_maxima(tree, dtype, N):
    """Scores that rise along the context by far more than a reference maximum's slack, of both signs, and of +-0 scale."""
    lens, S, H, D, G = [N + 900, N + 64], 16, 2, 64, 4
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=9)
    for b, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        k[table[b, t // S].long(), t % S] *= (1 + t.float() / 40)[:, None, None].to(dtype)
    q = (torch.randn((2, N, H * G, D), generator=gen(1), device="cuda") * 6).to(dtype)
    parents = i32(make_trees(2, N, 5).tolist())
    for scale in (None, 0.3, 0.0, -0.2):
        out, lse = tree.tree_attention(q, k, v, table, lengths, parents, scale, return_lse=True)
        check_attention(out, lse, q, k, v, table, lengths, parents, scale)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("N", [5, 30])
def test_trees_without_nodes_and_bad_parents(tree, dtype, N):
    lens, S, H, D = [N + 100] * 4, 16, 2, 128
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=2)
    q = torch.randn((4, N, 8, D), generator=gen(1), device="cuda").to(dtype)
    p = make_trees(4, N, 1, "random")
    p[0] = -2                 # nothing at all
    p[1, 2:] = np.arange(2, N)  # parents of themselves
    p[2, 1] = 2 ** 31 - 1     # far behind
    p[3, 0] = -2 ** 31        # no root: nobody below it either
    out, lse, status = tree.tree_attention(q, k, v, table, lengths, i32(p.tolist()), return_lse=True, debug=True)
    assert int(status) == tree.DATA_TREE_PARENT
    check_attention(out, lse, q, k, v, table, lengths, i32(p.tolist()))
    assert (out[0] == 0).all() and torch.isinf(lse[0]).all() and (out[3] == 0).all()


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("N", [5, 30])
def test_bad_pages_and_lengths(tree, dtype, N):
    from draft_verify_acceptance_gb300 import decode
    lens, S, H, D = [N + 100, N + 40, N + 77], 16, 2, 128
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=2)
    q = torch.randn((3, N, 8, D), generator=gen(1), device="cuda").to(dtype)
    parents = i32(make_trees(3, N, 1).tolist())
    bad = table.clone()
    bad[0, 1], bad[1, 0], bad[2, (N + 76) // S] = -5, k.shape[0], 2 ** 31 - 1
    out, lse, status = tree.tree_attention(q, k, v, bad, lengths, parents, return_lse=True, debug=True)
    assert int(status) == decode.DATA_PAGE_RANGE
    check_attention(out, lse, q, k, v, bad, lengths, parents)
    out, lse, status = tree.tree_attention(q, k, v, table, i32([-3, N + 40, 2 ** 31 - 1]), parents, return_lse=True, debug=True)
    assert int(status) & decode.DATA_LENGTH_RANGE
    assert (out[0] == 0).all() and torch.isinf(lse[0]).all()
    check_attention(out[1:2], lse[1:2], q[1:2], k, v, table[1:2], lengths[1:2], parents[1:2])


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("N", [7, 36])
def test_strides_and_shared_rows(tree, dtype, N):
    """q sliced from a fused projection, a layer of an interleaved cache, one tree and one table for all, sliced tables."""
    lens, S, H, D, G = [N + 60] * 3, 16, 2, 128, 4
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=6)
    qkv = torch.randn((3, N, (H * G + 2 * H) * D), generator=gen(1), device="cuda").to(dtype)
    q = qkv[..., :H * G * D].unflatten(-1, (H * G, D))
    p = make_trees(1, N, 8, "random")
    one = i32(p[0].tolist())
    want = tree.tree_attention(q.contiguous(), k, v, table, lengths, i32(np.repeat(p, 3, 0).tolist()))
    both = torch.stack((k, v), 1)
    wide = torch.full((3, table.shape[1] + 9), 77777, dtype=torch.int32, device="cuda")
    wide[:, 4:-5] = table
    trees = torch.full((3, N + 3), 99, dtype=torch.int32, device="cuda")
    trees[:, :N] = one
    for par in (one, one[None].expand(3, N), trees[:, :N]):
        got = tree.tree_attention(q, both[:, 0], both[:, 1], wide[:, 4:-5], lengths, par)
        assert torch.equal(got, want)
    got = tree.tree_attention(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, table, lengths, one)
    assert torch.equal(got, want)
    same = table[:1].expand(3, -1)
    assert torch.equal(tree.tree_attention(q, k, v, same, lengths, one), tree.tree_attention(q, k, v, same.contiguous(), lengths, one))


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("N", [5, 30, 64])
def test_out_streams_graphs_and_workspaces(tree, dtype, N):
    lens, S, H, D = [N + 700, N, 1100], 16, 2, 128
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=6)
    q = torch.randn((3, N, 8, D), generator=gen(1), device="cuda").to(dtype)
    parents = i32(make_trees(3, N, 8).tolist())
    want, wl = tree.tree_attention(q, k, v, table, lengths, parents, return_lse=True)
    out = torch.full_like(q, 7.0)
    version = out._version
    assert tree.tree_attention(q, k, v, table, lengths, parents, out=out) is out and torch.equal(out, want) and out._version > version
    with pytest.raises(Exception):
        tree.tree_attention(q, k, v, table, lengths, parents, out=q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [tree.tree_attention(q, k, v, table, lengths, parents, stream=side) for _ in range(3)]
    here = [tree.tree_attention(q, k, v, table, lengths, parents) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got + here)
    need = tree.attention_workspace_size(3, N, 8, H, D, dtype)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        assert torch.equal(tree.tree_attention(q, k, v, table, lengths, parents, workspace=ws), want)
    with pytest.raises(ValueError):
        tree.tree_attention(q, k, v, table, lengths, parents, workspace=ws[:-256])
    graphs = []
    for _ in range(2):  # two graphs, each with a workspace of its own, replayed in turn and at once
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = tree.tree_attention(q, k, v, table, lengths, parents)
        graphs.append((g, o))
    for _ in range(2):
        for g, o in graphs:
            o.fill_(3.0)
        torch.cuda.synchronize()
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for _, o in graphs)
    parents.fill_(-2)  # a replay reads the tree that is there
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert (graphs[0][1] == 0).all()


def test_a_cache_beyond_32_bits(tree):
    """Pages and layers' offsets past 2^32 bytes and past 2^31 elements."""
    S, H, D, N = 16, 8, 128, 20
    P = (5 << 30) // (S * H * D * 2)
    k = torch.zeros((P, S, H, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = i32([[P - 1, 3, P // 2 + 1, P - 7, 0]])
    lens = i32([70])
    for page in table[0].tolist():
        k[page] = torch.randn((S, H, D), generator=gen(page % 1000), device="cuda").to(torch.bfloat16)
        v[page] = torch.randn((S, H, D), generator=gen(page % 999 + 1), device="cuda").to(torch.bfloat16)
    q = torch.randn((1, N, 32, D), generator=gen(3), device="cuda").to(torch.bfloat16)
    parents = i32(make_trees(1, N, 3, "random").tolist())
    out, lse = tree.tree_attention(q, k, v, table, lens, parents, return_lse=True)
    few = [P - 1, 3, P // 2 + 1, P - 7, 0]
    check_attention(out, lse, q, k[few], v[few], i32([[0, 1, 2, 3, 4]]), lens, parents)
    kn, vn = (torch.randn((1, 3, H, D), generator=gen(8 + i), device="cuda").to(torch.bfloat16) for i in range(2))
    tree.cache_append_rotated(kn, vn, k, v, i32([[P - 1]]), i32([9]), torch.zeros(64, device="cuda"))
    assert torch.equal(k[P - 1, 6:9], kn[0]) and torch.equal(v[P - 1, 6:9], vn[0])
    mark = k[P - 1, 8].clone()
    tree.cache_keep(k, v, i32([[P - 1]]), i32([9]), i32([[0, 2, -1]]))
    assert torch.equal(k[P - 1, 7], mark)


# ---- rotated append -------------------------------------------------------------------------------

def check_rotated(got, x, positions, inv_freq, interleaved):
    """Rows x [T, heads, D] at `positions` against their rotation."""
    f = inv_freq.cpu().numpy()
    for t, p in enumerate(positions):
        o, mag = ref.rotate(f64(x[t]), p, f, interleaved)
        tol = mag * 2.0 ** -21.5 + (2.0 ** -8 * np.abs(o) if x.dtype == torch.bfloat16 else 0)
        err = np.abs(f64(got[t]) - o)
        assert (err <= tol).all(), (t, p, (err - tol).max())


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("counts,before,Hq,H,D,F,S", [
    ([1], [0], 1, 1, 64, 32, 16),
    ([1, 1, 1], [0, 500, 31], 4, 1, 128, 64, 16),
    ([0, 7, 1, 0, 33, 0], [3, 0, 15, 0, 60, 9], 3, 3, 64, 16, 1),    # half of a head's dimensions, pages of one token
    ([5, 130], [11, 3], 8, 2, 128, 64, 48),
    ([300], [7], 12, 4, 40, 8, 5),                                   # heads of 40, 16 of them rotated
    ([9, 9], [1, 2], 5, 1, 256, 128, 8),
    ([4, 4], [1, 2], 2, 2, 64, 0, 8),                                # nothing to rotate
    ([700, 1, 513], [0, 90, 1000], 8, 2, 128, 64, 16),
])
def test_append(tree, dtype, interleaved, counts, before, Hq, H, D, F, S):
    B, T = len(counts), sum(counts)
    lens = [a + b for a, b in zip(counts, before)]
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=T)
    qkv = torch.randn((T, (Hq + 2 * H) * D), generator=gen(T), device="cuda").to(dtype)
    q, kn, vn = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, H * D, H * D], 1))
    starts = i32(np.concatenate([[0], np.cumsum(counts)]).tolist())
    inv = (10000.0 ** (-torch.arange(F, dtype=torch.float64) / max(F, 1))).float().cuda()
    place = [(b, t) for b in range(B) for t in range(before[b], lens[b])]
    r = np.random.RandomState(1)
    for positions in (None, r.randint(-10, 2 ** 31 - 1, T), r.randint(0, 131072, T)):
        k2, v2 = k.clone(), v.clone()
        pos = [t for _, t in place] if positions is None else positions.tolist()
        got, status = tree.cache_append_rotated(kn, vn, k2, v2, table, lengths, inv, q, None if positions is None else i32(pos), starts,
                                                interleaved=interleaved, debug=True)
        assert int(status) == 0
        check_rotated(got, q, pos, inv, interleaved)
        b, t = (torch.tensor(x, device="cuda") for x in zip(*place))
        page, spot = table[b, t // S].long(), t % S
        check_rotated(k2[page, spot], kn, pos, inv, interleaved)
        assert torch.equal(v2[page, spot], vn)
        k2[page, spot], v2[page, spot] = k[page, spot], v[page, spot]
        assert torch.equal(k2, k) and torch.equal(v2, v)  # nothing else was written
        k2, v2 = k.clone(), v.clone()
        assert tree.cache_append_rotated(kn, vn, k2, v2, table, lengths, inv, positions=None if positions is None else i32(pos),
                                         starts=starts, interleaved=interleaved) is None
        whole = qkv.clone()
        qi = whole[:, :Hq * D].unflatten(1, (Hq, D))
        version = qi._version
        back = tree.cache_append_rotated(kn, vn, k2, v2, table, lengths, inv, qi, None if positions is None else i32(pos), starts,
                                         interleaved=interleaved, out=qi)
        assert back is qi and torch.equal(qi, got) and torch.equal(whole[:, Hq * D:], qkv[:, Hq * D:]) and qi._version > version


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_at_high_frequencies(tree, interleaved):
    """Frequencies from just above 1 to the largest, whose angles no double holds.  Sine, cosine and products as at the others."""
    H, D, S, T = 2, 64, 16, 7
    k, v, table, lengths = make_cache([T], S, H, D, torch.float32, seed=1)
    kn, vn, q = (torch.randn((1, T, H, D), generator=gen(i), device="cuda") for i in (1, 2, 3))
    r = np.random.RandomState(3)
    inv = np.concatenate(([1.0, 1 + 2.0 ** -23, 2.5, -1e4, 2.0 ** 24, 1e9, 3.4028235e38, -3e30], r.uniform(1, 2, 24) * 2.0 ** r.randint(0, 127, 24)))
    inv = torch.tensor(inv, dtype=torch.float32, device="cuda")
    pos = [0, 1, 17, 131071, 2 ** 31 - 1, -2 ** 31, 123456789]
    got = tree.cache_append_rotated(kn, vn, k, v, table, lengths, inv, q, i32([pos]), interleaved=interleaved)
    exact = np.array([[ref.turns(p, f) for f in inv.cpu().tolist()] for p in pos]) * 2 * np.pi
    one, two = (slice(0, D, 2), slice(1, D, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    t = torch.arange(T, device="cuda")
    for out, x in ((got[0], q[0]), (k[table[0, t // S].long(), t % S], kn[0])):
        u, w = f64(x)[..., one], f64(x)[..., two]
        c, s = np.cos(exact)[:, None], np.sin(exact)[:, None]
        tol = (np.abs(u) + np.abs(w)) * 2.0 ** -21.5
        assert (np.abs(f64(out)[..., one] - (u * c - w * s)) <= tol).all()
        assert (np.abs(f64(out)[..., two] - (w * c + u * s)) <= tol).all()


def test_append_without_rotation_is_append(tree):
    from draft_verify_acceptance_gb300 import decode
    k, v, table, lengths = make_cache([40, 33], 16, 2, 128, torch.bfloat16, seed=1)
    kn, vn = (torch.randn((2, 9, 2, 128), generator=gen(i), device="cuda").bfloat16() for i in (1, 2))
    a, b, c, d = k.clone(), v.clone(), k.clone(), v.clone()
    decode.cache_append(kn, vn, a, b, table, lengths)
    tree.cache_append_rotated(kn, vn, c, d, table, lengths, torch.zeros(64, device="cuda"))
    assert torch.equal(a, c) and torch.equal(b, d)


def test_append_rows_of_nobody_and_bad_places(tree):
    from draft_verify_acceptance_gb300 import decode
    S, H, D = 16, 2, 64
    k, v, table, _ = make_cache([40, 33, 20], S, H, D, torch.float32, seed=1)
    T = 12
    kn, vn, q = (torch.randn((T, H, D), generator=gen(i), device="cuda") for i in (1, 2, 3))
    inv = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda()
    starts = i32([0, 3, 6, 8])  # rows 8.. are nobody's
    k2, v2 = k.clone(), v.clone()
    got, status = tree.cache_append_rotated(kn, vn, k2, v2, table, i32([40, 33, 20]), inv, q, starts=starts, debug=True)
    assert int(status) == decode.DATA_LENGTH_RANGE and (got[8:] == 0).all()
    check_rotated(got[:8], q, [37, 38, 39, 30, 31, 32, 18, 19], inv, False)
    qi = q.clone()
    tree.cache_append_rotated(kn, vn, k2, v2, table, i32([40, 33, 20]), inv, qi, starts=starts, out=qi)
    assert torch.equal(qi[8:], q[8:]) and torch.equal(qi[:8], got[:8])
    # places before the start, behind the table, on a page out of range: not written, their queries rotated
    bad = table.clone()
    bad[2, 1] = k.shape[0]
    k2, v2 = k.clone(), v.clone()
    far = (table.shape[1] + 1) * S
    pos = i32(list(range(T)))
    got, status = tree.cache_append_rotated(kn, vn, k2, v2, bad, i32([1, far, 20]), inv, q, pos, starts, debug=True)
    assert int(status) == decode.DATA_LENGTH_RANGE | decode.DATA_PAGE_RANGE
    check_rotated(got[:8], q, list(range(8)), inv, False)
    check_rotated(k2[table[0, 0].long(), :1], kn[2:3], [2], inv, False)  # the third of three new tokens of one
    k2[table[0, 0].long(), 0], v2[table[0, 0].long(), 0] = k[table[0, 0].long(), 0], v[table[0, 0].long(), 0]
    assert torch.equal(k2, k) and torch.equal(v2, v)


def test_append_refusals(tree):
    k, v, table, lengths = make_cache([40, 33], 16, 2, 128, torch.bfloat16, seed=1)
    kn, vn = (torch.randn((2, 4, 2, 128), device="cuda").bfloat16() for _ in range(2))
    inv = torch.zeros(64, device="cuda")
    q = torch.randn((2, 4, 8, 128), device="cuda").bfloat16()
    ok = lambda **kw: tree.cache_append_rotated(*(kw.get(n, d) for n, d in (  # noqa: E731
        ("kn", kn), ("vn", vn), ("k", k), ("v", v), ("table", table), ("lengths", lengths), ("inv", inv), ("q", q))),
        **{n: x for n, x in kw.items() if n in ("positions", "starts", "out")})
    ok()
    from draft_verify_acceptance_gb300.binding import SpecVerifyError
    big = torch.randn((2, 9, 8, 128), device="cuda").bfloat16()
    for bad in (dict(kn=kn.float()), dict(vn=vn[:, :3]), dict(q=q.float()), dict(q=q[:, :3]), dict(q=q[..., :64]), dict(inv=inv.double()),
                dict(inv=inv[::2]), dict(inv=torch.zeros(72, device="cuda")), dict(inv=torch.zeros(12, device="cuda")),
                dict(positions=i32([0] * 8)), dict(positions=torch.zeros((2, 4), dtype=torch.int64, device="cuda")),
                dict(starts=i32([0, 4, 8])), dict(lengths=lengths[:1]), dict(out=big[:, 1:5]), dict(out=q.float()),
                dict(q=big[:, :4], out=big[:, 1:5]), dict(out=kn.view(2, 4, 2, 128)), dict(inv=inv.cpu()), dict(q=q.cpu())):
        with pytest.raises((TypeError, ValueError, SpecVerifyError, IndexError)):
            ok(**bad)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("order", ["qkv", "kvq", "kqv"])
@pytest.mark.parametrize("B,n", [(1, 1), (2, 1), (2, 7), (1, 300)])
def test_append_in_place_between_the_rows_it_reads(tree, dtype, order, B, n):
    """The queries of a fused projection rotated where they lie, keys and values in the gaps between them; where keys or values
    are the queries' own bytes the call is refused."""
    from draft_verify_acceptance_gb300.binding import SpecVerifyError
    Hq, H, D, S = 8, 2, 64, 16
    k, v, table, lengths = make_cache([n + 5] * B, S, H, D, dtype, seed=n)
    fused = torch.randn((B, n, (Hq + 2 * H) * D), generator=gen(n), device="cuda").to(dtype)
    heads = {"q": Hq, "k": H, "v": H}

    def slices(x):
        at, r = 0, {}
        for c in order:
            r[c] = x[..., at:at + heads[c] * D].unflatten(-1, (-1, D))
            at += heads[c] * D
        return r
    inv = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda()
    x = slices(fused.clone())
    wk, wv = k.clone(), v.clone()
    want = tree.cache_append_rotated(x["k"], x["v"], wk, wv, table, lengths, inv, x["q"])
    whole = fused.clone()
    x = slices(whole)
    assert tree.cache_append_rotated(x["k"], x["v"], k, v, table, lengths, inv, x["q"], out=x["q"]) is x["q"]
    assert torch.equal(x["q"], want) and torch.equal(k, wk) and torch.equal(v, wv)
    assert torch.equal(x["k"], slices(fused)["k"]) and torch.equal(x["v"], slices(fused)["v"])
    for bad in (x["q"][..., :H, :], x["q"][..., -H:, :]):
        for kn, vn in ((bad, x["v"]), (x["k"], bad)):
            if kn.stride() != vn.stride():
                continue
            with pytest.raises(SpecVerifyError):
                tree.cache_append_rotated(kn, vn, k, v, table, lengths, inv, x["q"], out=x["q"])
    assert torch.equal(k, wk) and torch.equal(v, wv)


# ---- accept and keep ------------------------------------------------------------------------------

@pytest.mark.parametrize("B,N", [(1, 1), (7, 2), (40, 13), (5, 31), (5, 32), (5, 33), (300, 64), (10, 255), (10, 256), (3, 0)])
def test_accept(tree, B, N):
    r = np.random.RandomState(N)
    p = make_trees(B, N, N)
    tokens = r.randint(0, 6, (B, N))  # few tokens: twins among siblings
    drawn = r.randint(0, 6, (B, N))
    if N:
        chain = np.flatnonzero(np.arange(B) % 5 == 1)  # chains accepted to the end, and to one before it
        tokens[chain], drawn[chain] = 3, 3
        drawn[chain[1:], N - 1 - (N > 1)] = 4
        p[0, 0] = -1 if B < 5 else -2
    got = tree.tree_accept(i32(tokens.tolist()).view(B, N), i32(p.tolist()).view(B, N), i32(drawn.tolist()).view(B, N), debug=True)
    n, out, path = ref.accept(tokens, p, drawn)
    assert int(got.status) == 0
    assert np.array_equal(got.accepted_len.cpu().numpy(), n)
    assert np.array_equal(got.out_tokens.cpu().numpy(), out) and np.array_equal(got.path.cpu().numpy(), path)
    plain = tree.tree_accept(i32(tokens.tolist()).view(B, N), i32(p.tolist()).view(B, N), i32(drawn.tolist()).view(B, N))
    assert plain.status is None and all(torch.equal(a, b) for a, b in zip(plain[:3], got[:3]))


def test_accept_one_tree_for_all_and_bad_parents(tree):
    p = i32([-1, 0, 0, 1, 1])
    tokens, drawn = i32([[0, 1, 2, 3, 4]] * 3), i32([[1, 4, 0, 0, 9], [2, 4, 7, 0, 9], [5, 0, 0, 0, 0]])
    got = tree.tree_accept(tokens, p, drawn)
    assert got.accepted_len.tolist() == [2, 1, 0]
    assert got.path.tolist() == [[0, 1, 4, -1, -1], [0, 2, -1, -1, -1], [0, -1, -1, -1, -1]]
    assert got.out_tokens.tolist() == [[1, 4, 9, -1, -1], [2, 7, -1, -1, -1], [5, -1, -1, -1, -1]]
    wide = torch.full((3, 9), 5, dtype=torch.int32, device="cuda")
    wide[:, :5] = p
    for par in (p[None].expand(3, 5), wide[:, :5]):
        assert all(torch.equal(a, b) for a, b in zip(tree.tree_accept(tokens, par, drawn)[:3], got[:3]))
    bad = i32([-1, 1, 4, 0, 3])  # node 1 its own parent, node 2 below a later one
    got = tree.tree_accept(i32([[7, 7, 7, 7, 7]]), bad[None], i32([[7, 7, 7, 7, 7]]), debug=True)
    assert int(got.status) == tree.DATA_TREE_PARENT and got.path.tolist() == [[0, 3, 4, -1, -1]]


def test_accept_in_place(tree):
    """Through the C entry point: path and out_tokens written over the rows that they are made from."""
    B, N = 37, 64
    r = np.random.RandomState(2)
    host = [r.randint(0, 4, (B, N)), make_trees(B, N, 3), r.randint(0, 4, (B, N))]
    n, out, path = ref.accept(*host)
    for over in ((0, 1), (1, 0), (2, 1), (1, 2), (0, 2), (2, 0), (2, None), (None, 2)):
        ins = [i32(x.tolist()) for x in host]
        got_n, fresh = i32([7] * B), [i32(x.tolist()) for x in host]
        to = [ins[o] if o is not None else fresh[i] for i, o in enumerate(over)]
        rc = tree._lib.spec_tree_accept(ins[0].data_ptr(), ins[1].data_ptr(), N, ins[2].data_ptr(), B, N, got_n.data_ptr(),
                                        to[0].data_ptr(), to[1].data_ptr(), torch.cuda.current_stream().cuda_stream, None)
        assert rc == 0
        assert np.array_equal(got_n.cpu().numpy(), n)
        assert np.array_equal(to[0].cpu().numpy(), out) and np.array_equal(to[1].cpu().numpy(), path), over


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("N,S,L,H,D,lens", [
    (1, 16, 1, 1, 64, [1, 5]), (5, 1, 2, 2, 64, [5, 9, 0]), (13, 16, 3, 2, 64, [13, 40, 100]), (64, 8, 2, 8, 128, [64, 200, 77]),
    (200, 16, 1, 1, 64, [200, 1000]), (300, 32, 1, 2, 128, [300, 317]), (40, 16, 2, 3, 8, [40, 55]),
])
def test_keep(tree, dtype, N, S, L, H, D, lens):
    r = np.random.RandomState(N)
    B = len(lens)
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=N, layers=L)
    for share in (0.2, 0.7, 1.0):
        path = np.full((B, N), -1)
        for b in range(B):
            kept = np.flatnonzero(r.rand(N) < share)
            if lens[b] >= N:
                path[b, :len(kept)] = kept
        new, moves = ref.keep(table.cpu().numpy(), lens, path, k.shape[1], S)
        wk, wv = k.clone(), v.clone()
        for (p, t), (p2, t2) in moves:
            wk[:, p2, t2], wv[:, p2, t2] = wk[:, p, t], wv[:, p, t]
        gk, gv = k.clone(), v.clone()
        got, status = tree.cache_keep(gk, gv, table, lengths, i32(path.tolist()), debug=True)
        assert int(status) == 0 and got.tolist() == new.tolist()
        assert torch.equal(gk, wk) and torch.equal(gv, wv)
        gk, gv = torch.stack((k, v), 2).unbind(2)  # K and V interleaved by token blocks
        version = gk._version
        assert tree.cache_keep(gk, gv, table, lengths, i32(path.tolist())).tolist() == new.tolist() and gk._version > version
        assert torch.equal(gk, wk) and torch.equal(gv, wv)
    one, two = k[0].clone(), v[0].clone()  # a cache of one layer without the dimension
    tree.cache_keep(one, two, table, lengths, i32(path.tolist()))
    assert torch.equal(one, wk[0]) and torch.equal(two, wv[0])


def test_keep_bad_paths_pages_and_lengths(tree):
    from draft_verify_acceptance_gb300 import decode
    N, S = 6, 4
    k, v, table, _ = make_cache([30] * 6, S, 1, 64, torch.float32, seed=1)
    lengths = i32([30, 30, 30, 4, 30, -7])
    path = i32([[0, 3, 3, 4, -1, -1], [1, 6, -1, -1, -1, -1], [2, 1, -1, -1, -1, -1], [0, 2, -1, -1, -1, -1], [0, 2, 5, -1, -1, -1],
                [-1] * 6])
    table[4, 29 // S] = 2 ** 31 - 1
    new, moves = ref.keep(table.cpu().numpy(), lengths.tolist(), path.cpu().numpy(), k.shape[0], S)
    assert new.tolist() == [26, 25, 25, 4, 27, 0]
    wk, wv = k.clone(), v.clone()
    for (p, t), (p2, t2) in moves:
        wk[p2, t2], wv[p2, t2] = wk[p, t], wv[p, t]
    got, status = tree.cache_keep(k, v, table, lengths, path, debug=True)
    assert got.tolist() == new.tolist() and torch.equal(k, wk) and torch.equal(v, wv)
    assert int(status) == tree.DATA_PATH_RANGE | decode.DATA_PAGE_RANGE | decode.DATA_LENGTH_RANGE
    assert tree.cache_keep(k, v, table, lengths, path[:, :0].contiguous()).tolist() == [30, 30, 30, 4, 30, 0]


def test_append_accept_and_keep_on_streams_and_in_graphs(tree):
    N, S, H, D, lens = 9, 16, 2, 64, [60, 33, 9]
    k0, v0, table, lengths = make_cache(lens, S, H, D, torch.bfloat16, seed=1)
    kn, vn, q = (torch.randn((3, N, h, D), generator=gen(i), device="cuda").bfloat16() for i, h in ((1, H), (2, H), (3, 8)))
    inv = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda()
    p = make_trees(3, N, 4, "random")
    parents, tokens = i32(p.tolist()), i32([[1] * N] * 3)

    def step(k, v, **kw):
        a = tree.cache_append_rotated(kn, vn, k, v, table, lengths, inv, q, **kw)
        o = tree.tree_attention(a, k, v, table, lengths, parents, **kw)
        r = tree.tree_accept(tokens, parents, tokens, **kw)
        return o, r.path, tree.cache_keep(k, v, table, lengths, r.path, **kw), k, v
    want = step(k0.clone(), v0.clone())
    side = torch.cuda.Stream()
    args = k0.clone(), v0.clone()
    side.wait_stream(torch.cuda.current_stream())
    got = step(*args, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    k, v = k0.clone(), v0.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(k, v)
    for _ in range(2):
        k.copy_(k0)
        v.copy_(v0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_gradient_and_the_native_calls_refuse_what_the_others_do(tree):
    """Results carry no gradient; wrong types, shapes and devices are told, not computed."""
    k, v, table, lengths = make_cache([20], 16, 1, 64, torch.float32, seed=1)
    q = torch.randn((1, 4, 1, 64), device="cuda", requires_grad=True)
    par = i32([[-1, 0, 0, 1]])
    assert not tree.tree_attention(q, k, v, table, lengths, par).requires_grad
    for args in ((q.bfloat16(), k, v, table, lengths, par), (q[0], k, v, table, lengths, par), (q, k, v[:1], table, lengths, par),
                 (q, k, v, table.long(), lengths, par), (q, k, v, table, lengths.long(), par), (q, k, v, table, lengths, par.long()),
                 (q, k, v, table, lengths, par[:, :3]), (q, k, v, table, lengths, par.cpu()), (q, k, v, table, lengths.cpu(), par),
                 (q, k.cpu(), v.cpu(), table, lengths, par)):
        with pytest.raises((TypeError, ValueError)):
            tree.tree_attention(*args)
    from draft_verify_acceptance_gb300.binding import SpecVerifyError
    with pytest.raises(SpecVerifyError):
        tree.tree_attention(torch.zeros((1, 257, 1, 64), device="cuda"), k, v, table, lengths, i32([[-1] * 257]))
    with pytest.raises(SpecVerifyError):
        tree.tree_accept(i32([[0] * 257]), i32([[-1] * 257]), i32([[0] * 257]))
    empty = torch.zeros((0, 4, 1, 64), device="cuda")
    assert tree.tree_attention(empty, k, v, table[:0], lengths[:0], par[:0]).shape == empty.shape
    assert tree.tree_attention(torch.zeros((1, 0, 1, 64), device="cuda"), k, v, table, lengths, par[:, :0].contiguous()).numel() == 0
    kn = torch.zeros((0, 3, 1, 64), device="cuda")
    assert tree.cache_append_rotated(kn, kn, k, v, table[:0], lengths[:0], torch.zeros(32, device="cuda")) is None
    assert tree.cache_keep(k, v, table[:0], lengths[:0], par[:0]).shape == (0,)
    assert tree.tree_accept(par[:0], par[:0], par[:0]).path.shape == (0, 4)
