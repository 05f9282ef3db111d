"""The decode-side operators against plain 64-bit references, at the sizes and masks where they can go wrong.

Tolerances.  Attention: a score is a sum of D products in fp32, off by at most (D + 8) 2^-24 sum|q||k|
scale, which moves a weight by that relative amount (twice: numerator and sum); weights, scaling and
joining add less than 2^-18 of sum p|v|; a bf16 output is rounded once, by at most 2^-8 of itself, which
is at most 2^-9 (sum p|v| + |out|).  lse is off by the score's error plus 2^-20 of its own size.  The cache operators
and the sampler's tokens are whole numbers or copies and must be equal; p = w / S is a quotient of weights
within 2^-21 of the exponential each and two roundings: 2^-19 relative for p above 2^-18 of the largest,
whose whole-number weights are rounded by 2^-22 at most.
"""
import math
import sys
import threading

import numpy as np
import pytest
import torch

import decode_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def decode():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    from draft_verify_acceptance_gb300 import decode
    return decode


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


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


def f64(t):
    return t.double().cpu().numpy()


def check_attention(out, lse, q, k, v, table, lengths, scale=None):
    D = q.shape[-1]
    scale = 1 / math.sqrt(D) if scale is None else scale
    o, l, mag, spread = ref.attention(f64(q), f64(k), f64(v), table.cpu().numpy(), lengths.cpu().numpy(), scale)
    score = (D + 8) * 2.0 ** -24 * spread
    tol = mag * (2 * score[..., None] + 2.0 ** -18) + 1e-30
    if q.dtype == torch.bfloat16:
        tol += 2.0 ** -9 * mag + 2.0 ** -9 * np.abs(o)
    err = np.abs(f64(out) - o)
    assert (err <= tol).all(), (err - tol).max()
    if lse is not None:
        got = f64(lse)
        empty = np.isinf(l)
        assert np.array_equal(np.isinf(got), empty)
        e = np.abs(got[~empty] - l[~empty])
        assert (e <= score[~empty] + 2.0 ** -20 * (1 + np.abs(l[~empty]))).all(), e.max()


# ---- attention ----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,Q,Hq,H,D,S,lens", [
    (1, 1, 1, 1, 64, 16, [1]),
    (3, 1, 4, 1, 128, 1, [1, 0, 5]),                 # an empty sequence, pages of one token
    (4, 1, 8, 2, 64, 16, [15, 16, 17, 300]),
    (3, 5, 6, 2, 128, 5, [3, 5, 77]),                # queries before the sequence's start see nothing
    (2, 7, 7, 1, 64, 48, [7, 129]),                  # odd group, page not a power of two
    (2, 17, 16, 2, 128, 8, [17, 513]),               # 136 rows a cache head
    (5, 2, 5, 5, 128, 64, [2, 63, 64, 65, 1025]),
    (1, 65, 2, 1, 64, 16, [400]),
    (40, 1, 12, 4, 128, 32, list(range(1, 41))),
    (1, 3, 8, 8, 128, 128, [6001]),                  # one sequence, cut over many blocks
    (2, 9, 32, 4, 128, 16, [2000, 31]),              # 72 rows a cache head
])
def test_attention(decode, dtype, B, Q, Hq, H, D, S, lens):
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=B * 1000 + Q)
    q = (torch.randn((B, Q, Hq, D), generator=gen(5), device="cuda") * 2).to(dtype)
    out, lse, status = decode.paged_attention(q, k, v, table, lengths, return_lse=True, debug=True)
    assert int(status) == 0
    check_attention(out, lse, q, k, v, table, lengths)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Q,G,D", [(1, 4, 128), (6, 4, 64), (4, 8, 128), (9, 8, 128), (17, 3, 64)])
def test_attention_unseen_tokens_do_not_matter(decode, dtype, Q, G, D):
    """NaN and infinities where no query looks: past the length, in unused pages, and -- for each query --
    at the later new tokens; the type's lowest value among the scores."""
    lens, S, H = [Q, 50, 333], 16, 2
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=3)
    q = torch.randn((3, Q, H * G, D), generator=gen(1), device="cuda").to(dtype)
    clean = decode.paged_attention(q, k, v, table, lengths)
    used = torch.zeros(k.shape[:2], dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for t in range(n):
            used[table[b, t // S], t % S] = True
    for bad in (math.nan, math.inf, -math.inf):
        k2, v2 = k.clone(), v.clone()
        k2[~used] = bad
        v2[~used] = bad
        assert torch.equal(decode.paged_attention(q, k2, v2, table, lengths), clean)
        for i in range(Q - 1):  # everything after query i is bad: queries up to i do not change
            for b, n in enumerate(lens):
                for t in range(max(0, n - Q + i + 1), n):
                    k2[table[b, t // S], t % S] = bad
                    v2[table[b, t // S], t % S] = bad
            if i in (0, Q // 2, Q - 2):
                k3, v3 = k2.clone(), v2.clone()
                got = decode.paged_attention(q, k3, v3, table, lengths)
                assert torch.equal(got[:, :1], clean[:, :1])
            break
        for i in range(Q - 1):
            k2, v2 = k.clone(), v.clone()
            for b, n in enumerate(lens):
                for t in range(max(0, n - Q + i + 1), n):
                    k2[table[b, t // S], t % S] = bad
                    v2[table[b, t // S], t % S] = bad
            got = decode.paged_attention(q, k2, v2, table, lengths)
            assert torch.equal(got[:, :i + 1], clean[:, :i + 1]), (bad, i)
    # a seen token's infinity or NaN does reach the result
    v2 = v.clone()
    v2[table[2, 0], 0, 0, 5] = math.nan
    got = decode.paged_attention(q, k, v2, table, lengths)
    assert torch.isnan(got[2, :, :G, 5]).all() and not torch.isnan(got[:2]).any()
    assert not torch.isnan(got[2, :, G:]).any() and torch.equal(got[2, :, :G, :5], clean[2, :, :G, :5])
    low = torch.finfo(dtype).min
    k2 = k.clone()
    k2[table[1, 0], 3] = low * 1e-3
    q1 = q.abs()
    o, l = decode.paged_attention(q1, k2, v, table, lengths, return_lse=True)
    assert torch.isfinite(o).all() and torch.isfinite(l[1]).all()


def check_nonfinite_values_of_no_weight(decode, dtype, Q, G, D, **kw):
    """A value that is not finite reaches the rows that see its token also where its weight is too small for 32 bits,
    among the last tokens (which some rows do not see) as before them."""
    n = 333
    k, v, table, lengths = make_cache([n], 16, 2, D, dtype, seed=3, **kw)
    q = torch.randn((1, Q, 2 * G, D), generator=gen(1), device="cuda").abs().to(dtype)
    for t in (5, n - Q, n - 2, n - 1):
        k2 = k.clone()
        k2[table[0, t // 16], t % 16] = -1e4
        clean = decode.paged_attention(q, k2, v, table, lengths)
        for bad in (math.inf, -math.inf, math.nan):
            v2 = v.clone()
            v2[table[0, t // 16], t % 16, 1, 3] = bad
            out = decode.paged_attention(q, k2, v2, table, lengths)
            sees = max(0, t - (n - Q))
            assert not torch.isfinite(out[0, sees:, G:, 3]).any(), (t, bad)
            out[0, sees:, G:, 3] = clean[0, sees:, G:, 3]
            assert torch.equal(out, clean), (t, bad)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Q,G,D", [(4, 4, 64), (3, 4, 128)])
def test_attention_nonfinite_values_of_no_weight(decode, dtype, Q, G, D):
    check_nonfinite_values_of_no_weight(decode, dtype, Q, G, D)


@pytest.mark.parametrize("Q,G", [(4, 8), (9, 8)])
def test_attention_many_rows_nonfinite_values_of_no_weight(decode, Q, G):
    check_nonfinite_values_of_no_weight(decode, torch.bfloat16, Q, G, 128, extra_cols=10000)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Q,G,D,extra", [(4, 4, 64, 2), (3, 4, 128, 2), (6, 4, 128, 2), (9, 8, 128, 10000)])
def test_attention_rows_do_not_depend_on_one_another(decode, dtype, Q, G, D, extra):
    """Keys that move the maximum of the queries that see them leave the other queries' results as they were, to the
    bit."""
    lens, S, H = [Q, 50, 333], 16, 2
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=3, extra_cols=extra)
    q = torch.randn((3, Q, H * G, D), generator=gen(1), device="cuda").to(dtype)
    clean = decode.paged_attention(q, k, v, table, lengths, return_lse=True)
    for size in (30.0, 1e4, 1e30):
        for i in range(Q - 1):
            k2 = k.clone()
            for b, n in enumerate(lens):
                for t in range(max(0, n - Q + i + 1), n):
                    k2[table[b, t // S], t % S] *= size
            got = decode.paged_attention(q, k2, v, table, lengths, return_lse=True)
            assert all(torch.equal(a[:, :i + 1], c[:, :i + 1]) for a, c in zip(got, clean)), (size, i)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Q,G,D,extra", [(4, 4, 64, 2), (3, 4, 128, 2), (9, 8, 128, 10000)])
def test_attention_largest_values(decode, dtype, Q, G, D, extra):
    """The type's largest values where no query looks change nothing."""
    lens, S, H = [Q, 50, 333], 16, 2
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=3, extra_cols=extra)
    q = torch.randn((3, Q, H * G, D), generator=gen(1), device="cuda").to(dtype)
    clean = decode.paged_attention(q, k, v, table, lengths)
    for most in (torch.finfo(dtype).max, torch.finfo(dtype).min):
        for i in range(Q - 1):
            k2, v2 = k.clone(), v.clone()
            for b, n in enumerate(lens):
                for t in range(max(0, n - Q + i + 1), n):
                    k2[table[b, t // S], t % S] = most
                    v2[table[b, t // S], t % S] = most
            got = decode.paged_attention(q, k2, v2, table, lengths)
            assert torch.equal(got[:, :i + 1], clean[:, :i + 1]), (most, i)


@pytest.fixture
def roomy_tables(monkeypatch):
    """Page tables with room for many tokens, which with many rows a cache head are read by another kernel."""
    plain = make_cache
    monkeypatch.setattr(sys.modules[__name__], "make_cache",
                        lambda lens, S, H, D, *args, **kw: plain(lens, S, H, D, *args, **kw,
                                                                 extra_cols=300000 // (len(lens) * S * H) + 1))


@pytest.mark.parametrize("B,Q,Hq,H,S,lens", [
    (3, 13, 6, 3, 5, [3, 13, 77]),                   # 26 rows; queries before the sequence's start see nothing
    (2, 5, 7, 1, 16, [0, 128]),                      # 35 rows, an empty sequence
    (4, 3, 32, 2, 48, [127, 128, 129, 385]),         # 48 rows, ends around a tile's
    (2, 9, 32, 4, 16, [2000, 31]),                   # 72 rows
    (1, 1, 96, 1, 64, [6001]),                       # 96 rows, one sequence cut over many blocks
    (2, 17, 16, 2, 8, [17, 513]),                    # 136 rows
    (40, 6, 8, 1, 1, list(range(1, 41))),
    (30, 10, 4, 1, 16, [300 * (i % 7) + 1 for i in range(30)]),
])
def test_attention_many_rows(decode, roomy_tables, B, Q, Hq, H, S, lens):
    test_attention(decode, torch.bfloat16, B, Q, Hq, H, 128, S, lens)


@pytest.mark.parametrize("Q,G", [(4, 8), (9, 8), (17, 6)])
def test_attention_many_rows_unseen_tokens(decode, roomy_tables, Q, G):
    test_attention_unseen_tokens_do_not_matter(decode, torch.bfloat16, Q, G, 128)


def test_attention_many_rows_repeats(decode, roomy_tables):
    """Repeated calls, and calls on a workspace that others have used, give the same bits."""
    for lens, Q, Hq, H, S in (([5000, 40], 4, 32, 4, 16), ([300] * 50, 9, 8, 2, 32)):
        k, v, table, lengths = make_cache(lens, S, H, 128, torch.bfloat16, seed=7)
        q = torch.randn((len(lens), Q, Hq, 128), generator=gen(8), device="cuda").to(torch.bfloat16)
        first = decode.paged_attention(q, k, v, table, lengths, return_lse=True)
        for _ in range(20):
            again = decode.paged_attention(q, k, v, table, lengths, return_lse=True)
            assert all(torch.equal(x, y) for x, y in zip(again, first))


def check_nan_in_a_cut_item(decode, dtype, Q, G, D, **kw):
    """A row of NaN scores, and one NaN key alone in the last tile: whichever part of a sequence that is cut over blocks
    they fall into (the number of tiles moves the cuts), the rows that see them become NaN, and no others change."""
    step = 128 if kw else 96 if dtype == torch.float32 and D == 128 else 64
    for tiles in range(9, 25):
        n = step * (tiles - 1) + Q
        k, v, table, lengths = make_cache([n], 16, 2, D, dtype, seed=tiles, **kw)
        q = torch.randn((1, Q, 2 * G, D), generator=gen(1), device="cuda").to(dtype)
        clean = decode.paged_attention(q, k, v, table, lengths, return_lse=True)
        q2 = q.clone()
        q2[0, Q - 1, G - 1, 3] = math.nan
        out, lse = decode.paged_attention(q2, k, v, table, lengths, return_lse=True)
        assert torch.isnan(out[0, Q - 1, G - 1]).all() and torch.isnan(lse[0, Q - 1, G - 1]), tiles
        out[0, Q - 1, G - 1], lse[0, Q - 1, G - 1] = clean[0][0, Q - 1, G - 1], clean[1][0, Q - 1, G - 1]
        assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])
        k2 = k.clone()
        k2[table[0, (n - Q) // 16], (n - Q) % 16, 1, 7] = math.nan  # the last tile's first token, seen by every query
        out, lse = decode.paged_attention(q, k2, v, table, lengths, return_lse=True)
        assert torch.isnan(out[0, :, G:]).all() and torch.isnan(lse[0, :, G:]).all(), tiles
        assert torch.equal(out[0, :, :G], clean[0][0, :, :G]) and torch.equal(lse[0, :, :G], clean[1][0, :, :G])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Q,G,D", [(1, 1, 64), (1, 4, 128), (3, 4, 128), (3, 8, 64)])
def test_attention_nan_in_a_cut_item(decode, dtype, Q, G, D):
    check_nan_in_a_cut_item(decode, dtype, Q, G, D)


@pytest.mark.parametrize("Q,G", [(1, 32), (9, 8)])
def test_attention_many_rows_nan_in_a_cut_item(decode, Q, G):
    check_nan_in_a_cut_item(decode, torch.bfloat16, Q, G, 128, extra_cols=10000)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_attention_layouts(decode, dtype):
    """Query from a fused projection, K and V interleaved by page, a layer of a larger cache, a table of
    strided rows, a scale, another stream: the same bits as from contiguous tensors."""
    B, Q, Hq, H, D, S = 3, 4, 8, 2, 128, 16
    k, v, table, lengths = make_cache([70, 4, 1000], S, H, D, dtype, seed=8)
    q = torch.randn((B, Q, Hq, D), generator=gen(2), device="cuda").to(dtype)
    want = decode.paged_attention(q, k, v, table, lengths, scale=0.3)
    check_attention(want, None, q, k, v, table, lengths, 0.3)
    fused = torch.zeros((B, Q, (Hq + 2 * H) * D), dtype=dtype, device="cuda")
    fused[..., :Hq * D] = q.flatten(2)
    qs = fused[..., :Hq * D].unflatten(2, (Hq, D))
    assert torch.equal(decode.paged_attention(qs, k, v, table, lengths, 0.3), want)
    qt = q.permute(1, 2, 0, 3).contiguous().permute(2, 0, 1, 3)
    assert torch.equal(decode.paged_attention(qt, k, v, table, lengths, 0.3), want)
    kv = torch.stack((k, v), 1)
    assert torch.equal(decode.paged_attention(q, kv[:, 0], kv[:, 1], table, lengths, 0.3), want)
    deep = torch.stack((v, k, v), 1), torch.stack((k, v, k), 1)
    assert torch.equal(decode.paged_attention(q, deep[0][:, 1], deep[1][:, 1], table, lengths, 0.3), want)
    wide = torch.full((B, table.shape[1] + 9), 7, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    assert torch.equal(decode.paged_attention(q, k, v, wide[:, :table.shape[1]], lengths, 0.3), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = decode.paged_attention(q, k, v, table, lengths, 0.3, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_attention_repeats_bit_for_bit_and_leaves_its_workspace_fit(decode):
    shapes = [([5000], 1, 8, 8, 128), ([3, 900, 77], 6, 8, 2, 64), ([300] * 50, 2, 4, 2, 128), ([12], 17, 16, 2, 128)]
    cases = []
    for j, (lens, Q, Hq, H, D) in enumerate(shapes):
        k, v, table, lengths = make_cache(lens, 16, H, D, torch.bfloat16, seed=j)
        q = torch.randn((len(lens), Q, Hq, D), generator=gen(j), device="cuda").to(torch.bfloat16)
        cases.append((q, k, v, table, lengths))
    want = [decode.paged_attention(*c, return_lse=True) for c in cases]
    for _ in range(30):
        for c, (o, l) in zip(cases, want):
            a, b = decode.paged_attention(*c, return_lse=True)
            assert torch.equal(a, o) and torch.equal(b, l)


def test_attention_in_a_cuda_graph(decode):
    k, v, table, lengths = make_cache([40, 700], 16, 2, 128, torch.bfloat16, seed=4)
    q = torch.randn((2, 1, 8, 128), generator=gen(4), device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    decode.paged_attention(q, k, v, table, lengths, out=out)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.zeros(decode.attention_workspace_size(2, 1, 8, 2, 128, q.dtype), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        decode.paged_attention(q, k, v, table, lengths, out=out, workspace=ws)
    for n in ([40, 700], [1, 3], [39, 0]):
        lengths.copy_(i32(n))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, decode.paged_attention(q, k, v, table, lengths))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_attention_data_errors(decode, dtype):
    """Pages out of range are skipped, lengths beyond the table are clamped, both reported."""
    lens, S, H, D = [40, 64, 33], 16, 1, 64
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=6, extra_cols=0)
    q = torch.randn((3, 2, 4, D), generator=gen(6), device="cuda").to(dtype)
    table[0, 1] = k.shape[0] + 5
    table[2, 0] = -7
    out, lse, status = decode.paged_attention(q, k, v, table, lengths, return_lse=True, debug=True)
    assert int(status) == decode.DATA_PAGE_RANGE
    check_attention(out, lse, q, k, v, table, lengths)
    lengths = i32([40, 10 ** 9, -5])
    out, lse, status = decode.paged_attention(q, k, v, table, lengths, return_lse=True, debug=True)
    assert int(status) == decode.DATA_PAGE_RANGE | decode.DATA_LENGTH_RANGE
    check_attention(out, lse, q, k, v, table, lengths)
    assert (out[2] == 0).all() and torch.isinf(lse[2]).all()


@pytest.mark.parametrize("Q", [1, 9])
def test_one_page_table_row_for_every_sequence(decode, Q):
    """Continuations that share a prompt's pages: one row expanded gives what its copies give, in every call that takes
    a table, ordinary or not; rows that overlap otherwise are refused."""
    S, H, D, N = 16, 2, 128, 5
    k, v, row, _ = make_cache([400], S, H, D, torch.bfloat16, seed=9, layers=2, spare=40, extra_cols=2400)
    table, lengths = row.expand(N, -1), i32([400, 17, 90, 0, 399])
    q = torch.randn((N, Q, 8 * H, D), generator=gen(2), device="cuda").to(torch.bfloat16)
    for kw in ({}, {"debug": True}):
        a = decode.paged_attention(q, k[0], v[0], table, lengths, return_lse=True, **kw)
        b = decode.paged_attention(q, k[0], v[0], table.contiguous(), lengths, return_lse=True, **kw)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        new = torch.randn((N, 1, H, D), generator=gen(3), device="cuda").to(torch.bfloat16)
        pools = [[x.clone() for x in (k[1], v[1])] for _ in range(2)]
        for pool, t in zip(pools, (table, table.contiguous())):
            decode.cache_append(new, new, *pool, t, lengths, **kw)
        assert all(torch.equal(x, y) for x, y in zip(*pools)) and not torch.equal(pools[0][0], k[1])
        parents, keep = i32([0, 0, 2, 4]), i32([400, 33, 90, 1])
        pools = [[x.clone() for x in (k, v)] for _ in range(2)]
        for f in (lambda c, t: decode.cache_fork(*c, t, lengths, parents, keep, 3, **kw)[:5],
                  lambda c, t: decode.cache_compact(*c, t, **kw)[:3]):
            a, b = f(pools[0], table), f(pools[1], table.contiguous())
            assert all(torch.equal(x, y) for x, y in zip(a, b)) and all(torch.equal(x, y) for x, y in zip(*pools))
    M = table.shape[1]
    overlap = torch.zeros(M + 4 * N, dtype=torch.int32, device="cuda").as_strided((N, M), (4, 1))
    for call, args in ((decode.paged_attention, (q, k[0], v[0], overlap, lengths)),
                       (decode.cache_append, (new, new, k[1], v[1], overlap, lengths)),
                       (decode.cache_fork, (k, v, overlap, lengths, parents, keep)),
                       (decode.cache_compact, (k, v, overlap))):
        with pytest.raises(ValueError):
            call(*args)


def test_attention_offsets_past_32_bits(decode):
    """Pages beyond 2^32 bytes and 2^31 elements of the pool."""
    S, H, D = 16, 8, 128
    P = (1 << 31) // (S * H * D) + 40
    k = torch.empty((P, S, H, D), dtype=torch.bfloat16, device="cuda")
    lens = [100, 37]
    ids = [P - 1, 3, P - 9, P // 2 + 1, P - 2, 11, P - 30]
    table = i32([ids, [P - 5, 7, P - 6, -1, -1, -1, -1]])
    for p in set(table.flatten().tolist()) - {-1}:
        k[p] = torch.randn((S, H, D), generator=gen(p % 1000), device="cuda").to(torch.bfloat16)
    q = torch.randn((2, 3, 16, D), generator=gen(1), device="cuda").to(torch.bfloat16)
    out, lse = decode.paged_attention(q, k, k, table, i32(lens), return_lse=True)
    flat = sorted(set(table.flatten().tolist()) - {-1})
    small = k[flat]
    remap = {p: i for i, p in enumerate(flat)}
    t2 = i32([[remap.get(p, -1) for p in row] for row in table.tolist()])
    check_attention(out, lse, q, small, small, t2, i32(lens))
    new = torch.randn((2, 3, H, D), generator=gen(9), device="cuda").to(torch.bfloat16)
    decode.cache_append(new, new, k, k, table, i32(lens))
    assert torch.equal(k[P - 30, 1:4], new[0]) and torch.equal(k[P - 6, 2:5], new[1])


# ---- append ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S,H,D,counts,before", [
    (16, 2, 64, [1, 1, 1], [0, 15, 16]),
    (5, 1, 128, [7, 0, 13, 1], [3, 9, 0, 0]),
    (64, 8, 128, [300, 2], [63, 1000]),
    (1, 3, 8, [4, 4], [0, 2]),
])
def test_append(decode, dtype, S, H, D, counts, before):
    lens = [a + b for a, b in zip(counts, before)]
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=2)
    T = sum(counts)
    new = torch.randn((T, 3, H, D), generator=gen(7), device="cuda").to(dtype)  # rows strided
    starts = i32([sum(counts[:i]) for i in range(len(counts) + 1)])
    want_k, want_v, row = k.clone(), v.clone(), 0
    for b, c in enumerate(counts):
        for i in range(c):
            t = lens[b] - c + i
            want_k[table[b, t // S], t % S] = new[row, 0]
            want_v[table[b, t // S], t % S] = new[row, 2]
            row += 1
    status = decode.cache_append(new[:, 0], new[:, 2], k, v, table, lengths, starts, debug=True)
    assert int(status) == 0 and torch.equal(k, want_k) and torch.equal(v, want_v)
    if len(set(counts)) == 1:
        k.zero_(), v.zero_()
        n = counts[0]
        decode.cache_append(new[:, 0].unflatten(0, (-1, n)), new[:, 2].unflatten(0, (-1, n)), k, v, table, lengths)
        at = [(b, lens[b] - n + i) for b in range(len(counts)) for i in range(n)]
        for r, (b, t) in enumerate(at):
            assert torch.equal(k[table[b, t // S], t % S], new[r, 0])


def test_append_data_errors(decode):
    """Rows without a sequence, position or page are skipped and reported; nothing else is written."""
    k, v, table, lengths = make_cache([20, 5], 16, 1, 64, torch.float32, seed=1, extra_cols=0)
    new = torch.randn((6, 1, 64), generator=gen(7), device="cuda")
    before = k.clone()
    lengths2 = i32([2, 5])  # sequence 0 gets four rows but has two positions
    status = decode.cache_append(new, new, k, v, table, lengths2, i32([0, 4, 6]), debug=True)
    assert int(status) == decode.DATA_LENGTH_RANGE
    want = before.clone()
    want[table[0, 0], 0:2] = new[2:4]
    want[table[1, 0], 3:5] = new[4:6]
    assert torch.equal(k, want)
    k.copy_(before)
    bad = table.clone()
    bad[0, 1] = k.shape[0]
    status = decode.cache_append(new, new, k, v, bad, i32([18, 5]), i32([1, 5, 6]), debug=True)
    assert int(status) == decode.DATA_PAGE_RANGE | decode.DATA_LENGTH_RANGE  # row 0 is nobody's
    want = before.clone()
    want[table[0, 0], 14:16] = new[1:3]
    want[table[1, 0], 4] = new[5]
    assert torch.equal(k, want)


# ---- fork and compact ----------------------------------------------------------------------------

def check_fork(decode, k, v, table, lengths, parents, keep, room, expect=0):
    S, P = k.shape[-3], k.shape[-4]
    k0, v0 = k.clone(), v.clone()
    new, lens, refs, free, copies = ref.fork(table.cpu().numpy(), lengths.cpu().numpy(), parents, keep, room, P, S)
    for _ in range(2):  # twice: the call can be repeated
        r = decode.cache_fork(k, v, table, lengths, i32(parents), i32(keep), room, debug=True)
        assert int(r.status) == expect
        assert r.page_table.tolist() == new.tolist()
        assert r.lengths.tolist() == lens.tolist()
        assert r.ref_counts.tolist() == refs.tolist()
        assert int(r.n_free) == len(free)
        assert r.free_pages.tolist() == free + [-1] * (P - len(free))
        for x, x0 in ((k, k0), (v, v0)):
            want = x0.clone()
            for a, b, n in copies:
                want[..., b, :n, :, :] = x0[..., a, :n, :, :]
            assert torch.equal(x, want)
    return r


@pytest.mark.parametrize("S,H,D,dtype,layers", [(16, 2, 64, torch.bfloat16, 3), (5, 1, 8, torch.float32, None),
                                                (1, 1, 8, torch.float32, 2), (32, 8, 128, torch.bfloat16, 1)])
def test_fork(decode, S, H, D, dtype, layers):
    lens = [3 * S + 2, 2 * S, 1, 0, 7 * S - 1]
    k, v, table, lengths = make_cache(lens, S, H, D, dtype, seed=S, layers=layers, spare=40, extra_cols=4)
    same = list(range(5))
    check_fork(decode, k, v, table, lengths, same, lens, 0)                          # nothing happens
    check_fork(decode, k, v, table, lengths, same, [max(0, n - 3) for n in lens], 4)  # rejected tokens leave
    check_fork(decode, k, v, table, lengths, [0, 0, 0, 4, 4, 1, 1, 3, -1],
               [lens[0], lens[0] - 1, S, lens[4], lens[4] - S, lens[1], 0, 0, 0], 3)  # forks, trims, an end, a start
    check_fork(decode, k, v, table, lengths, [], [], 9)                               # all end
    r = check_fork(decode, k, v, table, lengths, [4, 0, 4], [lens[4] - 1, 1, lens[4] - 1], 1)
    # and once more on its results
    check_fork(decode, k, v, r.page_table, r.lengths, [2, 0, 1, 0], [lens[4] - 1, S, 1, lens[4] - 1], 2 * S)


def test_fork_random(decode):
    rng = np.random.RandomState(3)
    for trial in range(25):
        S = int(rng.randint(1, 20))
        lens = [int(n) for n in rng.randint(0, 9 * S, rng.randint(1, 9))]
        k, v, table, lengths = make_cache(lens, S, 1, 8, torch.float32, seed=trial, spare=int(rng.randint(20, 90)),
                                          extra_cols=3)
        for _ in range(2):
            C = int(rng.randint(0, 12))
            have = lengths.tolist()
            parents = rng.randint(0, len(have), C).tolist()
            keep = [int(rng.randint(0, have[p] + 1)) if rng.rand() < 0.7 else have[p] for p in parents]
            # pages enough for every outcome, or an expected shortage
            new, lens2, refs, free, _ = ref.fork(table.cpu().numpy(), np.array(have), parents, keep, 2, k.shape[0], S)
            short = any((new[c] >= 0).sum() < min(table.shape[1], -(-(lens2[c] + 2) // S)) for c in range(C))
            full = any(-(-(int(n) + 2) // S) > table.shape[1] for n in lens2)
            r = check_fork(decode, k, v, table, lengths, parents, keep, 2,
                           (decode.DATA_CACHE_FULL if short else 0) | (decode.DATA_LENGTH_RANGE if full else 0))
            if C == 0 or short or full:
                break
            table, lengths = r.page_table, r.lengths


def test_fork_many_pages(decode):
    """More pages and sequences than one block has threads."""
    rng = np.random.RandomState(5)
    lens = rng.randint(1, 60, 700).tolist()
    k, v, table, lengths = make_cache(lens, 4, 1, 8, torch.float32, seed=1, spare=9000, extra_cols=3)
    parents = rng.randint(0, 700, 2500).tolist()
    keep = [int(rng.randint(0, lens[p] + 1)) for p in parents]
    check_fork(decode, k, v, table, lengths, parents, keep, 5)


def test_fork_data_errors(decode):
    k, v, table, lengths = make_cache([20, 33], 16, 1, 64, torch.float32, seed=1, spare=2, extra_cols=0)
    check_fork(decode, k, v, table, lengths, [0, 5, -2, 1, -1], [21, 1, 0, 33, 3], 0, decode.DATA_LENGTH_RANGE)
    check_fork(decode, k, v, table, lengths, [1, 1, 1], [33, 33, 33], 0, 0)
    check_fork(decode, k, v, table, lengths, [1, 1, 1, 0, 0, 0], [33] * 3 + [20] * 3, 0, decode.DATA_CACHE_FULL)
    check_fork(decode, k, v, table, lengths, [1], [33], 100, decode.DATA_LENGTH_RANGE | decode.DATA_CACHE_FULL
               if k.shape[0] < 3 else decode.DATA_LENGTH_RANGE)
    table[1, 1] = 99
    check_fork(decode, k, v, table, lengths, [1, 0], [33, 20], 0, decode.DATA_PAGE_RANGE)


@pytest.mark.parametrize("P,M,B,live,layers", [(1, 1, 1, 1, None), (40, 9, 5, 17, 2), (40, 9, 5, 0, 1), (64, 70, 3, 64, None),
                                               (5000, 300, 40, 2300, 1)])
def test_compact(decode, P, M, B, live, layers):
    g = gen(P)
    shape = (P, 4, 1, 8) if layers is None else (layers, P, 4, 1, 8)
    k, v = (torch.randn(shape, generator=g, device="cuda") for _ in range(2))
    ids = torch.randperm(P, generator=g, device="cuda")[:live].to(torch.int32)
    table = torch.full((B * M,), -1, dtype=torch.int32, device="cuda")
    at = torch.randperm(B * M, generator=g, device="cuda")[:min(live, B * M)]
    table[at] = ids[:len(at)]
    if live > 5:  # shared pages
        table[at[0]] = table[at[1]]
    table = table.view(B, M)
    k0, v0 = k.clone(), v.clone()
    new, refs, n, moves = ref.compact(table.cpu().numpy(), P)
    for _ in range(2):
        r = decode.cache_compact(k, v, table, debug=True)
        assert int(r.status) == 0 and int(r.n_live) == n
        assert r.page_table.tolist() == new.tolist() and r.ref_counts.tolist() == refs.tolist()
        for x, x0 in ((k, k0), (v, v0)):
            want = x0.clone()
            for a, b in moves.items():
                want[..., b, :, :, :] = x0[..., a, :, :, :]
            assert torch.equal(x, want)


@pytest.mark.parametrize("P,M,B,live", [(20000, 300, 40, 9000),     # a plan of several rounds of 8192 pages
                                        (20000, 400, 300, 11000),   # more entries than one block counts
                                        (60000, 300, 200, 20011),   # more pages than its shared memory holds
                                        (60000, 400, 300, 59990)])
def test_compact_large_pools(decode, P, M, B, live):
    g = gen(P + live)
    k, v = (torch.randn((P, 4, 1, 8), generator=g, device="cuda") for _ in range(2))
    table = torch.full((B * M,), -1, dtype=torch.int32, device="cuda")
    ids = torch.randperm(P, generator=g, device="cuda")[:live].to(torch.int32)
    at = torch.randperm(B * M, generator=g, device="cuda")
    count = min(live, B * M)
    table[at[:count]] = ids[:count]
    table[at[0]] = table[at[1]]  # a shared page
    table = table.view(B, M)
    have = table.cpu().numpy()
    used = np.unique(have[have >= 0])
    n, to = len(used), np.arange(P)
    source, dest = used[used >= n], np.setdiff1d(np.arange(n), used)
    to[source] = dest
    new = np.where(have >= 0, to[have], -1)
    refs = np.bincount(new[new >= 0], minlength=P)
    source, dest = torch.tensor(source, device="cuda"), torch.tensor(dest, device="cuda")
    want = [x.index_copy(0, dest, x[source]) for x in (k, v)]
    r = decode.cache_compact(k, v, table, debug=True)
    assert int(r.status) == 0 and int(r.n_live) == n and len(source) > 0
    assert np.array_equal(r.page_table.cpu().numpy(), new) and np.array_equal(r.ref_counts.cpu().numpy(), refs)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_compact_strided_and_errors(decode):
    kv = torch.randn((30, 2, 4, 2, 64), generator=gen(2), device="cuda").to(torch.bfloat16)
    k0 = kv.clone()
    table = i32([[29, 3, -1], [500, 7, -9]])
    r = decode.cache_compact(kv[:, 0], kv[:, 1], table, debug=True)
    assert int(r.status) == decode.DATA_PAGE_RANGE and int(r.n_live) == 3
    assert r.page_table.tolist() == [[1, 0, -1], [-1, 2, -1]] or r.page_table.tolist() == [[2, 0, -1], [-1, 1, -1]]
    for a, b in zip([3, 7, 29], [0, 1, 2]):
        assert torch.equal(kv[b], k0[a])


# ---- sampling ---------------------------------------------------------------------------------------

def check_sample(decode, x, u, settings, filtered=True, bits=0):
    """x [R, V] on the GPU, settings one (T, k, p, m) a row."""
    R, V = x.shape
    T, k, p, m = (list(c) for c in zip(*settings))
    f = lambda c: torch.tensor(c, dtype=torch.float32, device="cuda")  # noqa: E731
    r = decode.filtered_sample(x, u, f(T), top_k=i32(k), top_p=f(p), min_p=f(m), return_filtered=filtered, debug=True)
    assert int(r.status) == bits
    xs, us = x.float().cpu().numpy(), u.cpu().numpy()
    tok, ps, cnt = r.tokens.tolist(), r.p.tolist(), r.n_kept.tolist()
    fl = r.filtered.float().cpu().numpy() if filtered else None
    for i in range(R):
        j, want, kept = ref.sample_row(xs[i], us[i], T[i], k[i], p[i], m[i])
        assert (tok[i], cnt[i]) == (j, len(kept)), (i, settings[i])
        assert abs(ps[i] - want) <= 2.0 ** -19 * want + 2.0 ** -40, (i, ps[i], want)
        if filtered:
            w = np.full(V, -np.inf, np.float32)
            w[kept] = xs[i][kept]
            assert np.array_equal(fl[i], w), (i, settings[i])
    return r


MIX = [(1.0, 0, 1.0, 0.0), (0.7, 50, 0.95, 0.0), (0.8, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05), (0.6, 20, 0.8, 0.02),
       (0.0, 0, 1.0, 0.0), (1.2, 400, 1.0, 0.0), (0.9, 0, 0.6, 0.01), (1.5, 0, 0.99, 0.0), (1.0, 1, 1.0, 0.0),
       (2.0, 700, 0.9999, 1e-6), (0.05, 0, 0.5, 0.0), (1.0, 0, 0.0, 0.0), (1.0, 0, 1.0, 1.0), (30.0, 0, 0.7, 0.0),
       (1.0, 5000, 0.3, 0.0), (0.3, -4, 2.0, -1.0)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 4096, 12001, 32000, 128256, 152064, 300001])
def test_sample_settings(decode, dtype, V):
    R = len(MIX)
    for std in (3.0, 0.3):
        x = (torch.randn((R, V), generator=gen(V), device="cuda") * std).to(dtype)
        u = torch.rand(R, generator=gen(V + 1), device="cuda")
        check_sample(decode, x, u, MIX)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_ties_and_masks(decode, dtype):
    """Rows of equal logits, of two values, mostly -inf, signed zeros, the type's lowest value; uniforms at both ends."""
    for V in (5, 2048, 40008, 70001):
        base = torch.zeros((6, V), device="cuda")
        base[1] = torch.randint(0, 2, (V,), generator=gen(1), device="cuda") * 1.5
        base[2] = -math.inf
        base[2, V // 3], base[2, V - 1] = 2.0, 1.5
        base[3] = torch.where(torch.rand(V, generator=gen(2), device="cuda") < 0.5, 0.0, -0.0)
        base[4] = torch.finfo(dtype).min
        base[4, V // 2] = -3.0
        base[5] = torch.randint(0, 4, (V,), generator=gen(3), device="cuda").float()
        x = base.to(dtype)
        for u in (0.0, 0.5, 1 - 2.0 ** -24):
            for s in ((1.0, 0, 1.0, 0.0), (1.0, 3, 1.0, 0.0), (1.0, 0, 0.37, 0.0), (0.0, 0, 1.0, 0.0),
                      (0.5, V // 2, 0.9, 0.2), (3.0, 1500, 0.5, 0.0)):
                check_sample(decode, x, torch.full((6,), u, device="cuda"), [s] * 6)


def test_sample_sorted_rows_and_many_rows(decode):
    V = 32000
    x = torch.sort(torch.randn((40, V), generator=gen(4), device="cuda") * 3, dim=1).values
    x[::2] = x[::2].flip(1)
    u = torch.rand(40, generator=gen(5), device="cuda")
    check_sample(decode, x.to(torch.bfloat16), u, [MIX[i % len(MIX)] for i in range(40)])
    check_sample(decode, x, u, [MIX[i % len(MIX)] for i in range(40)], filtered=False)
    R = 1500
    x = (torch.randn((R, 700), generator=gen(6), device="cuda") * 4).to(torch.bfloat16)
    check_sample(decode, x, torch.rand(R, generator=gen(7), device="cuda"), [MIX[i % len(MIX)] for i in range(R)])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [3, 701, 5000, 40009])
def test_sample_filtered_rows_of_a_batch(decode, dtype, V):
    """Batches that several kernels share: filtered rows apart from the logits (rows on and off 16 bytes), in their
    place, flat rows and rows that are refused among them."""
    R = 330
    x = (torch.randn((R, V), generator=gen(V), device="cuda") * 3).to(dtype)
    x[5::50] *= 0.1
    u = torch.rand(R, generator=gen(V + 1), device="cuda")
    settings = [MIX[i % len(MIX)] for i in range(R)]
    want = check_sample(decode, x, u, settings)
    x[7, V // 2], x[8, V - 1], x[9] = math.nan, math.inf, -math.inf
    T, k, p, m = (list(c) for c in zip(*settings))
    f = lambda c: torch.tensor(c, dtype=torch.float32, device="cuda")  # noqa: E731
    kw = dict(temperature=f(T), top_k=i32(k), top_p=f(p), min_p=f(m), debug=True)
    good = torch.ones(R, dtype=torch.bool, device="cuda")
    good[7:10] = False
    apart = decode.filtered_sample(x, u, out=torch.full_like(x, 5.0), **kw)
    place = x.clone()
    inside = decode.filtered_sample(place, u, out=place, **kw)
    for r in (apart, inside):
        assert int(r.status) == 2  # SPEC_DATA_NONFINITE_LOGIT
        for a, b in zip(r[:4], want[:4]):
            assert torch.equal(a[good], b[good])
        assert (r.filtered[~good] == -math.inf).all() and (r.n_kept[~good] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1000, 32000, 40000, 128256, 500003])
def test_sample_sums_are_the_definition_s(decode, dtype, V):
    """p is fp32(w) / fp32(S) of the whole-number weights to the bit, so a sum that is off by little shows; the
    largest uniform draws the last token of any weight."""
    x = (torch.randn((12, V), generator=gen(V + 9), device="cuda") * 2.5).to(dtype)
    u = torch.rand(12, generator=gen(V), device="cuda")
    u[::4] = 1 - 2.0 ** -24
    for top_p in (1.0, 0.9, 0.3):
        r = decode.filtered_sample(x, u, 0.8, top_p=top_p)
        for i in range(12):
            row = x[i].float().cpu().numpy()
            j, _, kept = ref.sample_row(row, float(u[i]), 0.8, 0, top_p)
            w = ref.weights(row, 0.8)
            assert int(r.tokens[i]) == j and int(r.n_kept[i]) == len(kept)
            assert float(r.p[i]) == float(np.float32(w[j]) / np.float32(w[kept].sum()))


@pytest.mark.parametrize("V", [700, 701])
def test_sample_more_rows_than_are_listed_at_a_time(decode, V):
    """5120 rows (a batch of 1024 sequences with 4 drafted tokens), flat ones among them; in their place too."""
    R = 5120
    x = (torch.randn((R, V), generator=gen(8), device="cuda") * 4).to(torch.bfloat16)
    x[11::100] = x[11::100] * 0.02
    u = torch.rand(R, generator=gen(9), device="cuda")
    settings = [MIX[i % len(MIX)] for i in range(R)]
    want = check_sample(decode, x, u, settings)
    T, k, p, m = (list(c) for c in zip(*settings))
    f = lambda c: torch.tensor(c, dtype=torch.float32, device="cuda")  # noqa: E731
    got = decode.filtered_sample(x, u, f(T), top_k=i32(k), top_p=f(p), min_p=f(m), out=x)
    assert all(torch.equal(a, b) for a, b in zip(got[:4], want[:4]))


def test_sample_scalars_strides_and_streams(decode):
    big = (torch.randn((9, 5000), generator=gen(1), device="cuda") * 3).to(torch.bfloat16)
    u = torch.rand(9, generator=gen(2), device="cuda")
    for cols in (slice(0, 4000), slice(3, 4004), slice(8, 4009)):
        x = big[:, cols]
        want = decode.filtered_sample(x.contiguous(), u, 0.7, top_k=40, top_p=0.9, return_filtered=True)
        got = decode.filtered_sample(x, u, torch.full((9,), 0.7, device="cuda"), top_k=i32([40] * 9), top_p=0.9,
                                     return_filtered=True)
        assert all(torch.equal(a, b) for a, b in zip(got[:4], want[:4]))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        other = decode.filtered_sample(x, u, 0.7, top_k=40, top_p=0.9, return_filtered=True, stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(other[:4], want[:4]))
    x3 = big[:, :4000].contiguous().view(3, 3, 4000)
    r = decode.filtered_sample(x3, u.view(3, 3), 0.7, top_k=40, top_p=0.9)
    assert r.tokens.shape == (3, 3) and r.filtered is None
    for j in range(9):
        assert int(r.tokens.flatten()[j]) == ref.sample_row(x3.view(9, -1)[j].float().cpu().numpy(), float(u[j]), 0.7, 40, 0.9)[0]


def test_sample_out_over_other_logits_is_refused(decode):
    buf = torch.randn((5, 4008), generator=gen(1), device="cuda")
    x, u = buf[:, :4000], torch.rand(5, generator=gen(2), device="cuda")
    before = buf.clone()
    for out in (buf.view(-1)[:20000].view(5, 4000), buf.view(-1)[8:20008].view(5, 4000)):
        with pytest.raises(decode.SpecVerifyError):
            decode.filtered_sample(x, u, top_k=9, out=out)
    assert torch.equal(buf, before)
    r = decode.filtered_sample(x[:1], u[:1], top_k=9, out=x[:1])  # one row: in its place whatever the stride
    assert torch.equal(r.filtered, decode.filtered_sample(before[:1, :4000], u[:1], top_k=9, return_filtered=True).filtered)


@pytest.mark.parametrize("V", [100, 40000, 300001])
def test_sample_data_errors(decode, V):
    x = torch.randn((6, V), generator=gen(1), device="cuda")
    x[1, V // 2] = math.nan
    x[2, V - 1] = math.inf
    x[3] = -math.inf
    u = torch.full((6,), 0.5, device="cuda")
    for kw in ({}, {"top_k": 5}, {"top_p": 0.5}):
        r = decode.filtered_sample(x, u, 1.0, return_filtered=True, debug=True, **kw)
        assert int(r.status) == 2  # SPEC_DATA_NONFINITE_LOGIT
        for i in (1, 2, 3):
            assert (int(r.tokens[i]), float(r.p[i]), int(r.n_kept[i])) == (0, 0.0, 0)
            assert (r.filtered[i] == -math.inf).all()
        good = decode.filtered_sample(x[[0, 4, 5]].contiguous(), u[:3], 1.0, return_filtered=True, **kw)
        for a, b in zip(r[:4], good[:4]):
            assert torch.equal(a[[0, 4, 5]], b)
    y = x[[0, 4, 5]].contiguous()
    r = decode.filtered_sample(y, torch.tensor([0.5, 1.0, -0.1], device="cuda"), 1.0, debug=True)
    assert int(r.status) == 4 and (r.tokens >= 0).all() and (r.tokens < V).all()
    T = torch.tensor([math.nan, -1.0, 0.5], device="cuda")
    r = decode.filtered_sample(y, u[:3], T, debug=True)
    assert int(r.status) == decode.DATA_PARAM_RANGE
    for i, t in enumerate((1.0, 1.0, 0.5)):
        assert int(r.tokens[i]) == ref.sample_row(y[i].cpu().numpy(), 0.5, t)[0]


def test_filtered_rows_feed_the_verifier(decode):
    """Truncated target and drafter rows: the verifier's outputs equal the oracle's on the rows that the
    definition gives, and no token outside the kept sets is ever emitted."""
    import oracle
    from draft_verify_acceptance_gb300 import binding
    B, K, V, T = 24, 4, 5003 // 8 * 8, 0.9
    t = (torch.randn((B, K + 1, V), generator=gen(1), device="cuda") * 3).to(torch.bfloat16)
    d = (t[:, :K].float() + 0.5 * torch.randn((B, K, V), generator=gen(2), device="cuda")).to(torch.bfloat16)
    u = torch.rand((B, K + 1), generator=gen(3), device="cuda")
    draft = decode.filtered_sample(d, torch.rand((B, K), generator=gen(4), device="cuda"), T, top_k=40, top_p=0.95,
                                   return_filtered=True)
    target = decode.filtered_sample(t, u, T, top_k=40, top_p=0.95, return_filtered=True).filtered
    res = binding.verify_ex(target, draft.filtered, draft.tokens, u, T)
    assert int(res["status"]) == 0
    raw = lambda x: x.cpu().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    want = oracle.verify_ref(raw(target), raw(draft.filtered), draft.tokens.cpu().numpy(), u.cpu().numpy(), T, 0,
                             want_debug=True)
    ok = want["flags"] == 0
    assert ok.sum() > B // 2
    assert np.array_equal(res["accepted_len"].cpu().numpy()[ok], want["accepted_len"][ok])
    assert np.array_equal(res["out_tokens"].cpu().numpy()[ok], want["out_tokens"][ok])
    n, out = res["accepted_len"].tolist(), res["out_tokens"].tolist()
    for b in range(B):
        for i in range(n[b] + 1):
            assert float(target[b, i, out[b][i]]) > -math.inf


# ---- the calls themselves -----------------------------------------------------------------------

def test_ordinary_calls_and_others_agree(decode):
    """The ordinary call of each operator is made without decode.py's steps; with any further argument decode.py makes
    it.  Both give the same, and what decode.py refuses is refused."""
    calls = decode._decode_calls
    k, v, table, lengths = make_cache([40, 7, 300], 16, 2, 64, torch.bfloat16, seed=1, layers=2, spare=60, extra_cols=4)
    q = torch.randn((3, 5, 8, 64), generator=gen(2), device="cuda").to(torch.bfloat16)
    a = (q, k[0], v[0], table, lengths)
    decode.paged_attention(*a)
    plain = calls.paged_attention(*a, return_lse=True)
    out, lse, status = decode.paged_attention(*a, return_lse=True, debug=True)
    assert int(status) == 0 and torch.equal(plain[0], out) and torch.equal(plain[1], lse)
    assert torch.equal(calls.paged_attention(*a, 0.5), decode.paged_attention(*a, 0.5, debug=True)[0])
    new = torch.randn((3, 5, 2, 64), generator=gen(3), device="cuda").to(torch.bfloat16)
    kk, vv = k.clone(), v.clone()
    assert calls.cache_append(new, new * 2, k[1], v[1], table, lengths) is None
    decode.cache_append(new, new * 2, kk[1], vv[1], table, lengths, debug=True)
    assert torch.equal(k, kk) and torch.equal(v, vv)
    ragged = (new.flatten(0, 1), new.flatten(0, 1), k[0], v[0], table, lengths, i32([0, 3, 3, 15]))
    assert calls.cache_append(*ragged) is None
    parents, keep = i32([0, 2, 2, -1]), i32([40, 299, 17, 0])
    decode.cache_fork(kk, vv, table, lengths, parents, keep, 5)
    got = calls.cache_fork(kk.clone(), vv.clone(), table, lengths, parents, keep, room=5)
    want = decode.cache_fork(kk.clone(), vv.clone(), table, lengths, parents, keep, 5, debug=True)
    assert type(got) is type(want) and got.status is None and int(want.status) == 0
    assert all(torch.equal(x, y) for x, y in zip(got[:5], want[:5]))
    decode.cache_compact(kk.clone(), vv.clone(), table)
    got = calls.cache_compact(kk.clone(), vv.clone(), table)
    want = decode.cache_compact(kk.clone(), vv.clone(), table, debug=True)
    assert type(got) is type(want) and all(torch.equal(x, y) for x, y in zip(got[:3], want[:3]))
    x = (torch.randn((4, 6, 3001), generator=gen(4), device="cuda") * 3).to(torch.bfloat16)
    u = torch.rand((4, 6), generator=gen(5), device="cuda")
    kw = dict(top_k=torch.full((4, 6), 50, dtype=torch.int32, device="cuda"), top_p=0.9, return_filtered=True)
    got = calls.filtered_sample(x, u, 0.7, **kw)
    want = decode.filtered_sample(x, u, 0.7, debug=True, **kw)
    assert type(got) is type(want) and all(torch.equal(p, r) for p, r in zip(got[:4], want[:4]))
    big = (x[0, :1].expand(700, -1).contiguous(), torch.rand(700, generator=gen(6), device="cuda"))
    first = decode.filtered_sample(*big, top_p=0.9)  # (makes the workspace)
    assert torch.equal(calls.filtered_sample(*big, top_p=0.9).tokens, first.tokens)
    # everything that decode.py makes of its own, or refuses
    side = torch.cuda.Stream()
    cpu = lengths.cpu()
    for call, args, kw in ((calls.paged_attention, a, dict(debug=True)), (calls.paged_attention, a, dict(out=out)),
                           (calls.paged_attention, a, dict(stream=side)), (calls.paged_attention, a, dict(nothing=None)),
                           (calls.paged_attention, a + (0.1, True), {}), (calls.paged_attention, a, dict(scale="x")),
                           (calls.paged_attention, a, dict(q=q)), (calls.paged_attention, a[:4], {}),
                           (calls.paged_attention, (q.float(),) + a[1:], {}),
                           (calls.paged_attention, (q[:2],) + a[1:], {}),
                           (calls.paged_attention, (q, k[0], v[0].clone()[:, :8]) + a[3:], {}),
                           (calls.paged_attention, a[:4] + (lengths.long(),), {}),
                           (calls.paged_attention, a[:4] + (cpu,), {}), (calls.paged_attention, a[:3] + (table.t(), lengths), {}),
                           (calls.paged_attention, a, dict(scale=math.nan)), (calls.paged_attention, (None,) * 5, {}),
                           (calls.cache_append, (new, new, k[1], v[1], table, lengths[:2]), {}),
                           (calls.cache_append, (new, new.float(), k[1], v[1], table, lengths), {}),
                           (calls.cache_append, ragged[:6] + (i32([0, 3]),), {}),
                           (calls.cache_append, (new, new, k, v, table, lengths), {}),
                           (calls.cache_fork, (k, v, table, lengths, parents, keep[:2], 5), {}),
                           (calls.cache_fork, (k, v, table, lengths, parents, keep, 1 << 40), {}),
                           (calls.cache_fork, (k, v, table, lengths, parents, keep, -1), {}),
                           (calls.cache_fork, (k, v, table, lengths, parents, keep, 0.5), {}),
                           (calls.cache_compact, (k, v, table[0]), {}), (calls.cache_compact, (k.half(), v.half(), table), {}),
                           (calls.filtered_sample, (x, u[:2]), {}), (calls.filtered_sample, (x, u.double()), {}),
                           (calls.filtered_sample, (x, u), dict(top_k=1.5)), (calls.filtered_sample, (x, u), dict(top_p="x")),
                           (calls.filtered_sample, (x, u), dict(temperature=torch.ones(5, device="cuda"))),
                           (calls.filtered_sample, (x, u), dict(temperature=-1.0)),
                           (calls.filtered_sample, (x, u, 1.0, 5), {}), (calls.filtered_sample, (x[..., :0], u), {}),
                           (calls.filtered_sample, (x[..., ::2], u), {})):
        assert call(*args, **kw) is NotImplemented, (call, kw)


@pytest.mark.parametrize("kw", [{}, {"debug": True}])
def test_autograd_sees_what_is_written_in_place(decode, kw):
    """Results carry no gradient; a backward pass that needs what a call has overwritten raises, and does not use what
    is there now.  Inference tensors, which keep no versions, are taken too."""
    k, v, table, lengths = make_cache([20, 33], 16, 2, 64, torch.float32, seed=1, spare=9)
    new = torch.randn((2, 1, 2, 64), generator=gen(2), device="cuda")
    x, u = torch.randn((2, 500), generator=gen(3), device="cuda"), torch.rand(2, generator=gen(4), device="cuda")
    q = torch.randn((2, 1, 4, 64), generator=gen(3), device="cuda", requires_grad=True)
    out = decode.paged_attention(q, k, v, table, lengths, **kw)
    assert not (out[0] if kw else out).requires_grad
    place = torch.empty_like(q, requires_grad=False)
    calls = [(k, lambda: decode.cache_append(new, new, k, v, table, lengths, **kw)),
             (v, lambda: decode.cache_append(new, new, k, v, table, lengths, **kw)),
             (k, lambda: decode.cache_fork(k, v, table, lengths, i32([0, 0]), i32([20, 19]), 1, **kw)),
             (v, lambda: decode.cache_compact(k, v, table, **kw)),
             (place, lambda: decode.paged_attention(q, k, v, table, lengths, out=place, **kw)),
             (x, lambda: decode.filtered_sample(x, u, out=x, **kw))]
    for t, call in calls:
        for _ in range(2):  # (the first makes a workspace)
            w = torch.ones((), device="cuda", requires_grad=True)
            y = (t * w).sum()
            call()
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                y.backward()
    with torch.inference_mode():
        ki, vi = k.clone(), v.clone()
    decode.cache_append(new, new, ki, vi, table, lengths, **kw)
    decode.cache_append(new, new, k, v, table, lengths, **kw)
    assert torch.equal(ki, k) and torch.equal(vi, v)


def test_threads_on_one_stream(decode):
    """Four threads make calls of several launches on the same stream and kept workspaces, ordinary ones and others: each
    gets its own results."""
    def job(seed):
        rng = np.random.RandomState(seed)
        lens = rng.randint(1, 400, 12).tolist()
        k, v, table, lengths = make_cache(lens, 16, 1, 64, torch.float32, seed=seed, spare=90, extra_cols=3)
        parents = rng.randint(0, 12, 30).tolist()
        keep = [int(rng.randint(0, lens[p] + 1)) for p in parents]
        x = (torch.randn((330, 1000 + seed), generator=gen(seed), device="cuda") * 3).to(torch.bfloat16)
        u = torch.rand(330, generator=gen(seed), device="cuda")
        q = torch.randn((12, 1, 4, 64), generator=gen(seed), device="cuda")
        parents, keep = i32(parents), i32(keep)

        def run(**kw):
            k2, v2 = k.clone(), v.clone()
            f = decode.cache_fork(k2, v2, table, lengths, parents, keep, 5, **kw)
            c = decode.cache_compact(k2, v2, f.page_table, **kw)
            s = decode.filtered_sample(x, u, 0.9, top_p=0.8, return_filtered=True, **kw)
            a = decode.paged_attention(q, k, v, table, lengths, return_lse=True, **kw)
            return [k2, v2, *f[:5], *c[:3], *s[:4], *a[:2]]
        return run
    jobs = [job(seed) for seed in range(4)]
    want = [run() for run in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(run, want):
        for i in range(60):
            got = run(debug=True) if i % 2 else run()
            if not all(torch.equal(a, b) for a, b in zip(got, want)):
                wrong.append(i)
    threads = [threading.Thread(target=work, args=a) for a in zip(jobs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_workspaces_are_zero_filled_no_further_than_needed(decode, monkeypatch):
    """Beyond its first bytes a workspace may hold anything, and a captured call, whose workspace is made fit at every
    replay, fills no more than those."""
    k, v, table, lengths = make_cache([40, 700, 9000], 16, 2, 128, torch.bfloat16, seed=1, spare=90)
    few, many = (torch.randn((3, n, 16, 128), generator=gen(2), device="cuda").to(torch.bfloat16) for n in (1, 9))
    wide = torch.cat([table, torch.full((3, 9000), -1, dtype=torch.int32, device="cuda")], 1)
    x = (torch.randn((400, 4001), generator=gen(4), device="cuda") * 3).to(torch.bfloat16)
    x[::9] *= 0.1
    u = torch.rand(400, generator=gen(5), device="cuda")
    parents, keep = i32([2, 1, 1]), i32([77, 3, 700])
    lib = decode._lib
    calls = [("attention", decode.attention_workspace_size(3, 9, 16, 2, 128, few.dtype),
              lambda **kw: [decode.paged_attention(few, k, v, table, lengths, **kw)]),
             ("attention", decode.attention_workspace_size(3, 9, 16, 2, 128, few.dtype),
              lambda **kw: [decode.paged_attention(many, k, v, wide, lengths, **kw)]),
             ("sample", lib.spec_filtered_sample_workspace_size(400, 4001, 1),
              lambda **kw: decode.filtered_sample(x, u, top_p=0.9, return_filtered=True, **kw)[:4]),
             ("fork", lib.spec_cache_fork_workspace_size(k.shape[0], 3),
              lambda **kw: decode.cache_fork(k.clone(), v.clone(), table, lengths, parents, keep, 5, **kw)[:5]),
             ("compact", lib.spec_cache_compact_workspace_size(k.shape[0]),
              lambda **kw: decode.cache_compact(k.clone(), v.clone(), table, **kw)[:3])]
    for kind, nbytes, call in calls:
        want = call()
        for fill in (0xff, 0x01):
            ws = torch.full((nbytes,), fill, dtype=torch.uint8, device="cuda")
            ws[:decode._KINDS[kind][1]] = 0
            for _ in range(2):
                assert all(torch.equal(a, b) for a, b in zip(call(workspace=ws), want)), kind
    filled = []
    zeros, zero_ = torch.zeros, torch.Tensor.zero_
    monkeypatch.setattr(torch, "zeros", lambda n, *a, **kw: filled.append(n) or zeros(n, *a, **kw))
    monkeypatch.setattr(torch.Tensor, "zero_", lambda t: filled.append(t.numel()) or zero_(t))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
        for _, _, call in calls:
            call()
    assert filled == [2048, 2048, 64]


def test_calls_in_a_graph_own_their_workspaces(decode):
    """Captured calls without a workspace of the caller's: replays are right after eager calls that need larger
    workspaces, and eager calls after a capture that was never replayed."""
    k, v, table, lengths = make_cache([40, 700, 3000], 16, 2, 128, torch.bfloat16, seed=1)
    q = torch.randn((3, 1, 8, 128), generator=gen(2), device="cuda").to(torch.bfloat16)
    x = (torch.randn((400, 4001), generator=gen(4), device="cuda") * 3).to(torch.bfloat16)
    u = torch.rand(400, generator=gen(5), device="cuda")
    parents, keep = i32([2, 1, 1]), i32([77, 3, 700])

    def run():
        return (decode.paged_attention(q, k, v, table, lengths), decode.filtered_sample(x, u, top_p=0.9).tokens,
                *decode.cache_fork(k.clone(), v.clone(), table, lengths, parents, keep, 5)[:5],
                *decode.cache_compact(k.clone(), v.clone(), table)[:3])
    want = run()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()  # (workspaces of this stream exist before the capture)
        side.synchronize()
        graph, never = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(never, stream=side):
            run()
        with torch.cuda.graph(graph, stream=side):
            got = run()
        big = make_cache([4000] * 40, 16, 8, 128, torch.bfloat16, seed=3)
        for _ in range(3):
            decode.paged_attention(torch.randn((40, 4, 32, 128), generator=gen(2), device="cuda").to(torch.bfloat16), *big)
            decode.filtered_sample(x.repeat(4, 1), u.repeat(4), top_p=0.9)
            assert all(torch.equal(a, b) for a, b in zip(run(), want))
            for t in got:
                t.fill_(-7)
            graph.replay()
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
