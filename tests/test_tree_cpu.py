"""CPU-only checks of the tree operators' entry points: exports, constants, refusals on the host before any launch, and the
binding's own checks.  No kernel is launched here."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import tree_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "spec_tree.h")
FAKE = 1 << 20  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def tree():
    import __graft_entry__
    __graft_entry__.build()
    from draft_verify_acceptance_gb300 import tree
    return tree


def test_exports_and_constants(tree):
    from draft_verify_acceptance_gb300 import binding, decode
    src = open(HEADER).read()
    names = set(re.findall(r"SPEC_API\s+[\w\s\*]+?\b(spec_\w+)\s*\(", src))
    assert names == set(tree.EXPORTS)
    for n in names:
        assert getattr(tree._lib, n)._flags_ & 4, n  # keeps the interpreter's lock
    defs = {k: int(v) for k, v in re.findall(r"#define\s+SPEC_(\w+)\s+(\d+)", src)}
    assert defs == {"DATA_TREE_PARENT": tree.DATA_TREE_PARENT, "DATA_PATH_RANGE": tree.DATA_PATH_RANGE,
                    "TREE_MAX_NODES": tree.MAX_NODES, "TREE_ATTENTION_ZERO_BYTES": decode._KINDS["tree"][1]}
    taken = [getattr(m, k) for m in (binding, decode) for k in dir(m) if k.startswith("DATA_")] + [binding.DEVICE_WAIT_TIMEOUT, 32]
    assert not {tree.DATA_TREE_PARENT, tree.DATA_PATH_RANGE} & set(taken)


def test_header_is_plain_c(tmp_path):
    f = tmp_path / "h.c"
    f.write_text('#include "spec_tree.h"\nint main(void) { return SPEC_TREE_MAX_NODES - 256; }\n')
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-I", os.path.dirname(HEADER),
                        str(f)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def cache(tree, **kw):
    d = dict(k=FAKE, v=FAKE, layer_stride=0, page_stride=16 * 2 * 64, token_stride=128, layers=1, pages=8, page_size=16,
             heads=2, head_dim=64, dtype=0)
    d.update(kw)
    return tree._Cache(*(d[n] for n, _ in tree._Cache._fields_))


BAD_CACHES = [(dict(k=0), 1), (dict(v=FAKE + 4), 1), (dict(layers=0), 1), (dict(pages=-1), 1), (dict(page_size=0), 1),
              (dict(heads=0), 1), (dict(dtype=2), 1), (dict(token_stride=127), 1), (dict(page_stride=100), 1),
              (dict(page_size=1 << 17), 2)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_cache_refusals(tree, kw, code):
    c, lib = cache(tree, **kw), tree._lib
    assert lib.spec_cache_keep(ctypes.byref(c), FAKE, 4, 4, FAKE, 2, FAKE, 3, FAKE + 64, None, None) == code
    assert lib.spec_cache_append_rotated(FAKE, FAKE, 128, 4, None, None, 0, 0, None, 0, None, FAKE, 32, 0, ctypes.byref(c), FAKE, 4,
                                         4, FAKE, 2, None, None) == code
    assert lib.spec_tree_attention(FAKE, 256, 256, 64, ctypes.byref(c), FAKE, 4, 4, FAKE, FAKE, 1, 2, 1, 4, 0.1, FAKE + 4096,
                                   None, FAKE, 1 << 30, None, None) == code


def test_attention_refusals(tree):
    lib = tree._lib
    need = lib.spec_tree_attention_workspace_size(2, 3, 4, 2, 64, 0)
    assert need > 0 and need % 256 == 0

    def call(q=FAKE, qs=(768, 256, 64), c=None, table=FAKE, ts=4, M=4, lens=FAKE, par=FAKE, ps=3, B=2, N=3, Hq=4, scale=0.1,
             out=FAKE + 8192, lse=None, ws=FAKE, n=None, st=None):
        c = c if c is not None else cache(tree)
        return lib.spec_tree_attention(q, *qs, ctypes.byref(c), table, ts, M, lens, par, ps, B, N, Hq, scale, out, lse, ws,
                                       need if n is None else n, None, st)
    for bad in (dict(q=0), dict(q=FAKE + 8), dict(qs=(2, 256, 64)), dict(qs=(-256, 256, 64)), dict(table=0), dict(ts=3),
                dict(M=-1), dict(lens=0), dict(lens=FAKE + 2), dict(par=0), dict(par=FAKE + 1), dict(ps=2), dict(ps=-3),
                dict(B=-1), dict(N=-1), dict(Hq=3), dict(Hq=0), dict(out=0), dict(out=FAKE), dict(out=FAKE + 6128),
                dict(out=FAKE - 16), dict(lse=FAKE + 1), dict(ws=0), dict(n=need - 1), dict(ws=FAKE + 8),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(st=FAKE + 2),
                dict(c=cache(tree, layers=2, layer_stride=1 << 14))):
        assert call(**bad) == 1, bad
    assert call(c=cache(tree, head_dim=96, token_stride=192, page_stride=4096)) == 2
    assert call(N=257, ps=257) == 2
    assert call(M=1 << 28, ts=1 << 28) == 2
    assert call(B=0, q=0, lens=0, out=0, ws=0, par=0) == 0
    assert call(N=0, q=0, lens=0, out=0, ws=0, par=0) == 0
    for bad in ((-1, 1, 4, 2, 64, 0), (2, 1, 3, 2, 64, 0), (2, 1, 4, 2, 96, 0), (2, 1, 4, 0, 64, 0), (2, 1, 4, 2, 64, 5),
                (2, 257, 4, 2, 64, 0), (2, -1, 4, 2, 64, 0)):
        assert lib.spec_tree_attention_workspace_size(*bad) == 0


def test_append_refusals(tree):
    lib = tree._lib

    def call(k=FAKE, v=FAKE, stride=128, T=4, starts=None, q=FAKE + 65536, qs=256, hq=4, out=FAKE + (2 << 16), os_=256, pos=None,
             freq=FAKE, F=32, c=None, lens=FAKE, B=2):
        c = c if c is not None else cache(tree)
        return lib.spec_cache_append_rotated(k, v, stride, T, starts, q, qs, hq, out, os_, pos, freq, F, 0, ctypes.byref(c), FAKE,
                                             4, 4, lens, B, None, None)
    for bad in (dict(k=0), dict(v=FAKE + 4), dict(stride=127), dict(stride=129), dict(T=-1), dict(T=5), dict(B=0), dict(B=-1),
                dict(lens=0), dict(starts=FAKE + 1), dict(q=0), dict(q=FAKE + 8), dict(qs=255), dict(qs=258), dict(hq=-1),
                dict(out=0), dict(out=FAKE + 65536 + 16), dict(os_=255), dict(os_=257), dict(pos=FAKE + 2), dict(freq=0), dict(freq=FAKE + 1),
                dict(F=-8), dict(F=40), dict(out=FAKE + 65536, os_=260), dict(out=FAKE + 16), dict(out=FAKE),
                dict(c=cache(tree, layers=2, layer_stride=1 << 14))):
        assert call(**bad) == 1, bad
    assert call(F=12) == 2
    assert call(c=cache(tree, heads=1, head_dim=264, token_stride=264, page_stride=264 * 16), hq=0) == 2
    assert call(c=cache(tree, heads=1, head_dim=12, token_stride=12, page_stride=192), F=0, hq=0) == 2
    assert call(T=0, k=0, v=0) == 0


def test_accept_and_keep_refusals(tree):
    lib, c = tree._lib, cache(tree)

    def accept(tok=FAKE, par=FAKE, ps=5, drawn=FAKE, B=2, N=5, n=FAKE, out=FAKE, path=FAKE, st=None):
        return lib.spec_tree_accept(tok, par, ps, drawn, B, N, n, out, path, None, st)
    for bad in (dict(tok=0), dict(tok=FAKE + 1), dict(par=0), dict(ps=4), dict(ps=-5), dict(drawn=0), dict(B=-1), dict(N=-1),
                dict(n=0), dict(out=FAKE + 2), dict(path=0), dict(st=FAKE + 1)):
        assert accept(**bad) == 1, bad
    assert accept(N=257, ps=257) == 2
    assert accept(B=0, tok=0, par=0, drawn=0, n=0, out=0, path=0) == 0

    def keep(table=FAKE, ts=4, M=4, lens=FAKE, B=2, path=FAKE, N=3, new=FAKE + 64, st=None, c=c):
        return lib.spec_cache_keep(ctypes.byref(c), table, ts, M, lens, B, path, N, new, None, st)
    for bad in (dict(table=0), dict(ts=3), dict(lens=0), dict(B=-1), dict(path=0), dict(N=-1), dict(new=0), dict(new=FAKE),
                dict(new=FAKE + 4), dict(st=FAKE + 3)):
        assert keep(**bad) == 1, bad
    assert keep(N=(1 << 20) + 1) == 2
    assert keep(B=1 << 29, c=cache(tree, layers=32, layer_stride=1 << 14)) == 2
    assert keep(B=0, lens=0, path=0, new=0) == 0


def test_binding_refuses_cpu_tensors_and_bad_parents(tree):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    pages = torch.zeros(3, 4, 1, 64)
    with pytest.raises(ValueError):
        tree.tree_attention(torch.zeros(1, 2, 1, 64), pages, pages, i32(1, 1), i32(1), i32(1, 2))
    with pytest.raises(ValueError):
        tree.cache_append_rotated(torch.zeros(1, 2, 1, 64), torch.zeros(1, 2, 1, 64), pages, pages, i32(1, 1), i32(1), torch.zeros(32))
    with pytest.raises(ValueError):
        tree.tree_accept(i32(1, 2), i32(1, 2), i32(1, 2))
    with pytest.raises(ValueError):
        tree.cache_keep(pages, pages, i32(1, 1), i32(1), i32(1, 2))
    p = i32(3, 5)
    assert tree._parents(p, 3, 5, -1) == (p.data_ptr(), 5)
    assert tree._parents(p[0], 3, 5, -1) == (p.data_ptr(), 0)
    assert tree._parents(p[:1].expand(3, 5), 3, 5, -1) == (p.data_ptr(), 0)
    assert tree._parents(i32(3, 9)[:, :5], 3, 5, -1)[1] == 9
    for bad in (i32(5, 3).t(), i32(2, 5), i32(4), torch.arange(9, dtype=torch.int32).as_strided((3, 5), (2, 1))):
        with pytest.raises(ValueError):
            tree._parents(bad, 3, 5, -1)
    with pytest.raises(TypeError):
        tree._parents(p.long(), 3, 5, -1)


def test_the_turns_and_the_series():
    """Angles in fixed point and the sine and cosine by their series, as tree_cache.cu has them: within 2^-31 of a turn and
    2^-23 of the functions.  Its fused multiply-adds are a 64-bit product and sum rounded once."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    f, pi = np.float32, Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    src = open(os.path.join(ROOT, "draft_verify_acceptance_gb300", "csrc", "tree_cache.cu")).read()
    inv = int(re.search(r"kInv2Pi = (0x[0-9a-f]+)ull", src).group(1), 16)
    assert inv == int(Decimal(2) ** 64 / (2 * pi))

    def turns(x):
        u = int(f(x).view(np.uint32))
        e, m = (u >> 23) & 255, (u & 0x7fffff) | (0x800000 if (u >> 23) & 255 else 0)
        s = 150 - (e or 1)
        t = (m * inv >> s if s >= 0 else m * inv << -s) & (2 ** 64 - 1)
        return -t if u >> 31 else t
    for x in [500000.0 ** (-i / 64) for i in range(64)] + [10000.0 ** (-i / 32) for i in range(32)] + [0.0, 2.5, -0.3, 1e-40]:
        for p in (0, 1, 131072, 1000000, 2 ** 31 - 1, -5):
            d = abs(Decimal(p * turns(x) % 2 ** 64) / 2 ** 64 - Decimal(p) * Decimal(float(f(x))) / (2 * pi)) % 1
            assert min(d, 1 - d) < Decimal(2) ** -31

    phase = np.random.RandomState(0).randint(0, 2 ** 32, 1 << 20, dtype=np.uint64)
    quarter = ((phase + 0x20000000) & 0xffffffff) >> 30
    fma = lambda a, b, c: (np.float64(a) * np.float64(b) + np.float64(c)).astype(f)  # noqa: E731
    x = ((phase - (quarter << 30)) & 0xffffffff).astype(np.uint32).view(np.int32).astype(f) * f(1.46291807926716e-9)
    z = x * x
    s = fma(z, f(2.7557319e-6), f(-1.9841270e-4))
    s = fma(z * x, fma(z, fma(z, s, f(8.3333333e-3)), f(-1.6666667e-1)), x)
    c = fma(z, f(-2.7557319e-7), f(2.4801587e-5))
    c = fma(z, fma(z, fma(z, fma(z, c, f(-1.3888889e-3)), f(4.1666667e-2)), f(-0.5)), f(1))
    a, b = np.where(quarter & 1, s, c), np.where(quarter & 1, c, s)
    a, b = np.where((quarter + 1) & 2, -a, a), np.where(quarter & 2, -b, b)
    t = phase.astype(np.float64) * (2 * np.pi / 2 ** 32)
    assert np.abs(a - np.cos(t)).max() < 2.0 ** -23 and np.abs(b - np.sin(t)).max() < 2.0 ** -23
    for k in ("1.46291807926716e-9f", "2.7557319e-6f", "-1.9841270e-4f", "8.3333333e-3f", "-1.6666667e-1f", "-2.7557319e-7f",
              "2.4801587e-5f", "-1.3888889e-3f", "4.1666667e-2f"):
        assert k in src


def test_the_reference_walk():
    """The reference's own pieces, by hand: a tree of two branches."""
    parents = np.array([[-1, 0, 0, 1, 2, 2, -2, 6, 8]])
    assert ref.line(parents[0], 5) == [5, 2, 0]
    assert all(ref.line(parents[0], i) is None for i in (6, 7, 8))
    tokens, drawn = np.array([[9, 4, 5, 6, 7, 7, 1, 1, 1]]), np.array([[5, 0, 7, 0, 3, 0, 0, 0, 0]])
    n, out, path = ref.accept(tokens, parents, drawn)
    assert n[0] == 2 and path[0, :4].tolist() == [0, 2, 4, -1] and out[0, :4].tolist() == [5, 7, 3, -1]
    new, moves = ref.keep(np.array([[3, 1, 0]]), np.array([13]), path, 4, 5)
    assert new[0] == 7 and moves == [((1, 1), (1, 0)), ((1, 3), (1, 1))]


def test_append_in_place_refuses_new_rows_that_share_its_queries(tree):
    """q rotated in place (q_out is q): another warp of the token may already have written the queries that new keys or values
    share bytes with.  Rows that lie in one another's gaps are no overlap (test_gpu_tree.py runs those)."""
    lib, Q = tree._lib, FAKE + 65536
    c = cache(tree)  # rows of 128 floats

    def call(k=FAKE, v=FAKE, stride=128, T=4, q=Q, qs=128, hq=2, out=None, os_=None):
        return lib.spec_cache_append_rotated(k, v, stride, T, None, q, qs, hq, q if out is None else out, qs if os_ is None else os_,
                                             None, FAKE, 32, 0, ctypes.byref(c), FAKE, 4, 4, FAKE, 2, None, None)
    row = 128 * 4
    for bad in (dict(k=Q), dict(v=Q), dict(k=Q, v=Q), dict(k=Q + 16), dict(v=Q - 16), dict(k=Q + 3 * row), dict(v=Q - 3 * row),
                # slices of a fused row of 512 floats: 256 of queries, then keys and values that begin too early or wrap
                dict(qs=512, stride=512, hq=4, k=Q + 2 * row - 16), dict(qs=512, stride=512, hq=4, v=Q + 3 * row + 16),
                dict(qs=512, stride=512, hq=4, k=Q - row + 16), dict(qs=512, stride=512, hq=4, v=Q + 8 * row),
                dict(qs=512, stride=512, hq=4, k=Q - 8 * row),
                # other strides, one row
                dict(qs=256, hq=4, k=Q), dict(qs=256, hq=4, v=Q + 6 * row), dict(T=2, qs=256, hq=4, k=Q + 512, stride=512)):
        assert call(**bad) == 1, bad
    lib_one = lambda **kw: lib.spec_cache_append_rotated(  # noqa: E731
        kw.get("k", FAKE), kw.get("v", FAKE), 128, 1, None, Q, 4096, 2, Q, 128, None, FAKE, 32, 0, ctypes.byref(c), FAKE, 4, 4, FAKE, 1,
        None, None)
    for bad in (dict(k=Q), dict(v=Q + row - 16), dict(k=Q - row + 16)):
        assert lib_one(**bad) == 1, bad


def test_the_rows_overlap_rule_against_bytes(tmp_path):
    """spec_checks.h's rule for rows of one stride, and its range rule else, against the bytes themselves."""
    src = tmp_path / "rows.cpp"
    src.write_text('#include "spec_checks.h"\n'
                   'extern "C" int rows(long a, long as, long na, long b, long bs, long nb, long T) {\n'
                   '  return specv::rows_overlap(reinterpret_cast<void*>(a), as, na, reinterpret_cast<void*>(b), bs, nb, T); }\n')
    out = tmp_path / "rows.so"
    from draft_verify_acceptance_gb300 import build
    r = subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC, "-I", os.path.join(os.path.dirname(os.path.dirname(build._nvcc())), "include"),
                        str(src), "-o", str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    rows = ctypes.CDLL(str(out)).rows
    rows.argtypes = [ctypes.c_long] * 7
    rng = np.random.RandomState(0)
    met = [0, 0]
    for _ in range(20000):
        T, s, na, nb = rng.randint(1, 6), rng.randint(4, 20), 0, 0
        na, nb = rng.randint(1, s + 1), rng.randint(1, s + 1)
        a, b = 1000, 1000 + rng.randint(-6 * s, 6 * s)
        bytes_a = {a + t * s + i for t in range(T) for i in range(na)}
        bytes_b = {b + t * s + i for t in range(T) for i in range(nb)}
        share = bool(bytes_a & bytes_b)
        assert rows(a, s, na, b, s, nb, T) == share, (T, s, na, nb, b - a)
        met[share] += 1
        if rows(a, s, na, b, s + 4, nb, T) == 0:  # of other strides: never too lax
            assert not bytes_a & {b + t * (s + 4) + i for t in range(T) for i in range(nb)}
    assert min(met) > 3000


def told_items_read_too_late(tiles, dual, items, held):
    """The protocol of attention_tree_tc.cuh's warps over one block's items of `tiles` tiles each, as a graph of what waits for
    what: (warp, item) pairs whose reading of an item is not ordered before the walker tells another into its place, and
    whether the whole comes to an end.  Waits for ring slots and score buffers are left out: they only order more."""
    n, after = len(tiles), {}

    def event(e, *before):
        after.setdefault(e, set()).update(b for b in before if b is not None)
    of = [k for k, t in enumerate(tiles) for _ in range(t)]  # a tile's item
    start = np.concatenate([[0], np.cumsum(tiles)]).tolist()
    for k in range(n + 1):  # the last says that there are no more
        event(("told", k), ("told", k - 1) if k else None)
        if k >= items:
            event(("told", k), *(("free", s, k - items) for s in (0, 1)))

    def read(warp, k, *before):  # a warp's reads come in order
        event((warp, k), ("told", k), (warp, k - 1) if k else None, *before)
    for pair in (0, 1):  # loaders of the even and the odd tiles, K's and V's alike
        seen = -1
        for u in range(pair, len(of) + 5, 2):  # looks up tile u, then copies tile u - 4
            last = of[u] if u < len(of) else n
            for k in range(seen + 1, last + 1):
                read(("load", pair), k, ("copied", u - 6) if u >= 6 else None)
            seen = max(seen, last)
            if 0 <= u - 4 < len(of):
                event(("copied", u - 4), (("load", pair), seen), ("copied", u - 6) if u >= 6 else None)
    for k in range(n + 1):
        read("queries", k, ("queried", k - 1) if 1 < k <= n else None)
        if 0 < k < n:
            event(("queried", k), ("queries", k), ("scores", 1, start[k] - 1))  # the scores of the item before are done
        for warp in ("scores", "outputs"):
            read((warp,), k, (warp, 1, start[k] - 1) if k else None)
        for s in (0, 1):
            mine = [start[j + 1] - 1 for j in range(k) if dual or s == 0 or tiles[j] > 1]
            event(("start", s, k), ("told", k), ("start", s, k - 1) if k else None,
                  ("outputs", 1, mine[-1]) if mine else None)
            if not dual and k:  # the streams' outputs are joined
                event(("start", s, k), ("start", 1 - s, k - 1), ("outputs", 1, start[k] - 1))
            if k >= held:
                event(("free", s, k - held), ("start", s, k))
    for t, k in enumerate(of):
        event(("scores", 1, t), (("scores",), k), ("scores", 1, t - 1) if t else None, ("copied", t),
              ("queried", k) if k else ("start", 0, 0))
        for s in ((0, 1) if dual else ((t - start[k]) % 2,)):
            event(("weights", s, t), ("scores", 1, t), ("start", s, k))
            event(("outputs", 1, t), ("weights", s, t))
        event(("outputs", 1, t), (("outputs",), k), ("outputs", 1, t - 1) if t else None, ("copied", t))

    order, state = [], {}
    for root in after:  # depth first; an event met again on its own line waits for itself
        stack = [(root, iter(after.get(root, ())))]
        if state.setdefault(root, 1) == 2:
            continue
        while stack:
            e, rest = stack[-1]
            x = next(rest, None)
            if x is None:
                state[e] = 2
                order.append(e)
                stack.pop()
            elif state.get(x) == 1:
                return None, False
            elif x not in state:
                state[x] = 1
                stack.append((x, iter(after.get(x, ()))))
    bit = {e: 1 << i for i, e in enumerate(order)}
    upto = {}
    for e in order:
        upto[e] = bit[e]
        for x in after.get(e, ()):
            upto[e] |= upto[x]
    readers = [("load", 0), ("load", 1), "queries", ("scores",), ("outputs",)]
    late = [(w, k) for k in range(n + 1 - items) for w in readers if not upto[("told", k + items)] & bit[(w, k)]]
    return late, True


def test_told_items_stay_until_every_warp_has_read_them():
    """An item's place is told again after the softmax warps give it up.  Given up as they start the next one, a block's first
    item was held for nobody else: the queries' warp and, after one tile, the odd tiles' loaders might not have looked."""
    src = open(os.path.join(ROOT, "draft_verify_acceptance_gb300", "csrc", "attention_tree_tc.cuh")).read()
    items = int(re.search(r"constexpr int kItems = (\d+);", src).group(1))
    held = re.search(r"constexpr int kHeld = (\d+);", src)
    held = int(held.group(1)) if held else 1
    assert f"items >= kHeld && row_in == 0) mbar_arrive(&sh.item_free[(items - kHeld) % kItems])" in src or held == 1
    late, ends = told_items_read_too_late([1] * 20, False, items, 1)
    assert ends and set(late) == {("queries", 0), (("load", 1), 0)}
    rng = np.random.RandomState(0)
    for dual in (False, True):
        for case in range(40):
            tiles = [1] * 20 if case == 0 else rng.randint(1, 2 + case % 5, 24).tolist()
            late, ends = told_items_read_too_late(tiles, dual, items, held)
            assert ends and late == [], (tiles, dual)


def test_turns_of_high_frequencies_and_the_phase():
    """tree_cache.cu's turns and the 32-bit phase that the sine takes, within 2^-31 of a turn for every finite frequency and
    position, against the exact fraction."""
    src = open(os.path.join(ROOT, "draft_verify_acceptance_gb300", "csrc", "tree_cache.cu")).read()
    inv = int(re.search(r"kInv2Pi = (0x[0-9a-f]+)ull", src).group(1), 16)
    words = re.search(r"kInv2PiWords\[7\] = \{[^\n]*\n([^}]*)\}", src)
    words = [int(w, 16) for w in re.findall(r"0x([0-9a-f]+)u", words.group(1))] if words else None
    low, full = (1 << 64) - 1, (1 << 32) - 1
    if words:
        assert len(words) == 7 and words[0] << 32 | words[1] == inv
        bits = sum(w << 192 - 32 * i for i, w in enumerate(words))
        assert abs(bits / 2 ** 224 - 1 / (2 * np.pi)) < 1e-16

    def kernel(x):
        u = int(np.float32(x).view(np.uint32))
        e, m = (u >> 23) & 255, (u & 0x7fffff) | (0x800000 if (u >> 23) & 255 else 0)
        shift = 150 - (e or 1)
        if words and u & 0x7fffffff > 0x3f800000:
            k = -shift
            at, bit = (k >> 5, k & 31) if k > 0 else (0, 0)
            w = [(words[at + i] << 32 | words[at + i + 1]) << bit >> 32 & full for i in range(3)]
            first, rest = m * w[0], m * w[1] + (m * w[2] >> 32)
            assert first <= low and rest <= low
            lo = rest + (first << 32) & low
            t = lo if k >= 0 else lo >> -k | ((first >> 32) + (lo < rest)) << 64 + k & low
        else:
            t = m * inv >> shift & low if shift >= 0 else (m * inv << -shift & low if shift > -64 else 0)
        return -t & low if u >> 31 else t
    rng = np.random.RandomState(1)
    some = [1.0, np.nextafter(np.float32(1), np.float32(0)), np.nextafter(np.float32(1), np.float32(2)), 1.75, 2.5, -3.0, 1e4, 2.0 ** 23,
            2.0 ** 24 - 1, 2.0 ** 24, 1e9, -1e20, 3.4028235e38, 500000.0 ** -0.3, 1e-40, 0.0]
    some += (rng.uniform(1, 2, 300) * 2.0 ** rng.randint(-30, 127, 300)).tolist()
    for x in some:
        x = float(np.float32(x))
        t = kernel(x)
        for p in (1, 2, 131071, 2 ** 31 - 1, -2 ** 31, int(rng.randint(1, 2 ** 31 - 1))):
            d = abs((p * t & low) >> 32) / 2 ** 32 - ref.turns(p, x)
            assert min(abs(d), 1 - abs(d)) < 2.0 ** -31, (x, p, d)


def test_accept_and_keep_refuse_outputs_over_what_others_read(tree):
    """Results over memory that another tree's warp, or another block, may still read."""
    lib, c, B, N = tree._lib, cache(tree), 4, 8
    far = [FAKE + (i << 12) for i in range(6)]

    def accept(tok=far[0], par=far[1], ps=N, drawn=far[2], n=far[3], out=far[4], path=far[5]):
        return lib.spec_tree_accept(tok, par, ps, drawn, B, N, n, out, path, None, None)
    row = 4 * N
    for bad in (dict(n=far[0]), dict(n=far[0] + B * row - 4), dict(n=far[1] + 16), dict(n=far[2] - 4), dict(n=far[4]), dict(n=far[5] + 4),
                dict(path=far[4]), dict(path=far[4] + row), dict(out=far[0] + row), dict(out=far[2] - row), dict(path=far[1] + 4),
                dict(path=far[1], ps=0), dict(out=far[1], ps=0), dict(path=far[1], ps=N + 2), dict(out=far[1] + row, ps=N)):
        assert accept(**bad) == 1, bad

    def keep(lens=far[0], table=far[1], path=far[2], new=far[3], ts=4):
        return lib.spec_cache_keep(ctypes.byref(c), table, ts, 4, lens, B, path, N, new, None, None)
    for bad in (dict(new=far[0]), dict(new=far[2]), dict(new=far[2] + B * row - 4), dict(new=far[2] - 12), dict(new=far[1]),
                dict(new=far[1] + 60), dict(new=far[1] + 12, ts=0), dict(new=far[1] + 72, ts=5)):
        assert keep(**bad) == 1, bad
