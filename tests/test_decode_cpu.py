"""CPU-only checks of the decode-side entry points: exports, constants, refusals on the host before any launch, and the
binding's own checks.  No kernel is launched here."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "spec_decode.h")
FAKE = 1 << 20  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def decode():
    import __graft_entry__
    __graft_entry__.build()
    from draft_verify_acceptance_gb300 import decode
    return decode


def test_exports_and_constants(decode):
    src = open(HEADER).read()
    names = set(re.findall(r"SPEC_API\s+[\w\s\*]+?\b(spec_\w+)\s*\(", src))
    assert names == set(decode.EXPORTS)
    for n in names:
        assert hasattr(decode._lib, n)
    defs = {k: int(v) for k, v in re.findall(r"#define\s+SPEC_(DATA_\w+)\s+(\d+)", src)}
    assert len(defs) == 4
    for k, v in defs.items():
        assert getattr(decode, k) == v
    other = open(os.path.join(os.path.dirname(HEADER), "spec_verify.h")).read()
    taken = [int(v) for v in re.findall(r"#define\s+SPEC_(?:DATA_\w+|DEVICE_WAIT_TIMEOUT|DEBUG_BOUNDS)\s+(\d+)", other)]
    assert not set(taken) & set(defs.values())


def test_workspaces_zero_bytes(decode):
    src = open(HEADER).read()
    zero = {k: int(v) for k, v in re.findall(r"#define\s+SPEC_(\w+)_ZERO_BYTES\s+(\d+)", src)}
    assert zero == {"ATTENTION": decode._KINDS["attention"][1], "SAMPLE": decode._KINDS["sample"][1]}
    assert decode._KINDS["fork"][1] == decode._KINDS["compact"][1] == 0


def test_native_calls_are_rebuilt_for_another_torch(decode, monkeypatch):
    """_decode_calls.so has torch's and the interpreter's layouts in it: one made for others is not kept."""
    from draft_verify_acceptance_gb300 import build
    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        return subprocess.CompletedProcess(cmd, 1, "", "not now")
    monkeypatch.setattr(build.subprocess, "run", run)
    assert build.build_calls() == build.CALLS and not runs
    for name, value in (("CALLS_FOR", build.CALLS_FOR + ".none"), ("_calls_abi", lambda: "torch 1.0, cpython-39")):
        with monkeypatch.context() as m:
            m.setattr(build, name, value, raising=False)
            with pytest.raises(RuntimeError):
                build.build_calls()
    assert len(runs) == 2 and os.path.exists(build.CALLS)


def test_header_is_plain_c(tmp_path):
    f = tmp_path / "h.c"
    f.write_text('#include "spec_decode.h"\nint main(void) { spec_cache_t c; (void)c; return 0; }\n')
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-I", os.path.dirname(HEADER),
                        str(f)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def cache(decode, **kw):
    d = dict(k=FAKE, v=FAKE, layer_stride=0, page_stride=16 * 2 * 64, token_stride=128, layers=1, pages=8, page_size=16,
             heads=2, head_dim=64, dtype=0)
    d.update(kw)
    return decode._Cache(*(d[n] for n, _ in decode._Cache._fields_))


BAD_CACHES = [(dict(k=0), 1), (dict(v=FAKE + 4), 1), (dict(layers=0), 1), (dict(pages=-1), 1), (dict(page_size=0), 1),
              (dict(heads=0), 1), (dict(dtype=2), 1), (dict(token_stride=127), 1), (dict(token_stride=130), 1),
              (dict(page_stride=100), 1), (dict(layers=2, layer_stride=64), 1), (dict(page_size=1 << 17), 2)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_cache_refusals(decode, kw, code):
    c = cache(decode, **kw)
    lib = decode._lib
    assert lib.spec_cache_append(FAKE, FAKE, 128, 4, None, ctypes.byref(c), FAKE, 4, 4, FAKE, 2, None, None) == code
    assert lib.spec_cache_compact(ctypes.byref(c), FAKE, 4, 4, 2, FAKE, FAKE, FAKE, FAKE, 1 << 20, None, None) == code
    assert lib.spec_cache_fork(ctypes.byref(c), FAKE, 4, 4, FAKE, 2, FAKE, FAKE, 2, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                               1 << 20, None, None) == code


def test_attention_refusals(decode):
    lib = decode._lib
    need = lib.spec_attention_workspace_size(2, 1, 4, 2, 64, 0)
    assert need > 0 and need % 256 == 0

    def call(q=FAKE, qs=(256, 256, 64), c=None, table=FAKE, ts=4, M=4, lens=FAKE, B=2, Q=1, Hq=4, scale=0.1, out=FAKE,
             lse=None, ws=FAKE, n=None, st=None):
        c = c if c is not None else cache(decode)
        return lib.spec_paged_attention(q, *qs, ctypes.byref(c), table, ts, M, lens, B, Q, Hq, scale, out, lse, ws,
                                        need if n is None else n, None, st)
    for bad in (dict(q=0), dict(q=FAKE + 8), dict(qs=(2, 256, 64)), dict(qs=(-256, 256, 64)), dict(table=0), dict(ts=3),
                dict(M=-1), dict(lens=0), dict(lens=FAKE + 2), dict(B=-1), dict(Q=-1), dict(Hq=3), dict(Hq=0), dict(out=0),
                dict(lse=FAKE + 1), dict(ws=0), dict(n=need - 1), dict(ws=FAKE + 8), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(st=FAKE + 2), dict(c=cache(decode, layers=2, layer_stride=1 << 14))):
        assert call(**bad) == decode.ERR_INVALID_ARG, bad
    assert call(c=cache(decode, head_dim=96, token_stride=192, page_stride=4096)) == decode.ERR_UNSUPPORTED
    assert call(Q=(1 << 20) + 1) == decode.ERR_UNSUPPORTED
    assert call(M=1 << 28, ts=1 << 28) == decode.ERR_UNSUPPORTED
    assert call(B=0, q=0, lens=0, out=0, ws=0) == decode.OK
    assert call(Q=0, q=0, lens=0, out=0, ws=0) == decode.OK
    for bad in ((-1, 1, 4, 2, 64, 0), (2, 1, 3, 2, 64, 0), (2, 1, 4, 2, 96, 0), (2, 1, 4, 0, 64, 0), (2, 1, 4, 2, 64, 5)):
        assert lib.spec_attention_workspace_size(*bad) == 0


def test_page_tables_of_one_row_and_of_overlapping_rows(decode):
    """One row expanded to every sequence keeps its stride of 0 (read at a stride of its length, the rows after the first
    would be other memory); rows that overlap otherwise are refused."""
    one = torch.arange(4, dtype=torch.int32)[None]
    t = one.expand(3, 4)
    assert decode._table(t, 3, -1) == (one.data_ptr(), 0, 4)
    assert decode._table(one, 1, -1) == (one.data_ptr(), 4, 4)
    assert decode._table(torch.zeros((3, 9), dtype=torch.int32)[:, :4], 3, -1)[1:] == (9, 4)
    with pytest.raises(ValueError):
        decode._table(torch.arange(9, dtype=torch.int32).as_strided((3, 4), (2, 1)), 3, -1)
    lib, c = decode._lib, cache(decode)
    for stride, code in ((0, decode.OK), (4, decode.OK), (3, decode.ERR_INVALID_ARG), (1, decode.ERR_INVALID_ARG),
                         (-4, decode.ERR_INVALID_ARG)):
        assert lib.spec_cache_append(FAKE, FAKE, 128, 0, None, ctypes.byref(c), FAKE, stride, 4, FAKE, 2, None, None) == code


def test_library_calls_keep_the_interpreter_s_lock(decode):
    """A call's launches share a workspace with other threads' calls on the stream, so none may come between them."""
    python_api = 4  # FUNCFLAG_PYTHONAPI: the lock is not released around the call
    for n in decode.EXPORTS:
        assert getattr(decode._lib, n)._flags_ & python_api, n


def test_append_refusals(decode):
    lib, c = decode._lib, cache(decode)

    def call(k=FAKE, v=FAKE, stride=128, T=4, starts=None, lens=FAKE, B=2, c=c):
        return lib.spec_cache_append(k, v, stride, T, starts, ctypes.byref(c), FAKE, 4, 4, lens, B, None, None)
    for bad in (dict(k=0), dict(v=FAKE + 4), dict(stride=127), dict(stride=129), dict(T=-1), dict(T=5), dict(B=0), dict(B=-1),
                dict(lens=0), dict(starts=FAKE + 1), dict(c=cache(decode, layers=2, layer_stride=1 << 14))):
        assert call(**bad) == decode.ERR_INVALID_ARG, bad
    assert call(T=0, k=0, v=0) == decode.OK
    assert call(c=cache(decode, heads=1, head_dim=3, token_stride=4, page_stride=64)) == decode.ERR_UNSUPPORTED


def test_fork_and_compact_refusals(decode):
    lib, c = decode._lib, cache(decode)
    need = lib.spec_cache_fork_workspace_size(8, 2)

    def fork(table=FAKE, ts=4, M=4, lens=FAKE, B=2, par=FAKE, keep=FAKE, C=2, room=0, new=FAKE, nl=FAKE, refs=FAKE,
             free=FAKE, nf=FAKE, ws=FAKE, n=need):
        return lib.spec_cache_fork(ctypes.byref(c), table, ts, M, lens, B, par, keep, C, room, new, nl, refs, free, nf, ws, n,
                                   None, None)
    for bad in (dict(table=0), dict(ts=3), dict(lens=0), dict(B=-1), dict(par=0), dict(keep=FAKE + 1), dict(C=-1),
                dict(room=-1), dict(new=0), dict(nl=0), dict(refs=0), dict(free=0), dict(nf=0), dict(ws=0), dict(n=need - 1)):
        assert fork(**bad) == decode.ERR_INVALID_ARG, bad
    assert fork(room=(1 << 30) + 1) == decode.ERR_UNSUPPORTED
    assert lib.spec_cache_fork_workspace_size(-1, 2) == 0 and lib.spec_cache_fork_workspace_size(2, -1) == 0
    need = lib.spec_cache_compact_workspace_size(8)

    def compact(B=2, new=FAKE, refs=FAKE, nl=FAKE, ws=FAKE, n=need):
        return lib.spec_cache_compact(ctypes.byref(c), FAKE, 4, 4, B, new, refs, nl, ws, n, None, None)
    for bad in (dict(B=-1), dict(new=0), dict(refs=0), dict(nl=0), dict(ws=0), dict(n=need - 1)):
        assert compact(**bad) == decode.ERR_INVALID_ARG, bad
    assert lib.spec_cache_compact_workspace_size(-1) == 0


def test_sample_refusals(decode):
    lib = decode._lib
    need = lib.spec_filtered_sample_workspace_size(4, 1000, 0)

    def call(x=FAKE, stride=1000, u=FAKE, R=4, V=1000, dtype=0, T=1.0, k=0, p=1.0, m=0.0, Ts=None, ks=None, ps=None, ms=None,
             tok=FAKE, prob=None, cnt=None, out=None, st=None):
        return lib.spec_filtered_sample(x, stride, u, R, V, dtype, T, k, p, m, Ts, ks, ps, ms, tok, prob, cnt, out,
                                        FAKE, need, None, st)
    nan = float("nan")
    for bad in (dict(x=0), dict(x=FAKE + 2), dict(stride=999), dict(u=0), dict(R=-1), dict(V=0), dict(dtype=3), dict(T=-0.5),
                dict(T=nan), dict(T=float("inf")), dict(p=nan), dict(m=nan), dict(Ts=FAKE + 1), dict(ks=FAKE + 2),
                dict(ps=FAKE + 3), dict(ms=FAKE + 1), dict(tok=0), dict(prob=FAKE + 1), dict(cnt=FAKE + 1), dict(out=FAKE + 2),
                dict(st=FAKE + 2)):
        assert call(**bad) == decode.ERR_INVALID_ARG, bad
    assert call(V=decode.MAX_V + 1, stride=1 << 23) == decode.ERR_UNSUPPORTED
    assert call(R=0, x=0, u=0, tok=0) == decode.OK


def test_filtered_rows_apart_from_the_logits_or_in_their_place(decode):
    lib = decode._lib
    need = lib.spec_filtered_sample_workspace_size(4, 1000, 0)

    def call(out, x=FAKE, stride=1000, R=4, V=1000, dtype=0):
        return lib.spec_filtered_sample(x, stride, FAKE, R, V, dtype, 1.0, 0, 1.0, 0.0, None, None, None, None, FAKE, None, None,
                                        out, FAKE, need, None, None)
    size = 4 * 1000 * 4
    for bad in (dict(out=FAKE + 4), dict(out=FAKE - 4), dict(out=FAKE + size - 4), dict(out=FAKE - size + 4),
                dict(out=FAKE, stride=1008), dict(out=FAKE + 3 * 4032 + 3996, stride=1008),
                dict(out=FAKE + 2, dtype=1), dict(out=FAKE + 4, R=1)):
        assert call(**bad) == decode.ERR_INVALID_ARG, bad
    for good in (dict(out=FAKE), dict(out=FAKE + size), dict(out=FAKE - size), dict(out=FAKE, stride=1008, R=1),
                 dict(out=FAKE + 3 * 4032 + 4000, stride=1008)):
        if not torch.cuda.is_available():  # (with a GPU it would be launched)
            assert call(**good) == 3, good  # SPEC_ERR_CUDA: no argument error


def test_binding_refuses_cpu_tensors(decode):
    x, pages = torch.zeros(2, 8), torch.zeros(3, 4, 1, 64)
    with pytest.raises(ValueError):
        decode.filtered_sample(x, torch.zeros(2))
    with pytest.raises(ValueError):
        decode.cache_compact(pages, pages, torch.zeros((1, 1), dtype=torch.int32))
    with pytest.raises(ValueError):
        decode.paged_attention(torch.zeros(1, 1, 1, 64), pages, pages, torch.zeros((1, 1), dtype=torch.int32),
                               torch.zeros(1, dtype=torch.int32))


def test_the_weight_polynomial():
    """The sampler's 2^f is within 2^-21 of the function in its own arithmetic, exactly 1 at 0, and rises."""
    import numpy as np

    import decode_reference as ref
    f = np.linspace(-0.5, 0.5, 1 << 20, dtype=np.float32)
    g = np.float32(ref.POLY[4])
    for c in (*ref.POLY[3::-1], 1.0):
        g = g * f + np.float32(c)
    assert np.abs(g.astype(np.float64) / 2.0 ** f.astype(np.float64) - 1).max() < 2.0 ** -21
    assert (np.diff(g) >= 0).all()
    src = open(os.path.join(ROOT, "draft_verify_acceptance_gb300", "csrc", "filtered_sample.cu")).read()
    for c in ref.POLY:
        assert repr(c) + "f" in src
