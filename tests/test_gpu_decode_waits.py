"""Waits of the decode-side kernels that run out, without a fault, in the -DSPEC_DEBUG variant of the library.

Sampling: a row whose uniform is a certain NaN is taken for one whose copy never landed on one block of its cluster.  The
row gets no result, the status word says so, and the other rows are right.  Attention on tcgen05: a bit of the status word
that the call passes makes the first block's first wait run out.  The call ends, says so, and the next one is right."""
import ctypes
import math
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
WAIT_TIMEOUT, UNIFORM_RANGE = 8, 4


@pytest.fixture(scope="module")
def libs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    from draft_verify_acceptance_gb300 import build, decode
    dbg = ctypes.CDLL(build.build(debug=True))
    for name in ("spec_filtered_sample", "spec_filtered_sample_workspace_size", "spec_paged_attention"):
        for attr in ("restype", "argtypes"):
            setattr(getattr(dbg, name), attr, getattr(getattr(decode._lib, name), attr))
    return dbg, decode


def call(lib, x, u, T, k, p, m, ws=None):
    R, V = x.shape
    dt = 1 if x.dtype == torch.bfloat16 else 0
    tokens, n_kept, status = (torch.full((n,), -5, dtype=torch.int32, device="cuda") for n in (R, R, 1))
    status.zero_()
    prob, out = torch.full((R,), -5.0, device="cuda"), torch.full_like(x, 5.0)
    need = lib.spec_filtered_sample_workspace_size(R, V, dt)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda") if ws is None else ws
    rc = lib.spec_filtered_sample(x.data_ptr(), V, u.data_ptr(), R, V, dt, T, k, p, m, None, None, None, None,
                                  tokens.data_ptr(), prob.data_ptr(), n_kept.data_ptr(), out.data_ptr(),
                                  ws.data_ptr() if need else None, need, None, status.data_ptr())
    assert rc == 0
    torch.cuda.synchronize()
    return tokens, prob, n_kept, out, int(status), ws


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.8, 0, 0.9, 0.0), (1.0, 40, 0.95, 0.0), (1.0, 0, 1.0, 0.05)]


@pytest.mark.parametrize("R,V", [(4, 128256), (200, 128256), (400, 1000)])  # the whole-row kernel; the list kernel
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_row_whose_copy_is_lost_on_one_block(libs, R, V, dtype):
    lib, decode = libs
    g = torch.Generator(device="cuda").manual_seed(R)
    x = (torch.randn((R, V), generator=g, device="cuda") * 3).to(dtype)
    u = torch.rand(R, generator=g, device="cuda")
    for s in SETTINGS:
        want = call(lib, x, u, *s)
        plain = decode.filtered_sample(x, u, s[0], top_k=s[1], top_p=s[2], min_p=s[3], return_filtered=True)
        assert want[4] == 0 and all(torch.equal(a, b) for a, b in zip(want, plain[:4]))
        lost = {R - 3: 0} if V < 2000 else {1: 2, R - 1: 0}
        u2 = u.clone()
        for row, rank in lost.items():
            u2.view(torch.int32)[row] = 0x7fc0d000 + rank
        got = call(lib, x, u2, *s)
        assert got[4] == WAIT_TIMEOUT | UNIFORM_RANGE
        rest = [r for r in range(R) if r not in lost]
        assert all(torch.equal(a[rest], b[rest]) for a, b in zip(got[:4], want[:4]))
        for row in lost:
            assert (int(got[0][row]), float(got[1][row]), int(got[2][row])) == (0, 0.0, 0)
            assert (got[3][row] == -math.inf).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_queued_row_whose_copy_is_lost(libs, dtype):
    """Flat rows among others go to the whole-row kernel by a queue: one lost there is reported too."""
    lib, decode = libs
    R, V = 400, 40000
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((R, V), generator=g, device="cuda") * 3
    x[7::15] *= 0.1
    x = x.to(dtype)
    u = torch.rand(R, generator=g, device="cuda")
    want = call(lib, x, u, 1.0, 0, 0.9, 0.0)
    plain = decode.filtered_sample(x, u, 1.0, top_p=0.9, return_filtered=True)
    assert want[4] == 0 and all(torch.equal(a, b) for a, b in zip(want, plain[:4]))
    row = 7 + 15 * 9
    u.view(torch.int32)[row] = 0x7fc0e000 + 1
    got = call(lib, x, u, 1.0, 0, 0.9, 0.0)
    assert got[4] == WAIT_TIMEOUT | UNIFORM_RANGE
    rest = [r for r in range(R) if r != row]
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip(got[:4], want[:4]))
    assert (int(got[0][row]), float(got[1][row]), int(got[2][row])) == (0, 0.0, 0)
    assert (got[3][row] == -math.inf).all()
    # the queue is as it was: the next call on this workspace is right
    u.view(torch.int32)[row] = 0
    assert call(lib, x, u, 1.0, 0, 0.9, 0.0, got[5])[4] == 0


def test_rows_after_a_lost_one(libs):
    """Clusters that take several queued rows each: a block that gave up waits for its copies before the next row's, so
    the rows after a lost one are right."""
    lib, decode = libs
    R, V = 600, 40000
    g = torch.Generator(device="cuda").manual_seed(6)
    x = (torch.randn((R, V), generator=g, device="cuda") * 0.3).to(torch.bfloat16)
    u = torch.rand(R, generator=g, device="cuda")
    want = call(lib, x, u, 1.0, 0, 0.9, 0.0)
    assert want[4] == 0
    lost = list(range(3, R, 97))
    for i, row in enumerate(lost):
        u.view(torch.int32)[row] = 0x7fc0e000 + i % 4
    got = call(lib, x, u, 1.0, 0, 0.9, 0.0)
    assert got[4] == WAIT_TIMEOUT | UNIFORM_RANGE
    rest = [r for r in range(R) if r not in lost]
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip(got[:4], want[:4]))
    assert (got[2][lost] == 0).all() and (got[3][lost] == -math.inf).all()


def test_attention_on_tcgen05_ends_after_a_wait_that_ran_out(libs):
    lib, decode = libs
    B, Q, Hq, H, D, S, n = 3, 9, 32, 4, 128, 16, 3000
    g = torch.Generator(device="cuda").manual_seed(7)
    pages = -(-n // S)
    k, v = (torch.randn((B * pages, S, H, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    table = torch.randperm(B * pages, generator=g, device="cuda").to(torch.int32).view(B, pages)
    table = torch.cat([table, torch.full((B, 2000), -1, dtype=torch.int32, device="cuda")], 1)
    lengths = torch.tensor([n, 1, n - 7], dtype=torch.int32, device="cuda")
    q = torch.randn((B, Q, Hq, D), generator=g, device="cuda").to(torch.bfloat16)
    want = decode.paged_attention(q, k, v, table, lengths)
    c = decode._Cache(k.data_ptr(), v.data_ptr(), 0, S * H * D, H * D, 1, B * pages, S, H, D, 1)
    need = decode.attention_workspace_size(B, Q, Hq, H, D, q.dtype)

    def run(bit):
        out, ws = torch.empty_like(q), torch.zeros(need, dtype=torch.uint8, device="cuda")
        status = torch.tensor([bit], dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        rc = lib.spec_paged_attention(q.data_ptr(), Q * Hq * D, Hq * D, D, ctypes.byref(c), table.data_ptr(), table.shape[1],
                                      table.shape[1], lengths.data_ptr(), B, Q, Hq, D ** -0.5, out.data_ptr(), None,
                                      ws.data_ptr(), need, None, status.data_ptr())
        torch.cuda.synchronize()
        assert rc == 0 and time.perf_counter() - t0 < 5.0
        return out, int(status)
    for _ in range(3):
        assert run(1 << 30)[1] == 1 << 30 | WAIT_TIMEOUT
        out, status = run(0)
        assert status == 0 and torch.equal(out, want)
