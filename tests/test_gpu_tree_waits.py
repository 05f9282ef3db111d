"""Waits of the tree attention kernel on tcgen05 that run out, without a fault, in the -DSPEC_DEBUG variant of the library:
a bit of the status word that the call passes makes the first block's waits run out.  The call ends, says so, and the next
one on the same workspace is right."""
import ctypes
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
WAIT_TIMEOUT = 8


@pytest.mark.parametrize("N,G,D", [(9, 4, 128), (33, 8, 128), (20, 4, 64), (60, 4, 64)])  # one stream of rows, and two
def test_attention_ends_after_a_wait_that_ran_out(N, G, D):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    from draft_verify_acceptance_gb300 import build, tree
    lib = ctypes.CDLL(build.build(debug=True))
    lib.spec_tree_attention.restype, lib.spec_tree_attention.argtypes = (getattr(tree._lib.spec_tree_attention, a)
                                                                         for a in ("restype", "argtypes"))
    B, H, S, n = 3, 4, 16, 3000
    g = torch.Generator(device="cuda").manual_seed(7)
    pages = -(-n // S)
    k, v = (torch.randn((B * pages, S, H, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    table = torch.randperm(B * pages, generator=g, device="cuda").to(torch.int32).view(B, pages)
    lengths = torch.tensor([n, 1, n - 7], dtype=torch.int32, device="cuda")
    parents = torch.tensor([[-1] + [i // 2 for i in range(N - 1)]] * B, dtype=torch.int32, device="cuda")
    q = torch.randn((B, N, H * G, D), generator=g, device="cuda").to(torch.bfloat16)
    want = tree.tree_attention(q, k, v, table, lengths, parents)
    c = tree._Cache(k.data_ptr(), v.data_ptr(), 0, S * H * D, H * D, 1, B * pages, S, H, D, 1)
    need = tree.attention_workspace_size(B, N, H * G, H, D, q.dtype)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def run(bit):
        out = torch.empty_like(q)
        status = torch.tensor([bit], dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        rc = lib.spec_tree_attention(q.data_ptr(), N * H * G * D, H * G * D, D, ctypes.byref(c), table.data_ptr(), pages, pages,
                                     lengths.data_ptr(), parents.data_ptr(), N, B, N, H * G, D ** -0.5, out.data_ptr(), None,
                                     ws.data_ptr(), need, None, status.data_ptr())
        torch.cuda.synchronize()
        assert rc == 0 and time.perf_counter() - t0 < 5.0
        return out, int(status)
    for _ in range(3):
        assert run(1 << 30)[1] == 1 << 30 | WAIT_TIMEOUT
        out, status = run(0)
        assert status == 0 and torch.equal(out, want)


@pytest.mark.parametrize("B,N,Hq,H,D,most", [(400, 7, 32, 8, 64, 60), (600, 9, 32, 8, 128, 60), (500, 7, 32, 8, 64, 190),
                                              (800, 40, 16, 4, 64, 60), (500, 60, 32, 8, 128, 190)])
def test_warps_that_start_late_miss_nothing(B, N, Hq, H, D, most):
    """Twenty and more short items a block (more than are kept), most of one tile, and the warps that copy the second item's queries and the odd tiles a
    millisecond behind: what they have not read yet is still there."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    from draft_verify_acceptance_gb300 import build, tree
    lib = ctypes.CDLL(build.build(debug=True))
    lib.spec_tree_attention.restype, lib.spec_tree_attention.argtypes = (getattr(tree._lib.spec_tree_attention, a)
                                                                         for a in ("restype", "argtypes"))
    S = 16
    g = torch.Generator(device="cuda").manual_seed(N)
    lengths = torch.randint(0, most + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    pages = -(-most // S)
    k, v = (torch.randn((B * pages, S, H, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    table = torch.randperm(B * pages, generator=g, device="cuda").to(torch.int32).view(B, pages)
    parents = torch.tensor([[-1] + [i // 2 for i in range(N - 1)]] * B, dtype=torch.int32, device="cuda")
    q = torch.randn((B, N, Hq, D), generator=g, device="cuda").to(torch.bfloat16)
    want, lse = tree.tree_attention(q, k, v, table, lengths, parents, return_lse=True)
    c = tree._Cache(k.data_ptr(), v.data_ptr(), 0, S * H * D, H * D, 1, B * pages, S, H, D, 1)
    need = tree.attention_workspace_size(B, N, Hq, H, D, q.dtype)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for bit in (1 << 29, 0, 1 << 29):
        out, l2 = torch.full_like(q, 7.0), torch.full_like(lse, 7.0)
        status = torch.tensor([bit], dtype=torch.int32, device="cuda")
        rc = lib.spec_tree_attention(q.data_ptr(), N * Hq * D, Hq * D, D, ctypes.byref(c), table.data_ptr(), pages, pages,
                                     lengths.data_ptr(), parents.data_ptr(), N, B, N, Hq, D ** -0.5, out.data_ptr(), l2.data_ptr(),
                                     ws.data_ptr(), need, None, status.data_ptr())
        torch.cuda.synchronize()
        assert rc == 0 and int(status) == bit and torch.equal(out, want) and torch.equal(l2, lse)
