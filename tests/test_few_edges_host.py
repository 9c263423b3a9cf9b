"""Edges of the operators for a few tokens that need no GPU: what is checked, kept or sized before any launch."""
import ctypes

import torch

import bit_quantized_routed_amd as M
from test_few_host import FAKE, Parts, _block

BF16 = torch.bfloat16


def test_block_workspace_at_any_offset():
    """The block lays its workspace out from a multiple of 256 on, wherever the caller's begins (a reader's cached line may hold
    nothing that another work-group writes later): the size that the library names has room for that, and a smaller one is
    refused where the gap takes what the call needs."""
    for T in (1, 4, 16):
        B = Parts()
        have = M.lib().moe_block_decode_workspace_bytes(ctypes.byref(B.c), T)
        need = have - 240                        # at a multiple of 256
        assert need % 256 == 0
        for at in range(0, 256, 16):
            gap = -at % 256
            # never launched
            assert _block(B, T=T, ws=FAKE + at, ws_bytes=need + gap - 1) == -3, (T, at)


def test_adapter_rows_of_one():
    """Matrices of one row count as contiguous whatever that row's stride: the library gets the rows' real distance."""
    n, K, r = 5, 64, 8
    scale = torch.ones(n)
    a, b = torch.zeros(1, n, K, dtype=BF16).permute(1, 0, 2), torch.zeros(n, r, 1, dtype=BF16).transpose(1, 2)
    assert a.is_contiguous() and a.stride(1) == n * K and b.is_contiguous() and b.stride(1) == 1
    w = M.AdapterWeights(a, torch.zeros(n, 32, 1, dtype=BF16), scale)  # rank 1: A is a row an adapter
    assert (w.c.lda, w.c.ldb) == (K, 8)
    w = M.AdapterWeights(torch.zeros(n, r, K, dtype=BF16), b, scale)   # one output
    assert (w.c.lda, w.c.ldb) == (K, r)
    w = M.AdapterWeights(torch.zeros(n, 5, 63, dtype=BF16), torch.zeros(n, 1, r, dtype=BF16)[:, :, :5], scale)       # copied
    assert (w.c.lda, w.c.ldb) == (64, 8)


def test_plan_before_it_is_filled():
    """A plan that no call has filled yet holds no tiles: the kernels take nothing from it."""
    for T, n in ((1, 1), (512, 1024), (513, 3), (8192, 100)):
        plan = M.AdapterPlan(T, n, device="cpu")
        assert plan.tiles.shape == (M.lib().moe_adapter_tiles(T, n), 2) and torch.all(plan.tiles[:, 0] == -2)
