"""Edges of the operators for a few tokens that need no GPU: what is checked, kept or sized before any launch."""
import ctypes

import pytest
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


class Launched(Exception):
    pass


def _stub_block(monkeypatch, H, I, T):
    """A block whose first launch is recorded and ends the call, and buffers for T tokens."""
    from types import SimpleNamespace
    from bit_quantized_routed_amd.block import MoeBlock
    block, calls = object.__new__(MoeBlock), []
    block.norm, block.hidden, block.sh_inter = None, H, I

    def norm(*a):
        calls.append("norm")
        raise Launched

    monkeypatch.setattr(M, "residual_norm", norm)
    return block, SimpleNamespace(T=T, n=None, q=None, q_scale=None), calls


@pytest.mark.parametrize("case", ["tokens", "adapters", "gate_up in", "gate_up out", "down in", "down out"])
def test_step_adapters_that_do_not_fit(case, monkeypatch):
    """Adapters of another step or block are refused before anything runs: the residual is updated in place."""
    from bit_quantized_routed_amd.block import StepAdapters
    H, I, T, n = 64, 32, 6, 3
    block, b, calls = _stub_block(monkeypatch, H, I, T)

    def weights(K, N, parts):
        return M.AdapterWeights(torch.zeros(n, 8 * parts, K, dtype=BF16), torch.zeros(n, N, 8, dtype=BF16), torch.ones(n), parts)

    def step(plan=None, gate_up=(H, 2 * I, 2), down=(I, H, 1)):
        plan = M.AdapterPlan(T, n, device="cpu") if plan is None else plan
        return StepAdapters(plan, None if gate_up is None else weights(*gate_up), None if down is None else weights(*down), device="cpu")

    for good in (None, step(), step(gate_up=None), step(down=None), step(gate_up=(H, 2 * I, 1))):
        with pytest.raises(Launched):
            block(None, None, b, None, good)
    assert len(calls) == 5
    bad = {"tokens": lambda: step(M.AdapterPlan(T + 1, n, device="cpu")), "adapters": lambda: step(M.AdapterPlan(T, n + 1, device="cpu")),
           "gate_up in": lambda: step(gate_up=(H + 8, 2 * I, 2)), "gate_up out": lambda: step(gate_up=(H, 2 * I + 2, 2)),
           "down in": lambda: step(down=(I + 8, H, 1)), "down out": lambda: step(down=(I, H + 1, 1))}[case]
    with pytest.raises(ValueError):
        block(None, None, b, None, bad())
    assert len(calls) == 5
