"""Edges of the operators for a few tokens on the GPU: workspaces anywhere, every form of the adapters' kernels."""
import pytest
import torch

import bit_quantized_routed_amd as M
from gpu_common import need_gpu
from test_gpu_dense import rnd
from test_gpu_few import BF16, Block, say

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ block
@pytest.mark.parametrize("T,H,I,sh", [(4, 7168, 256, 64), (16, 1024, 512, 128), (16, 2048, 264, 0)])
@pytest.mark.parametrize("at", [16, 80, 96, 112, 240])
def test_block_workspace_anywhere(T, H, I, sh, at):
    """A workspace that begins on any 16 bytes, with what another call left in it: the same bits as in one of its own."""
    need_gpu()
    say("block workspace", T, H, I, sh, at)
    b = Block(H, I, 16, 4, sh, seed=T)
    mem = torch.zeros(b.w.workspace(T).nbytes + 256, dtype=torch.uint8, device="cuda")
    ws = mem[at:at + b.w.workspace(T).nbytes]
    assert mem.data_ptr() % 256 == 0
    mem[at + ws.nbytes:] = 77
    for i in range(4):
        x, res = rnd(10 + i, T, H, std=0.5).cuda(), rnd(20 + i, T, H, std=2.0, dtype=BF16).cuda()
        y, r = b.run(x, res, ws=ws)
        want, q = b.run(x, res)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(r.topk_idx, q.topk_idx) and torch.equal(r.topk_w, q.topk_w)
        assert torch.all(mem[at + ws.nbytes:] == 77) and torch.all(mem[:at] == 0)


def test_example_of_a_block_that_the_few_do_not_take():
    """The example on a layer past moe_block_decode's limits, with few tokens: the operators one after another still run."""
    import os
    import sys
    need_gpu()
    say("example, inter 8200")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_block as B
    assert B.main(["--tokens", "3", "--hidden", "64", "--inter", "8200", "--experts", "8"]) < 0.05
