"""Edges of the operators for a few tokens on the GPU: workspaces anywhere, every form of the adapters' kernels."""
import pytest
import torch

import bit_quantized_routed_amd as M
from gpu_common import need_gpu
from test_gpu_dense import rnd
from test_gpu_few import BF16, F32, H24, Block, adapters_reference, check_adapters, make_adapters, say

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


@pytest.mark.parametrize("left", [(), (5,), (1, 6), (0, 2, 7)])
@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("softmax", False)])
def test_block_few_experts_left_against_64_bits(left, score, renorm):
    """Biases of -inf that leave fewer experts than k: y is what those and the shared expert give, the shared one alone where none is."""
    need_gpu()
    say("block experts left", left, score, renorm)
    b = Block(256, 128, 8, 4, 64, score=score, renorm=renorm, seed=3)
    keep = b.bias[list(left)].clone()
    b.bias[:] = -float("inf")
    b.bias[list(left)] = keep
    for T in (1, 3, 9):
        x, res = rnd(3, T, 256).cuda(), rnd(4, T, 256).cuda()
        _, _, idx, wt, want, bound = b.reference(x, res)
        y, r = b.run(x, res)
        torch.cuda.synchronize()
        assert torch.equal(r.topk_idx, idx) and torch.all((r.topk_w.double() - wt).abs() <= 3 * H24 * wt)
        assert torch.all(wt[:, len(left):] == 0) and torch.all(wt[:, :len(left)] > 0)
        assert torch.all((y.double() - want).abs() <= bound) and want.norm() > 0


def test_example_of_a_block_that_the_few_do_not_take():
    """The example on a layer past moe_block_decode's limits, with few tokens: the operators one after another still run."""
    import os
    import sys
    need_gpu()
    say("example, inter 8200")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_block as B
    assert B.main(["--tokens", "3", "--hidden", "64", "--inter", "8200", "--experts", "8"]) < 0.05


# ------------------------------------------------------------------ adapters
# tiles of 64 tokens whose rows are aligned: every type at every count of column fragments (16 columns each, 1 or 2, up to 4, 8, 16), with
# K that ends inside a step of 64 (32 of fp32) and, for fp32, inside a piece of 8 that A's zeros fill
WIDE = [(T, K, parts * 16, rank, parts, 3, kind, yt)
        for i, (rank, parts) in enumerate(((16, 1), (32, 1), (24, 2), (64, 1), (50, 2), (64, 2), (43, 3), (64, 4)))
        for T, K, kind, yt in ((513 + 37 * i, 2032, "i8", F32 if i % 2 else BF16), (600 + i, 16 + 64 * i, "i8", F32),
                               (577 + 64 * i, 520, BF16, F32 if i % 2 else BF16), (640 - i, 8 + 192 * i, BF16, F32),
                               (700 + i, 1004, F32, BF16 if i % 2 else F32), (515 + i, 4 + 32 * i, F32, F32))]


@pytest.mark.parametrize("T,K,N,r,parts,n,kind,yt", WIDE)
def test_adapters_wide(T, K, N, r, parts, n, kind, yt):
    need_gpu()
    say("adapters wide", T, K, N, r, parts, n, kind, yt)
    check_adapters(T + K, T, K, N, r, parts, n, kind, yt)
    check_adapters(T + K + 1, T, K, N, r, parts, n, kind, yt, pad=16, off=16, inplace=True)


@pytest.mark.parametrize("T", [16, 513])
@pytest.mark.parametrize("r,parts", [(8, 1), (40, 2), (64, 4)])
def test_adapters_codes_at_eight_bytes(T, r, parts):
    """Rows of codes that begin on 8 but not on 16 bytes."""
    need_gpu()
    say("adapters codes at 8 bytes", T, r, parts)
    check_adapters(T + r, T, 1160, 64 * parts, r, parts, 4, "i8", F32, pad=8, off=8)
    check_adapters(T + r, T, 1160, 64 * parts, r, parts, 4, "i8", BF16, pad=0, off=24, inplace=True)


# ------------------------------------------------------------------ together
def test_block_step_with_adapters_of_a_chunk():
    """A chunk of prompts through the block with its requests' adapters: tiles of 64 tokens beside both projections of the shared
    expert, bf16 rows and codes to fp32."""
    import os
    import sys
    need_gpu()
    say("chunk with adapters")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_block as B
    from bit_quantized_routed_amd.block import StepAdapters
    H, I, T, n = 512, 256, 600, 5
    block, _, _ = B.make(H, I, 16)
    up, down = make_adapters(11, n, H, 2 * I, 24, 2), make_adapters(21, n, I, H, 16, 1)
    ids = (torch.arange(T) // 37 % (n + 1) - 1).int()
    plan = M.AdapterPlan(T, n)
    M.adapter_plan(ids.cuda(), plan)
    step = StepAdapters(plan, M.AdapterWeights(*(t.cuda() for t in up), 2), M.AdapterWeights(*(t.cuda() for t in down)))
    x, res = rnd(71, T, H).cuda(), rnd(72, T, H, dtype=BF16).cuda()
    b, plain = B.BlockBuffers(block, T), B.BlockBuffers(block, T)
    y = block(x, res.clone(), b, adapters=step)
    z = block(x, res.clone(), plain)
    routed = torch.empty_like(y)
    M.ffn_prefill(block.layer, b.n, M.ACT_BF16, T, b.routing, routed, b.ws_ffn)
    torch.cuda.synchronize()
    assert b.path == M.PATH_PREFILL
    none = ids < 0
    assert torch.equal(y.cpu()[none], z.cpu()[none]) and not torch.equal(y.cpu()[~none], z.cpu()[~none])
    d = lambda t: t.double().cpu()                                     # noqa: E731
    want, bound = adapters_reference(*up, 2, ids, d(b.n), d(plain.gate_up), F32)
    assert torch.all((d(b.gate_up) - want).abs() <= bound)
    # the down rows on the codes of what they became: the int8 layer's three products and its sum with the routed part round
    wd, sd, _ = block.down.tensors
    h = d(b.h) * d(b.h_scale)[:, None]
    shared = h @ (d(wd) * d(sd)[:, None]).t()
    want, bound = adapters_reference(*down, 1, ids, h, d(routed) + shared, F32)
    assert torch.all((d(y) - want).abs() <= bound + 8 * H24 * (shared.abs() + d(routed).abs()))


@pytest.mark.parametrize("T,kind", [(40, BF16), (513, BF16), (600, "i8"), (577, F32), (530, "odd")])
def test_adapters_plan_of_anything(T, kind):
    """Plans that hold anything (read while another stream fills them, say): what lies around y, add and the workspace stays as
    it was, and so does what the call reads; the next call with a plan of its own is right."""
    need_gpu()
    K, N, r, parts, n = (1001 if kind == "odd" else 1008), 192, 16, 2, 5
    a, b, scale = make_adapters(7, n, K, N, r, parts)
    w = M.AdapterWeights(a.cuda(), b.cuda(), scale.cuda(), parts)
    g = torch.Generator().manual_seed(T)
    x = torch.randint(-127, 128, (T, K), generator=g).to(torch.int8) if kind == "i8" else rnd(3, T, K, dtype=F32 if kind == "odd" else kind)
    xs = torch.full((T,), 0.01) if kind == "i8" else None
    xd, xsd = x.cuda(), None if xs is None else xs.cuda()
    room = torch.full((T + 256, N), 77.0, device="cuda")
    y, size = room[128:128 + T], w.workspace(T).nbytes
    mem = torch.full((size + 65536,), 77, dtype=torch.uint8, device="cuda")
    ws = mem[32768:32768 + size]

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g).int().cuda()

    for i in range(8):
        plan, far = M.AdapterPlan(T, n), 2 ** 31 - 1 if i % 2 else T + 70
        plan.order, plan.offsets = ints(-far, far, T), ints(-far, far, n + 1)
        plan.tiles = torch.stack([ints(-3, n + 3, len(plan.tiles)), ints(-far, far, len(plan.tiles))], 1).contiguous()
        if i == 7:
            plan.tiles[:, 0] = ints(-2 ** 31, 2 ** 31 - 1, len(plan.tiles))
        say("adapters, a plan of anything", T, kind, i)
        M.adapters(w, plan, xd, xsd, y, None, ws)
        torch.cuda.synchronize()
        assert torch.all(room[:128] == 77) and torch.all(room[128 + T:] == 77)
        assert torch.all(mem[:32768] == 77) and torch.all(mem[32768 + size:] == 77)
    add = rnd(5, T, N)
    y.copy_(add)
    ids = torch.randint(-1, n, (T,), generator=g).int()
    M.adapter_plan(ids.cuda(), plan)
    M.adapters(w, plan, xd, xsd, y, None, ws)
    torch.cuda.synchronize()
    value = x.double() if xs is None else x.double() * xs.double()[:, None]
    want, bound = adapters_reference(a, b, scale, parts, ids, value, add, F32)
    assert torch.all((y.double().cpu() - want).abs() <= bound)
