"""Runs a MoE block (bit_quantized_routed_amd.block) on synthetic weights and
compares it with plain torch.

    python examples/moe_block.py [--tokens T] [--hidden H] [--inter I] [--experts E]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_routed_amd as M  # noqa: E402
import synthetic as S  # noqa: E402
from bit_quantized_routed_amd.block import BlockBuffers, MoeBlock  # noqa: E402
from workload import Workload  # noqa: E402


def make(hidden, inter, experts, top_k=4, groups=4, keep=2, seed=0, device="cuda"):
    """(block, its weights in float) on synthetic values."""
    cfg = dict(hidden=hidden, inter=inter, n_experts=experts, top_k=top_k, sh_inter=0, T=1, x_dtype="bf16", skew=False,
               fmt_gate_up=S.FMT_CB2, fmt_down=S.FMT_Q2K, index=40, name="block", seed=seed)
    layer = Workload(cfg, device=device).layer
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).to(device)  # noqa: E731
    norm = M.NormWeights(1.0 + rnd(hidden, std=0.1))
    router = M.RouterWeights(rnd(experts, hidden, std=hidden ** -0.5), top_k, "sigmoid", rnd(experts, std=0.05), groups, keep,
                             True, 2.5)
    gate_up, down = rnd(2 * inter, hidden, std=0.02), rnd(hidden, inter, std=0.02)
    block = MoeBlock(norm, router, layer, M.LinearI8.quantize(gate_up), M.LinearI8.quantize(down))
    return block, gate_up, down


def plain_shared(n, gate_up, down):
    """The shared expert on float weights."""
    a, b = (n.double() @ gate_up.double().t()).chunk(2, 1)
    return (a * torch.sigmoid(a) * b) @ down.double().t()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--tokens", type=int, default=32)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inter", type=int, default=512)
    ap.add_argument("--experts", type=int, default=16)
    a = ap.parse_args(argv)
    block, gate_up, down = make(a.hidden, a.inter, a.experts)
    b = BlockBuffers(block, a.tokens)
    g = torch.Generator().manual_seed(1)
    x = torch.randn((a.tokens, a.hidden), generator=g).cuda()
    residual = torch.randn((a.tokens, a.hidden), generator=g).bfloat16().cuda()
    # the routed experts alone, then the block: their difference is the shared expert's output
    block(x, residual.clone(), b)
    routed = torch.empty_like(b.y)
    (M.ffn_decode if b.path == M.PATH_DECODE else M.ffn_prefill)(block.layer, b.n, M.ACT_BF16, a.tokens, b.routing, routed, b.ws_ffn)
    want = plain_shared(b.n, gate_up, down)
    off = float((b.y.double() - routed.double() - want).norm() / want.norm())
    print("tokens %d: experts %s of the first, shared expert in 8 bits within %.1f%% of its float weights"
          % (a.tokens, np.sort(b.routing.topk_idx[0].cpu().numpy()).tolist(), 100 * off), flush=True)
    return off


if __name__ == "__main__":
    main()
