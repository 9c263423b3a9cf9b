"""One MoE block on the library's operators: residual + norm, scored router,
quantized routed experts, and the shared expert in 8 bits.

    s   = x + residual                        (kept as the new residual)
    n   = rms_norm(s)                         bf16 for the router and the experts, int8 for the shared expert
    y   = sum_j w_j FFN_{e_j}(n)              quantized routed experts, fp32
    y  += W_down silu(W_gate n) * (W_up n)    int8 rows and weights

x of the next block is y: it joins the residual in that block's norm.
"""
from __future__ import annotations

import bit_quantized_routed_amd as M

# tokens up to which the decode path of the routed experts is the faster one
DECODE_TOKENS = 64


class BlockBuffers:
    """What one block writes for T tokens; blocks that run one after another may share one."""

    def __init__(self, block: "MoeBlock", T: int, device="cuda"):
        import torch
        H, I = block.hidden, block.sh_inter
        f32 = dict(dtype=torch.float32, device=device)
        self.T = T
        self.n = torch.empty((T, H), dtype=torch.bfloat16, device=device)
        self.q, self.q_scale = M.empty_i8(T, H, device), torch.empty(T, **f32)
        self.routing = M.Routing(T, block.router.top_k, block.router.n_experts, device)
        self.y = torch.empty((T, H), **f32)
        self.gate_up = torch.empty((T, 2 * I), **f32)
        self.h, self.h_scale = M.empty_i8(T, I, device), torch.empty(T, **f32)
        self.path = M.PATH_DECODE if T <= DECODE_TOKENS else M.PATH_PREFILL
        self.ws_route = block.router.workspace(T, device)
        self.ws_ffn = block.layer.workspace(T, self.path, device)
        self.ws_up, self.ws_down = block.gate_up.workspace(T, device), block.down.workspace(T, device)


class MoeBlock:
    """norm: NormWeights; router: RouterWeights; layer: a DeviceLayer without a shared expert; gate_up: LinearI8 of
    rows [gate | up] (2 I x H); down: LinearI8 (H x I)."""

    def __init__(self, norm, router, layer, gate_up, down):
        self.norm, self.router, self.layer, self.gate_up, self.down = norm, router, layer, gate_up, down
        self.hidden, self.sh_inter = layer.hidden, down.in_features
        if layer.sh_inter:
            raise ValueError("the layer's own shared expert would be added twice")
        if gate_up.out_features != 2 * self.sh_inter or gate_up.in_features != self.hidden or down.out_features != self.hidden:
            raise ValueError("shared expert: gate_up %d x %d, down %d x %d do not fit hidden %d"
                             % (gate_up.out_features, gate_up.in_features, down.out_features, down.in_features, self.hidden))
        if (router.hidden, router.n_experts, router.top_k) != (layer.hidden, layer.n_experts, layer.top_k):
            raise ValueError("router and layer differ in hidden, experts or top k")

    def __call__(self, x, residual, b: BlockBuffers, stream=None):
        """x, residual: [T, H] rows; residual is updated in place.  Returns b.y."""
        M.residual_norm(self.norm, x, residual, residual, b.n, b.q, b.q_scale, stream)
        M.route_scored(self.router, b.n, b.routing, b.ws_route, stream)
        ffn = M.ffn_decode if b.path == M.PATH_DECODE else M.ffn_prefill
        ffn(self.layer, b.n, M.ACT_BF16, b.T, b.routing, b.y, b.ws_ffn, stream)
        M.linear_i8(self.gate_up, b.q, b.q_scale, b.gate_up, None, b.ws_up, stream)
        M.quant_i8(b.gate_up, b.h, b.h_scale, True, stream)
        M.linear_i8(self.down, b.h, b.h_scale, b.y, b.y, b.ws_down, stream)
        return b.y
