"""One MoE block on the library's operators: residual + norm, scored router,
quantized routed experts, and the shared expert in 8 bits.

    s   = x + residual                        (kept as the new residual)
    n   = rms_norm(s)                         bf16 for the router and the experts, int8 for the shared expert
    y   = sum_j w_j FFN_{e_j}(n)              quantized routed experts, fp32
    y  += W_down silu(W_gate n) * (W_up n)    int8 rows and weights

x of the next block is y: it joins the residual in that block's norm.

`MoeBlock.__call__` runs the operators one after the other, for any number of tokens and with the low-rank adapters of
the tokens' requests on the shared expert's projections; `MoeBlock.decode` runs the block of up to 16 tokens in two
kernels, with the shared expert's activations in full (they are not cut to 8 bits).
"""
from __future__ import annotations

import bit_quantized_routed_amd as M

# tokens up to which the decode path of the routed experts is the faster one
DECODE_TOKENS = 64
# tokens that moe_block_decode takes
FEW_TOKENS = 16


class StepAdapters:
    """The adapters of one step at one block: the step's plan (M.AdapterPlan, filled by M.adapter_plan) and the weights beside
    the shared expert's gate/up rows (two parts) and its down rows, either of them None.  Blocks that run one after another may
    share one; steps in flight at the same time need one each."""

    def __init__(self, plan, gate_up=None, down=None, device="cuda"):
        self.plan, self.gate_up, self.down = plan, gate_up, down
        sizes = [w.workspace(plan.T, device) for w in (gate_up, down) if w is not None]
        self.ws = max(sizes, key=lambda t: t.nbytes) if sizes else None

    def check(self, block: "MoeBlock", T: int):
        """Raises ValueError unless this is a step of T tokens and fits the block."""
        if self.plan.T != T:
            raise ValueError("adapters: a plan of %d tokens, a step of %d" % (self.plan.T, T))
        for name, w, K, N in (("gate_up", self.gate_up, block.hidden, 2 * block.sh_inter), ("down", self.down, block.sh_inter, block.hidden)):
            if w is not None and (w.in_features, w.out_features, w.n_adapters) != (K, N, self.plan.n_adapters):
                raise ValueError("adapters: %s of %d, %d x %d beside %d x %d, in a plan of %d"
                                 % (name, w.n_adapters, w.out_features, w.in_features, N, K, self.plan.n_adapters))


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
        self.ws_few = block.few.workspace(T, device) if block.few is not None and T <= FEW_TOKENS else None


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
        few = M.BlockWeights(norm, router, layer, gate_up, down)
        self.few = few if few.takes(1) else None

    def decode(self, x, residual, b: BlockBuffers, stream=None):
        """The block for up to 16 tokens in two kernels (see moe_block_decode).  x, residual: [T, H] rows; residual is updated in
        place.  Returns b.y, and b.routing is filled (n and what lies between stay in the kernels).  Buffers that may be in use
        at the same time need a BlockBuffers each.  Faster than __call__ for every batch that it takes: of the full layer (7168
        features, experts of 2048, 8 of 256) 1 token 56 us (66), 4 122 (190), 8 234 (391), 16 412 (560)."""
        if b.ws_few is None:
            raise ValueError("decode takes up to %d tokens of a CB2 / Q2_K layer, of at most 8192 features, 512 experts and top 16"
                             % FEW_TOKENS)
        M.block_decode(self.few, x, residual, residual, b.y, b.routing, b.ws_few, stream)
        return b.y

    def __call__(self, x, residual, b: BlockBuffers, stream=None, adapters: StepAdapters | None = None):
        """x, residual: [T, H] rows; residual is updated in place.  Returns b.y."""
        if adapters is not None:
            adapters.check(self, b.T)            # before the first launch changes the residual
        M.residual_norm(self.norm, x, residual, residual, b.n, b.q, b.q_scale, stream)
        M.route_scored(self.router, b.n, b.routing, b.ws_route, stream)
        ffn = M.ffn_decode if b.path == M.PATH_DECODE else M.ffn_prefill
        ffn(self.layer, b.n, M.ACT_BF16, b.T, b.routing, b.y, b.ws_ffn, stream)
        M.linear_i8(self.gate_up, b.q, b.q_scale, b.gate_up, None, b.ws_up, stream)
        if adapters is not None and adapters.gate_up is not None:
            M.adapters(adapters.gate_up, adapters.plan, b.n, None, b.gate_up, None, adapters.ws, stream)
        M.quant_i8(b.gate_up, b.h, b.h_scale, True, stream)
        M.linear_i8(self.down, b.h, b.h_scale, b.y, b.y, b.ws_down, stream)
        if adapters is not None and adapters.down is not None:
            M.adapters(adapters.down, adapters.plan, b.h, b.h_scale, b.y, None, adapters.ws, stream)
        return b.y
