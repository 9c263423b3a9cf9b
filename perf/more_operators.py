"""Cases of the operators for a few tokens of many requests: what they take, their plain forms and what they must move.

Three operators, each with its plain form here (elementary torch operations) and, where `own` is true, the calls that a
program makes of the library:

  block     s = x + residual, n = rms_norm(s), scored routing of n, y = sum_j w_j FFN_{e_j}(n) + FFN_shared(n) for a few tokens;
            routed experts with gate and up in the 2-bit codebook format and down in Q2_K, the shared expert's weights in int8
  plan      the tokens of a batch sorted by the adapter that their request has
  adapters  y[t] = add[t] + scale_a B_a (A_a x[t]) with a the adapter of token t, beside a projection of several parts
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4, "i8": 1, "none": 0}


# ------------------------------------------------------------------ cases
def _block(T, H, I, E, k, shared, n, res, score, groups, keep):
    return {"op": "block", "T": T, "H": H, "I": I, "E": E, "k": k, "shared": shared, "n": n, "res": res, "score": score,
            "groups": groups, "keep": keep}


def _plan(T, adapters, runs):
    return {"op": "plan", "T": T, "adapters": adapters, "runs": runs}


def _adapters(T, K, N, parts, rank, adapters, runs, x, y):
    return {"op": "adapters", "T": T, "K": K, "N": N, "parts": parts, "rank": rank, "adapters": adapters, "runs": runs, "x": x,
            "y": y}


def listed():
    return [
        # one decoded token through the full layer: 256 experts in 8 groups of which 4 are kept
        dict(_block(1, 7168, 2048, 256, 8, 2048, "bf16", "bf16", "sigmoid", 8, 4), name="block_1"),
        # three tokens through a narrow layer whose sizes fit no block of 256, softmax scores, no shared expert
        dict(_block(3, 1112, 712, 24, 5, 0, "f32", "f32", "softmax", 1, 1), name="block_odd"),
        # the steps of four sessions, or one session's guesses, through the full layer
        dict(_block(4, 7168, 2048, 256, 8, 2048, "bf16", "bf16", "sigmoid", 8, 4), name="block_4"),
        # a small batch through a mid-sized layer
        dict(_block(16, 2048, 768, 64, 6, 1408, "bf16", "bf16", "sigmoid", 1, 1), name="block_16"),
        # a decode batch, a request a token
        dict(_plan(64, 16, False), name="plan_64"),
        # prompts of many requests, one after another
        dict(_plan(8192, 100, True), name="plan_8192"),
        # one token beside the shared expert's gate and up rows
        dict(_adapters(1, 7168, 4096, 2, 16, 16, False, "bf16", "f32"), name="adapters_1"),
        # a decode batch of 64 requests with 32 adapters at the same place
        dict(_adapters(64, 7168, 4096, 2, 16, 32, False, "bf16", "f32"), name="adapters_64"),
        # a ragged chunk beside a projection whose sizes fit no tile
        dict(_adapters(333, 1111, 1003, 1, 13, 5, True, "f32", "bf16"), name="adapters_odd"),
        # a chunk beside the shared expert's down rows, whose inputs are codes
        dict(_adapters(512, 2048, 7168, 1, 32, 8, True, "i8", "f32"), name="adapters_512"),
        # prompts of a few requests
        dict(_adapters(8192, 7168, 4096, 2, 64, 8, True, "bf16", "bf16"), name="adapters_8192"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["block", "block", "plan", "adapters", "adapters"])
    if op == "plan":
        return _plan(_log(rng, 1, 8192), _log(rng, 1, 256), rng.random() < 0.5)
    if op == "adapters":
        T, K, N, rank = _log(rng, 1, 8192), _log(rng, 64, 7168), _log(rng, 64, 7168), _log(rng, 4, 64)
        parts = rng.choice([1, 1, 2, 3])
        N = parts * max(1, N // parts)
        while T * parts * rank * (K + N // parts) > 8192 * 128 * (7168 + 2048):
            T = (T + 1) // 2
        return _adapters(T, K, N, parts, rank, _log(rng, 1, 64), rng.random() < 0.5, rng.choice(["bf16", "bf16", "f32", "i8"]),
                         rng.choice(["bf16", "f32"]))
    T = rng.randint(1, 16)
    groups = rng.choice([1, 1, 4, 8])
    E = groups * _log(rng, 4, 256 // groups)
    keep = rng.randint(max(1, groups // 2), groups)
    k = rng.randint(1, min(8, keep * (E // groups)))
    H, I = 8 * _log(rng, 32, 896), 8 * _log(rng, 16, 256)
    while T * k * H * I > 4 * 8 * 7168 * 2048:
        T -= 1
    shared = rng.choice([0, _log(rng, 64, 2048)])
    return _block(T, H, I, E, k, shared, rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32", "none"]),
                  rng.choice(["sigmoid", "softmax"]), groups, keep)


# ------------------------------------------------------------------ inputs
def _round16(n):
    return (n + 15) // 16 * 16


def _blocks(g, matrices, rows, K, size):
    """Random bytes of quantized matrices [matrices, rows, blocks, size], their fp16 fields still to be set."""
    return torch.randint(0, 256, (matrices, rows, (K + 255) // 256, size), generator=g, device="cuda", dtype=torch.uint8)


def _half_field(blocks, at, values):
    """fp16 values into bytes at, at + 1 of every block."""
    blocks[..., at:at + 2] = values.to(torch.float16)[..., None].view(torch.uint8)


def _padding(blocks, K, fmt):
    """The last block's weights past K, as the packer leaves them: scales (and mins) of whole sub-blocks 0 past K. Codes of the
    rest of the sub-block that K ends in may be anything: they meet no input."""
    rest = K % 256
    if not rest:
        return
    if fmt == "cb2":
        first = (rest + 31) // 32
        for j in range(first, 8):
            blocks[:, :, -1, 2 + j // 2] &= 0xF0 if j % 2 == 0 else 0x0F
    else:
        blocks[:, :, -1, 4 + (rest + 15) // 16:20] = 0


def _i8_rows(g, N, K):
    q = torch.zeros((N, _round16(K)), dtype=torch.int8, device="cuda")
    q[:, :K] = torch.clamp(torch.round(torch.randn((N, K), generator=g, device="cuda") * 35), -127, 127).to(torch.int8)
    return q[:, :K], (0.5 + torch.rand(N, generator=g, device="cuda")) * (0.02 / 35)


def _ids(g, T, n, runs):
    """The adapter of every token, -1 for none: a request a token, or requests one after another."""
    if runs:
        lengths = torch.randint(1, max(2, 2 * T // max(1, n)), (T,), generator=g, device="cuda")
        request = torch.searchsorted(torch.cumsum(lengths, 0), torch.arange(T, device="cuda"), right=True)
    else:
        request = torch.arange(T, device="cuda")
    of = torch.randint(0, n, (T + 1,), generator=g, device="cuda")
    none = torch.rand(T + 1, generator=g, device="cuda") < 0.15
    none[request[0]] = False
    return torch.where(none, -1, of)[request].int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, kind="f32"):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(_TYPES[kind])

    c, T = case, case["T"]
    s = {"case": dict(case)}
    if c["op"] == "block":
        H, I, E = c["H"], c["I"], c["E"]
        s["x"] = normal(T, H, std=0.5)
        s["res"] = None if c["res"] == "none" else normal(T, H, std=2.0, kind=c["res"])
        s["g"], s["eps"] = 1.0 + normal(H, std=0.2), 1e-6
        s["router"] = normal(E, H, std=H ** -0.5)
        s["bias"] = normal(E, std=0.05 if c["score"] == "sigmoid" else 0.1 / E)
        s["scale"] = 2.5
        s["codebook"] = (torch.randint(0, 4, (256, 8), generator=g, device="cuda") * 2 - 3).to(torch.int8)
        for name in ("gate", "up"):
            w = _blocks(g, E, I, H, 38)
            _half_field(w, 0, 0.0007 + 0.0006 * torch.rand(w.shape[:3], generator=g, device="cuda"))
            _padding(w, H, "cb2")
            s[name] = w
        w = _blocks(g, E, H, I, 84)
        d = 0.0015 + 0.001 * torch.rand(w.shape[:3], generator=g, device="cuda")
        _half_field(w, 0, d)
        _half_field(w, 2, 1.5 * d)
        _padding(w, I, "q2k")
        s["down"] = w
        if c["shared"]:
            s["sh_up"], s["sh_up_scale"] = _i8_rows(g, 2 * c["shared"], H)
            s["sh_down"], s["sh_down_scale"] = _i8_rows(g, H, c["shared"])
    else:
        s["ids"] = _ids(g, T, c["adapters"], c["runs"])
    if c["op"] == "adapters":
        K, N, R, n = c["K"], c["N"], c["parts"] * c["rank"], c["adapters"]
        if c["x"] == "i8":
            s["x"], _ = _i8_rows(g, T, K)
            s["xs"] = (0.5 + torch.rand(T, generator=g, device="cuda")) / 35
        else:
            s["x"], s["xs"] = normal(T, K, kind=c["x"]), None
        s["a"] = normal(n, R, K, std=K ** -0.5, kind="bf16")
        s["b"] = normal(n, N, c["rank"], std=c["rank"] ** -0.5, kind="bf16")
        s["scale"] = 0.5 + torch.rand(n, generator=g, device="cuda")
        s["add"] = normal(T, N, kind=c["y"])
    if own:
        _keep(s)
    return s


# ------------------------------------------------------------------ the library's calls
def _keep(s):
    """What a program keeps between calls: the handle, the buffers and the workspace."""
    import bit_quantized_routed_amd as M
    c, T = s["case"], s["case"]["T"]

    def empty(*shape, kind="f32"):
        return torch.empty(shape, dtype=_TYPES[kind], device="cuda")

    s["M"], s["stream"] = M, torch.cuda.current_stream().cuda_stream
    if c["op"] == "block":
        router = M.RouterWeights(s["router"], c["k"], c["score"], s["bias"], c["groups"], c["keep"], True, s["scale"])
        layer = M.DeviceLayer(c["H"], c["I"], c["E"], c["k"], M.FMT_CB2, M.FMT_Q2K, s["gate"], s["up"], s["down"], s["codebook"],
                              s["router"])
        gate_up = down = None
        if c["shared"]:
            gate_up, down = M.LinearI8(s["sh_up"], s["sh_up_scale"]), M.LinearI8(s["sh_down"], s["sh_down_scale"])
        s["h"] = M.BlockWeights(M.NormWeights(s["g"], s["eps"]), router, layer, gate_up, down, _TYPES[c["n"]])
        s["total"] = None if s["res"] is None else torch.empty_like(s["res"])
        s["y"], s["r"], s["wksp"] = empty(T, c["H"]), M.Routing(T, c["k"], c["E"]), s["h"].workspace(T)
    else:
        s["plan"] = M.AdapterPlan(T, c["adapters"])
    if c["op"] == "adapters":
        s["h"] = M.AdapterWeights(s["a"], s["b"], s["scale"], c["parts"])
        s["y"], s["wksp"] = empty(T, c["N"], kind=c["y"]), s["h"].workspace(T)
        M.adapter_plan(s["ids"], s["plan"], s["stream"])      # one plan serves every projection of a step


def _own_block(s):
    r = s["r"]
    s["M"].block_decode(s["h"], s["x"], s["res"], s["total"], s["y"], r, s["wksp"], s["stream"])
    return [s["total"], s["y"], r.topk_idx, r.topk_w, r.offsets, r.perm, r.inv]


def _own_plan(s):
    s["M"].adapter_plan(s["ids"], s["plan"], s["stream"])
    return [s["plan"].order, s["plan"].offsets]


def _own_adapters(s):
    s["M"].adapters(s["h"], s["plan"], s["x"], s["xs"], s["y"], s["add"], s["wksp"], s["stream"])
    return [s["y"]]


# ------------------------------------------------------------------ plain forms
def run(state):
    op = state["case"]["op"]
    if own:
        return {"block": _own_block, "plan": _own_plan, "adapters": _own_adapters}[op](state)
    return {"block": _plain_block, "plan": _plain_plan, "adapters": _plain_adapters}[op](state)


def _half(blocks, at):
    return blocks[..., at:at + 2].contiguous().view(torch.float16).float()


def _plain_cb2(w, codebook, K):
    """[P, rows, blocks, 38] bytes to [P, rows, K] weights."""
    s = torch.stack([w[..., 2:6] & 15, w[..., 2:6] >> 4], -1).flatten(-2).float()              # eight sub-blocks of 32
    step = _half(w, 0) * s
    v = codebook.float()[w[..., 6:38].long()].unflatten(-2, (8, 4)) * step[..., None, None]
    return v.flatten(2)[..., :K]


def _plain_q2k(w, K):
    """[P, rows, blocks, 84] bytes to [P, rows, K] weights."""
    sc, m = (w[..., 4:20] & 15).float() * _half(w, 0), (w[..., 4:20] >> 4).float() * _half(w, 2)
    q = torch.stack([w[..., 20:84] >> (2 * i) & 3 for i in range(4)], -1).flatten(-2).unflatten(-1, (16, 16)).float()
    return (q * sc[..., None] - m[..., None]).flatten(2)[..., :K]


def _plain_ffn(x, gate, up, down):
    """down (silu(gate x) * up x) for rows x [P, K] and a matrix each [P, ...]."""
    a, u = torch.matmul(gate, x[:, :, None])[..., 0], torch.matmul(up, x[:, :, None])[..., 0]
    h = a / (1.0 + torch.exp(-a)) * u
    return torch.matmul(down, h[:, :, None])[..., 0]


def _plain_norm(s):
    """The residual's sum as it is kept, and its norm: the mean of squares in 64 bits, the products in 32, one after the other."""
    total, v = None, s["x"]
    if s["res"] is not None:
        total = (v + s["res"].float()).to(s["res"].dtype)
        v = total.float()
    r = (1.0 / torch.sqrt(v.double().square().mean(1, keepdim=True) + s["eps"])).float()
    return total, ((v * r) * s["g"]).to(_TYPES[s["case"]["n"]]).float()


def _plain_route(s, n):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    # 64 bits: which expert is taken turns on the last bits of scores that nearly tie
    l = n.double() @ s["router"].double().t()
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
    else:
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    chosen = p + s["bias"].double()
    if c["keep"] < G:
        of = chosen.view(T, G, E // G)
        best = torch.sort(of, dim=2, descending=True).values[:, :, :2].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        mask = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        chosen = torch.where(mask[:, :, None], of, -math.inf).view(T, E)
    idx = torch.sort(chosen, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(p, 1, idx)
    w = (w / w.sum(1, keepdim=True) * s["scale"]).float()
    flat = idx.reshape(-1)
    perm = torch.sort(flat, stable=True).indices
    inv = torch.empty_like(perm).scatter_(0, perm, torch.arange(T * k, device=l.device))
    offsets = torch.searchsorted(flat[perm], torch.arange(E + 1, device=l.device))
    return idx, w, offsets, perm, inv


def _plain_block(s):
    c = s["case"]
    total, n = _plain_norm(s)
    idx, w, offsets, perm, inv = _plain_route(s, n)
    at = idx.reshape(-1)
    each = _plain_ffn(n.repeat_interleave(c["k"], 0), _plain_cb2(s["gate"][at], s["codebook"], c["H"]),
                      _plain_cb2(s["up"][at], s["codebook"], c["H"]), _plain_q2k(s["down"][at], c["I"]))
    y = (each.unflatten(0, (c["T"], c["k"])) * w[..., None]).sum(1)
    if c["shared"]:
        a, u = ((n @ s["sh_up"].float().t()) * s["sh_up_scale"]).chunk(2, 1)
        y = y + ((a / (1.0 + torch.exp(-a)) * u) @ s["sh_down"].float().t()) * s["sh_down_scale"]
    return [total, y, idx.int(), w, offsets.int(), perm.int(), inv.int()]


def _plain_plan(s):
    n = s["case"]["adapters"]
    key = torch.where((s["ids"] >= 0) & (s["ids"] < n), s["ids"], n)
    order = torch.sort(key, stable=True).indices
    return [order.int(), torch.searchsorted(key[order], torch.arange(n + 1, dtype=key.dtype, device=key.device)).int()]


def _plain_adapters(s):
    c = s["case"]
    T, r, parts = c["T"], c["rank"], c["parts"]
    x = s["x"].float() if s["xs"] is None else s["x"].float() * s["xs"][:, None]
    # every adapter on every token, then each token's own
    low = torch.matmul(x, s["a"].float().flatten(0, 1).t()).unflatten(1, (c["adapters"], parts, r))
    has = s["ids"] >= 0
    of = torch.where(has, s["ids"], 0).long()
    factor = torch.where(has, s["scale"][of], 0.0)
    low = torch.zeros_like(low).scatter_(1, of[:, None, None, None].expand(T, 1, parts, r),
                                         low.gather(1, of[:, None, None, None].expand(T, 1, parts, r)) * factor[:, None, None, None])
    b = s["b"].float().unflatten(1, (parts, c["N"] // parts)).permute(1, 0, 3, 2).flatten(1, 2)     # [parts, adapters * r, N / parts]
    add = torch.matmul(low.permute(2, 0, 1, 3).flatten(2), b).permute(1, 0, 2).flatten(1)
    return [(s["add"].float() + add).to(s["add"].dtype)]


# ------------------------------------------------------------------ what a pass has to do
def work(case):
    c, T = case, case["T"]
    if c["op"] == "plan":
        return {"bytes": 8 * T + 4 * (c["adapters"] + 1), "flops": T}
    if c["op"] == "adapters":
        K, N, R = c["K"], c["N"], c["parts"] * c["rank"]
        # adapters in use, where each request's is drawn evenly and most have one
        requests = min(T, max(1, c["adapters"])) if c["runs"] else 0.85 * T
        used = c["adapters"] * (1.0 - (1.0 - 1.0 / c["adapters"]) ** max(1.0, requests))
        b = T * K * _SIZE[c["x"]] + 2 * T * N * _SIZE[c["y"]] + used * 2 * (R * K + N * c["rank"]) + 4 * T
        return {"bytes": int(b), "flops": 2 * T * (R * K + N * c["rank"])}
    H, I, E, k, sh = c["H"], c["I"], c["E"], c["k"], c["shared"]
    used = E * (1.0 - (1.0 - k / E) ** T)        # different experts among T tokens' k, drawn evenly
    expert = 2 * I * ((H + 255) // 256) * 38 + H * ((I + 255) // 256) * 84
    b = used * expert + 4 * E * H + 3 * H * sh + T * H * (4 + 2 * _SIZE[c["res"]] + 4) + 16 * T * k + 4 * (E + 1)
    return {"bytes": int(b), "flops": 2 * T * (3 * H * I * k + 3 * H * sh + E * H)}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    if case["op"] == "plan":
        return None                              # whole numbers
    s = prepare(case, seed)
    return _exact_block(s) if case["op"] == "block" else _exact_adapters(s)


def _exact_weights(w, K, codebook):
    """One matrix [rows, blocks, bytes] as [rows, K] in 64 bits."""
    half = lambda at: w[..., at:at + 2].contiguous().view(torch.float16).double()  # noqa: E731
    if codebook is not None:
        scales = torch.empty((*w.shape[:2], 8), dtype=torch.float64, device=w.device)
        scales[..., 0::2], scales[..., 1::2] = (w[..., 2:6] % 16).double(), (w[..., 2:6] // 16).double()
        v = codebook.double()[w[..., 6:38].int()].reshape(*w.shape[:2], 256) * (half(0) * scales).repeat_interleave(32, -1)
    else:
        at = torch.arange(256, device=w.device)
        q = w[..., 20 + at // 4].int().div(4 ** (at % 4), rounding_mode="floor") % 4
        sc, m = (w[..., 4:20] % 16).double(), (w[..., 4:20] // 16).double()
        v = q * (half(0) * sc).repeat_interleave(16, -1) - (half(2) * m).repeat_interleave(16, -1)
    return v.reshape(w.shape[0], -1)[:, :K]


def _exact_block(s):
    c = s["case"]
    E, k, G, size = c["E"], c["k"], c["groups"], c["E"] // c["groups"]
    d, total = s["x"].double(), None
    if s["res"] is not None:
        total = (d + s["res"].double()).float().to(s["res"].dtype).double()        # the sum as it is kept
        d = total
    # the norm's stated roundings: its factor and both products to 32 bits, the result to the type that the layer takes
    f = (d.pow(2).sum(-1, keepdim=True) / c["H"] + s["eps"]).pow(-0.5).float().double()
    n = ((d * f).float().double() * s["g"].double()).float().to(_TYPES[c["n"]]).double()
    l = torch.mm(n, s["router"].double().t())
    p = torch.special.expit(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
    v = p + s["bias"].double()
    rank_of = lambda v: ((v[:, None, :] > v[:, :, None]) | ((v[:, None, :] == v[:, :, None]) & _below(v.shape[1]))).sum(2)  # noqa: E731
    if c["keep"] < G:
        of = v.reshape(-1, G, size)
        top = of.amax(2)
        if size > 1:
            top = top + of.scatter(2, of.argmax(2, keepdim=True), -math.inf).amax(2)
        v = torch.where((rank_of(top) < c["keep"]).repeat_interleave(size, 1), v, torch.full_like(v, -math.inf))
    at = torch.argsort(rank_of(v), dim=1)[:, :k]
    part = p.gather(1, at)
    w = part / part.sum(1, keepdim=True) * s["scale"]
    y = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=d.device)
    for e in at.unique().tolist():
        t, j = torch.nonzero(at == e, as_tuple=True)
        x = n[t]
        a, u = (torch.mm(x, _exact_weights(s[name][e], c["H"], s["codebook"]).t()) for name in ("gate", "up"))
        y.index_add_(0, t, torch.mm(a * torch.special.expit(a) * u, _exact_weights(s["down"][e], c["I"], None).t()) * w[t, j][:, None])
    if c["shared"]:
        up, down = (s[name].double() * s[name + "_scale"].double()[:, None] for name in ("sh_up", "sh_down"))
        a, u = torch.mm(n, up.t()).split(c["shared"], dim=1)
        y += torch.mm(a * torch.special.expit(a) * u, down.t())
    return [total, y, None, w, None, None, None]


def _below(n):
    return torch.ones((n, n), dtype=torch.bool, device="cuda").tril(-1)


def _exact_adapters(s):
    c = s["case"]
    y = s["add"].double()
    x = s["x"].double() if s["xs"] is None else s["x"].double() * s["xs"].double()[:, None]
    wide = c["N"] // c["parts"]
    for a in s["ids"].unique().tolist():
        if a < 0:
            continue
        t = torch.nonzero(s["ids"] == a)[:, 0]
        low = torch.mm(x[t], s["a"][a].double().t()) * s["scale"][a].double()
        for q in range(c["parts"]):
            y[t, q * wide:(q + 1) * wide] += torch.mm(low[:, q * c["rank"]:(q + 1) * c["rank"]],
                                                      s["b"][a, q * wide:(q + 1) * wide].double().t())
    return [y]
