"""Cases of the operators around the routed experts: what they take, their plain forms and what they must move.

Four operators, each with its plain form here (elementary torch operations) and, where `own` is true, the calls that a
program makes of the library:

  norm    s = x + residual (rounded to the residual's type), v = s / rms(s) * g, as `out` and as int8 with a scale per token
  quant   rows to int8 with a scale each; with "swiglu" the row is silu(gate) * up of a row [gate | up]
  linear  y[t, n] = (sum_k x[t, k] w[n, k]) * xs[t] * ws[n] (+ bias[n]) (+ add[t, n]), x and w in int8
  route   router scores (sigmoid or softmax), a selection bias, groups of experts, top-k, weights, and the grouping by expert
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4, "none": 0}


# ------------------------------------------------------------------ cases
def _norm(T, H, x, res, out, q):
    return {"op": "norm", "T": T, "H": H, "x": x, "res": res, "out": out, "q": q}


def _quant(T, K, x, swiglu):
    return {"op": "quant", "T": T, "K": K, "x": x, "swiglu": swiglu}


def _linear(T, N, K, y, bias, add):
    return {"op": "linear", "T": T, "N": N, "K": K, "y": y, "bias": bias, "add": add}


def _route(T, H, E, k, x, score, groups, keep, renorm):
    return {"op": "route", "T": T, "H": H, "E": E, "k": k, "x": x, "score": score, "groups": groups, "keep": keep,
            "renorm": renorm}


def listed():
    return [
        # one decoded token: the expert layer's fp32 output joins the bf16 residual, then the next norm
        dict(_norm(1, 7168, "f32", "bf16", "bf16", True), name="norm_1"),
        # a ragged batch of a narrower model kept in fp32, no residual
        dict(_norm(333, 1112, "f32", "none", "f32", True), name="norm_odd"),
        # a long prompt of the full layer: bf16 for the router and the experts, int8 for the dense projections
        dict(_norm(8192, 7168, "f32", "bf16", "bf16", True), name="norm_8192"),
        # one token's shared-expert intermediate
        dict(_quant(1, 2048, "f32", True), name="quant_1"),
        # a prompt's shared-expert intermediate
        dict(_quant(8192, 2048, "bf16", True), name="quant_8192"),
        # one token through the shared expert's gate and up rows
        dict(_linear(1, 4096, 7168, "f32", False, False), name="linear_1"),
        # a decode batch through the shared expert's down rows, added to the routed experts' sum
        dict(_linear(32, 7168, 2048, "f32", False, True), name="linear_32"),
        # a ragged chunk through a projection whose sizes fit no tile
        dict(_linear(333, 1003, 1111, "bf16", True, False), name="linear_odd"),
        # a long prompt through the shared expert's gate and up rows
        dict(_linear(8192, 4096, 7168, "bf16", False, False), name="linear_8192"),
        # one decoded token: 256 experts in 8 groups of which 4 are kept
        dict(_route(1, 7168, 256, 8, "bf16", "sigmoid", 8, 4, True), name="route_1"),
        # a ragged chunk, softmax scores over all experts
        dict(_route(333, 1112, 160, 6, "f32", "softmax", 1, 1, False), name="route_odd"),
        # a long prompt
        dict(_route(8192, 7168, 256, 8, "bf16", "sigmoid", 8, 4, True), name="route_8192"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quant", "linear", "route"])
    T = _log(rng, 1, 8192)
    if op == "norm":
        return _norm(T, _log(rng, 64, 7168), rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32", "none"]),
                     rng.choice(["bf16", "f32"]), rng.random() < 0.7)
    if op == "quant":
        return _quant(T, _log(rng, 64, 4096), rng.choice(["bf16", "f32"]), rng.random() < 0.6)
    if op == "linear":
        N, K = _log(rng, 64, 7168), _log(rng, 64, 7168)
        while T * N * K > 8192 * 4096 * 7168:
            N = (N + 1) // 2
        return _linear(T, N, K, rng.choice(["bf16", "f32"]), rng.random() < 0.4, rng.random() < 0.4)
    groups = rng.choice([1, 1, 4, 8])
    E = groups * _log(rng, 4, 256 // groups)
    keep = rng.randint(max(1, groups // 2), groups)
    k = rng.randint(1, min(8, keep * (E // groups)))
    return _route(T, 8 * _log(rng, 8, 896), E, k, rng.choice(["bf16", "f32"]), rng.choice(["sigmoid", "softmax"]),
                  groups, keep, rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _round16(n):
    return (n + 15) // 16 * 16


def _rows8(v):
    """Rows of v as int8 codes (in rows of a multiple of 16 bytes) and their scales."""
    T, K = v.shape
    amax = v.abs().amax(1, keepdim=True)
    q = torch.zeros((T, _round16(K)), dtype=torch.int8, device=v.device)
    q[:, :K] = torch.round(v * (127.0 / amax)).to(torch.int8)
    return q[:, :K], (amax / 127.0).reshape(T).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, kind="f32"):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(_TYPES[kind])

    c, T = case, case["T"]
    s = {"case": dict(case)}
    if c["op"] == "norm":
        s["x"] = normal(T, c["H"], std=0.5, kind=c["x"])
        s["res"] = None if c["res"] == "none" else normal(T, c["H"], std=2.0, kind=c["res"])
        s["g"] = 1.0 + normal(c["H"], std=0.2)
        s["eps"] = 1e-6
    elif c["op"] == "quant":
        s["x"] = normal(T, c["K"] * (2 if c["swiglu"] else 1), kind=c["x"])
    elif c["op"] == "linear":
        s["x"], s["xs"] = _rows8(normal(T, c["K"]))
        s["w"], s["ws"] = _rows8(normal(c["N"], c["K"], std=0.02))
        s["bias"] = normal(c["N"], std=0.1) if c["bias"] else None
        s["add"] = normal(T, c["N"], kind=c["y"]) if c["add"] else None
    else:
        s["x"] = normal(T, c["H"], kind=c["x"])
        s["w"] = normal(c["E"], c["H"], std=c["H"] ** -0.5)
        s["bias"] = normal(c["E"], std=0.05 if c["score"] == "sigmoid" else 0.1 / c["E"])
        s["scale"] = 2.5
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
    if c["op"] == "norm":
        s["h"] = M.NormWeights(s["g"], s["eps"])
        s["total"] = None if s["res"] is None else torch.empty_like(s["res"])
        s["out"] = empty(T, c["H"], kind=c["out"])
    if c["op"] == "quant" or c["op"] == "norm" and c["q"]:
        n = c["H"] if c["op"] == "norm" else c["K"]
        s["q"], s["qs"], s["values"] = M.empty_i8(T, n), empty(T), empty(T, n, kind="bf16")
    if c["op"] == "linear":
        s["h"] = M.LinearI8(s["w"], s["ws"], s["bias"])
        s["y"], s["wksp"] = empty(T, c["N"], kind=c["y"]), s["h"].workspace(T)
    if c["op"] == "route":
        s["h"] = M.RouterWeights(s["w"], c["k"], c["score"], s["bias"], c["groups"], c["keep"], c["renorm"], s["scale"])
        s["r"], s["wksp"] = M.Routing(T, c["k"], c["E"]), s["h"].workspace(T)


def _values(s):
    """The values that the int8 codes stand for, and the scales."""
    return [torch.mul(s["q"], s["qs"][:, None], out=s["values"]), s["qs"]]


def _own_norm(s):
    coded = s["case"]["q"]
    s["M"].residual_norm(s["h"], s["x"], s["res"], s["total"], s["out"], s["q"] if coded else None,
                         s["qs"] if coded else None, s["stream"])
    return [s["total"], s["out"]] + (_values(s) if coded else [None, None])


def _own_quant(s):
    s["M"].quant_i8(s["x"], s["q"], s["qs"], s["case"]["swiglu"], s["stream"])
    return _values(s)


def _own_linear(s):
    s["M"].linear_i8(s["h"], s["x"], s["xs"], s["y"], s["add"], s["wksp"], s["stream"])
    return [s["y"]]


def _own_route(s):
    r = s["r"]
    s["M"].route_scored(s["h"], s["x"], r, s["wksp"], s["stream"])
    return [r.topk_idx, r.topk_w, r.offsets, r.perm, r.inv]


# ------------------------------------------------------------------ plain forms
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "quant": _own_quant, "linear": _own_linear, "route": _own_route}[op](state)
    return {"norm": _plain_norm, "quant": _plain_quant, "linear": _plain_linear, "route": _plain_route}[op](state)


def _plain_codes(v):
    """Rows of fp32 v: the values their int8 codes stand for, and the scales."""
    amax = v.abs().amax(1, keepdim=True)
    scale = amax / 127.0
    q = torch.round(v * torch.where(amax > 0, 127.0 / amax, 0.0))
    return (q * scale).to(torch.bfloat16), scale[:, 0]


def _plain_norm(s):
    c = s["case"]
    total, v = None, s["x"].float()
    if s["res"] is not None:
        total = (v + s["res"].float()).to(s["res"].dtype)
        v = total.float()
    # the mean of squares in 64 bits: codes next to a border turn on its last bits
    r = (1.0 / torch.sqrt(v.double().square().mean(1, keepdim=True) + s["eps"])).float()
    v = (v * r) * s["g"]
    vals, scale = _plain_codes(v) if c["q"] else (None, None)
    return [total, v.to(_TYPES[c["out"]]), vals, scale]


def _plain_quant(s):
    c, v = s["case"], s["x"].float()
    if c["swiglu"]:
        a, b = v[:, :c["K"]], v[:, c["K"]:]
        v = a / (1.0 + torch.exp(-a)) * b
    return list(_plain_codes(v))


def _plain_linear(s):
    c = s["case"]
    y = s["x"].float() @ s["w"].float().t()
    y = y * (s["xs"][:, None] * s["ws"][None, :])
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["add"] is not None:
        y = y + s["add"].float()
    return [y.to(_TYPES[c["y"]])]


def _plain_route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    # 64 bits: which expert is taken turns on the last bits of scores that nearly tie
    l = s["x"].double() @ s["w"].double().t()
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
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = (w * s["scale"]).float()
    flat = idx.reshape(-1)
    perm = torch.sort(flat, stable=True).indices
    inv = torch.empty_like(perm).scatter_(0, perm, torch.arange(T * k, device=l.device))
    offsets = torch.searchsorted(flat[perm], torch.arange(E + 1, device=l.device))
    return [idx.int(), w, offsets.int(), perm.int(), inv.int()]


# ------------------------------------------------------------------ what a pass has to do
def work(case):
    c, T = case, case["T"]
    if c["op"] == "norm":
        n = T * c["H"]
        b = n * (_SIZE[c["x"]] + 2 * _SIZE[c["res"]] + _SIZE[c["out"]] + (1 if c["q"] else 0)) + 4 * c["H"] + (4 * T if c["q"] else 0)
        return {"bytes": b, "flops": 6 * n}
    if c["op"] == "quant":
        n = T * c["K"]
        return {"bytes": n * (_SIZE[c["x"]] * (2 if c["swiglu"] else 1) + 1) + 4 * T, "flops": (8 if c["swiglu"] else 3) * n}
    if c["op"] == "linear":
        N, K = c["N"], c["K"]
        b = T * K + N * K + 4 * (T + N) + T * N * _SIZE[c["y"]] * (2 if c["add"] else 1) + (4 * N if c["bias"] else 0)
        return {"bytes": b, "flops": 2 * T * N * K}
    H, E, k = c["H"], c["E"], c["k"]
    return {"bytes": T * H * _SIZE[c["x"]] + 4 * E * H + 4 * E + 4 * T * k * 4 + 4 * (E + 1), "flops": 2 * T * H * E}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "norm":
        d = s["x"].double()
        total = None
        if s["res"] is not None:
            total = (d + s["res"].double()).to(s["res"].dtype).double()   # the sum as it is kept
            d = total
        v = d / (d.pow(2).sum(-1, keepdim=True) / c["H"] + s["eps"]).pow(0.5) * s["g"].double()
        vals, scale = _exact_codes(v) if c["q"] else (None, None)
        return [total, v, vals, scale]
    if c["op"] == "quant":
        d = s["x"].double()
        if c["swiglu"]:
            gate, up = d.split(c["K"], dim=1)
            d = gate * torch.special.expit(gate) * up
        return list(_exact_codes(d))
    if c["op"] == "linear":
        xd = s["x"].double() * s["xs"].double().unsqueeze(1)
        wd = s["w"].double() * s["ws"].double().unsqueeze(1)
        y = torch.mm(xd, wd.t())
        for more in (s["bias"], s["add"]):
            y = y if more is None else y + more.double()
        return [y]
    # the chosen experts from pairwise comparison counts, a block of tokens at a time
    E, k, G, size = c["E"], c["k"], c["groups"], c["E"] // c["groups"]
    rank_of = lambda v: ((v[:, None, :] > v[:, :, None]) | ((v[:, None, :] == v[:, :, None]) & _below(v.shape[1]))).sum(2)  # noqa: E731
    idx, w = [], []
    for t in range(0, c["T"], 256):
        l = torch.mm(s["x"][t:t + 256].double(), s["w"].double().t())
        p = torch.special.expit(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
        v = p + s["bias"].double()
        if c["keep"] < G:
            of = v.reshape(-1, G, size)
            top = of.amax(2)
            if size > 1:
                first = of.argmax(2, keepdim=True)
                top = top + of.scatter(2, first, -math.inf).amax(2)
            v = torch.where((rank_of(top) < c["keep"]).repeat_interleave(size, 1), v, torch.full_like(v, -math.inf))
        rank = rank_of(v)
        at = torch.argsort(rank, dim=1)[:, :k]
        part = p.gather(1, at)
        w.append(part / part.sum(1, keepdim=True) * s["scale"] if c["renorm"] else part * s["scale"])
        idx.append(at)
    return [torch.cat(idx).int(), torch.cat(w), None, None, None]


def _below(n):
    return torch.ones((n, n), dtype=torch.bool, device="cuda").tril(-1)


def _exact_codes(v):
    scale = v.abs().amax(-1, keepdim=True) / 127
    return torch.where(scale > 0, torch.round(v / scale) * scale, torch.zeros_like(v)), scale.squeeze(-1)
