"""The operators around the routed experts at the edges of what they take.

Tolerances count roundings: one to fp32 is off by at most 2^-24 relative to its value.
"""
import numpy as np
import pytest
import torch

import bit_quantized_routed_amd as M
from gpu_common import need_gpu
from test_gpu_dense import BF16, F32, H24, check_route, plain_route, rnd

pytestmark = pytest.mark.gpu


def say(*a):
    print("[dense]", *a, flush=True)


# ------------------------------------------------------------------ scored routing
@pytest.mark.parametrize("T,E,k,groups,keep", [(5300, 64, 8, 8, 4), (5300, 256, 8, 1, 1), (2600, 128, 8, 16, 3)])
def test_route_open_tokens_one_after_another(T, E, k, groups, keep):
    """More open tokens than work-groups, where a token's groups, its slots, or more experts than slots hold are too
    close: a work-group's waves settle one set of experts after the other in the same LDS."""
    need_gpu()
    say("route open", T, E, k, groups, keep)
    H = 512
    w = rnd(101, E, H, std=H ** -0.5)
    x = rnd(102, 1, H, dtype=BF16)
    p = 1 / (1 + np.exp(-(x.double().numpy() @ w.double().numpy().T)))[0]
    bias = torch.from_numpy((1.0 - p + np.random.default_rng(4).uniform(-1e-7, 1e-7, E)).astype(np.float32))
    xs = x.repeat(T, 1)
    xs[2::3] = rnd(103, len(xs[2::3]), H, dtype=BF16)
    for _ in range(3):
        check_route(T, H, E, k, BF16, "sigmoid", bias, groups, keep, True, x=xs, w=w)


def uneven_sums(sign, rng):
    """x (bf16 values) and w of 128 of H whose sum of about `sign` the bf16 matrix instruction gets 33 units of 2^-24 too
    large, where |x| |w| is 1.03: one product of 1, seven beside it that fall just short of what its group of 8 keeps,
    and group sums an odd multiple of half a last place (and a little) away from where they are added."""
    U = 2.0 ** -24
    x, w = np.zeros(128), np.zeros(128)
    x[0], w[0] = 1.0, sign
    x[1:8] = 2.0 ** -12 * (1 - 2.0 ** -8)
    w[1:8] = -x[1:8]
    second = 2.0 ** -15 * (1 + np.arange(128) / 128)
    for g in range(1, 16):
        for a in rng.permutation(2.0 ** -5 * (1 + (2 * np.arange(64) + 1) / 128)):
            fit = second[np.abs((sign * second * a / U) % 2 - 1.04) < 0.035]
            if len(fit):
                break
        # the first term's product is an odd multiple of U; the second term is there from the step on that has a sum to add to
        x[8 * g], w[8 * g] = a, sign * 2.0 ** -5 * (1 + (2 * rng.integers(0, 64) + 1) / 128)
        w[8 * g] += sign * fit[0] if g >= 4 else 0.0
        x[8 * g + 1], w[8 * g + 1] = 2.0 ** -15, 2.0 ** -14
    return x, w


def uneven_router(scale, pairs=1, w_scale=1.0):
    """(x, w) of 256 pairs + 8 of H: x w = 0, with every rounding of its parts' sums upwards."""
    rng = np.random.default_rng(1)
    parts = [uneven_sums(sign, rng) for _ in range(pairs) for sign in (1, -1)] + [(np.zeros(8), np.zeros(8))]
    x, w = (np.concatenate([p[i] for p in parts]) for i in (0, 1))
    x[-8], w[-8] = 2.0 ** -4, -16 * float(x @ w)
    x, w = torch.from_numpy(x * scale).bfloat16(), torch.from_numpy(w * w_scale).float()
    assert abs(float(x.double() @ w.double())) < 2.0 ** -24 * scale * w_scale
    return x, w


def test_route_decides_on_worst_roundings():
    """Two experts whose fp32 sums are as far off as the matrix instruction's roundings take them, in opposite directions."""
    need_gpu()
    say("route worst roundings")
    T, E = 2700, 64
    x, row = uneven_router(512.0)
    w = torch.zeros((E, 264))
    w[20], w[40] = row, -row
    p = 1 / (1 + np.exp(-np.array([1.0, -1.0]) * float(x.double() @ row.double())))
    bias = torch.full((E,), -0.25)
    bias[20] = 0.0
    bias[40] = float(np.float32(p[0] - p[1] + 1e-8))
    for k in (1, 2):
        r, _ = check_route(T, 264, E, k, BF16, "sigmoid", bias, 1, 1, True, x=x.repeat(T, 1), w=w)
        assert int(r.topk_idx[0, 0]) == 40


def weights_of(x, w, k, score, bias, groups, keep, renorm):
    E = w.shape[0]
    R = M.RouterWeights(w.cuda(), k, score, None if bias is None else bias.cuda(), groups, keep, renorm, 2.5)
    r = M.Routing(x.shape[0], k, E)
    M.route_scored(R, x.cuda(), r, R.workspace(x.shape[0]))
    idx, wt = plain_route(x.float().numpy(), w.numpy(), k, score, None if bias is None else bias.numpy(), groups, keep, renorm, 2.5)
    assert np.array_equal(r.topk_idx.cpu().numpy(), idx)
    return idx, wt, r.topk_w.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("T,H,E,xt,score,renorm", [
    (1, 7168, 256, BF16, "sigmoid", True), (17, 1112, 160, F32, "softmax", False), (128, 512, 64, BF16, "softmax", True),
    (333, 7168, 256, BF16, "sigmoid", True), (640, 264, 256, BF16, "sigmoid", False), (1500, 1112, 160, F32, "sigmoid", True),
    (2000, 512, 99, BF16, "softmax", False)])
def test_route_weights_of_fp64_logits(T, H, E, xt, score, renorm):
    """Where the logits are fp64 sums a weight is rounded once, to fp32 (and fp64's roundings: of H products of |x| |w|
    in all, through an exponent, 2^-29 of the weight at most)."""
    need_gpu()
    say("route weights", T, H, E, xt, score, renorm)
    _, wt, got = weights_of(rnd(111, T, H, dtype=xt), rnd(112, E, H, std=H ** -0.5), 6, score, None, 1, 1, renorm)
    assert np.all(np.abs(got - wt) <= wt * (H24 + 2.0 ** -29))


def split_bound(x, w, idx, H):
    """What a logit of a large batch may be off by: 2^-24 (60 + H / 128) |x| |w_e|."""
    xn = np.linalg.norm(x.double().numpy(), axis=1, keepdims=True)
    return H24 * (60 + -(-H // 128)) * xn * np.linalg.norm(w.double().numpy(), axis=1)[idx]


@pytest.mark.parametrize("T,H,E,groups", [(2048, 7168, 256, 8), (1700, 1112, 99, 1), (8192, 264, 70, 1), (3000, 2048, 250, 10)])
def test_route_weights_of_split_logits(T, H, E, groups):
    """Large batches of bf16 tokens with sigmoid scores, experts a multiple of four and not: a weight without
    renormalisation is off by what its logit is, |d ln p / d l| <= 1, and one rounding.  (Measured on random values:
    within 3.4 units of 2^-24 of the weight; those are held to 8.)"""
    need_gpu()
    say("route split weights", T, H, E, groups)
    x, w = rnd(113, T, H, dtype=BF16), rnd(114, E, H, std=H ** -0.5)
    idx, wt, got = weights_of(x, w, 8, "sigmoid", rnd(115, E, std=0.05), groups, max(1, groups // 2), False)
    off = np.abs(got - wt) / wt
    say("weights off by at most", off.max() / H24, "2^-24")
    assert np.all(off <= 1.01 * H24 + split_bound(x, w, idx, H))
    assert off.max() <= 2.0 ** -21


def test_route_split_weights_at_worst_roundings():
    need_gpu()
    say("route split weights, worst roundings")
    T, E = 2700, 64
    x, row = uneven_router(512.0)
    w = torch.zeros((E, 264))
    w[20], w[40] = row, -row
    bias = torch.full((E,), -0.5)
    bias[20], bias[40] = 1.0, 0.5                  # far apart: the weights are those of the fp32 sums
    xs = x.repeat(T, 1)
    idx, wt, got = weights_of(xs, w, 2, "sigmoid", bias, 1, 1, False)
    off, bound = np.abs(got - wt) / wt, split_bound(xs, w, idx, 264)
    say("off by", off.max(), "of", bound.max(), "in units of 2^-24 |x| |w|:", 2 * off.max() * (60 + 3) / bound.max())
    assert np.all(off <= 1.01 * H24 + bound)


@pytest.mark.parametrize("scale,w_scale", [(2.0 ** -64, 2.0 ** 60), (2.0 ** -60, 2.0 ** 60), (2.0 ** 60, 2.0 ** -64), (2.0 ** 60, 2.0 ** -68)])
def test_route_squares_below_the_smallest_float(scale, w_scale):
    """Ordinary logits of tokens (or router rows) whose elements have squares that fp32 does not hold, against large rows
    (or tokens): the worst roundings still leave the order to fp64."""
    need_gpu()
    say("route small squares", scale, w_scale)
    T, E, pairs = 2700, 64, 32
    x, row = uneven_router(scale, pairs, w_scale)
    w = torch.zeros((E, len(x)))
    w[20], w[40] = row, -row
    p = 1 / (1 + np.exp(-np.array([1.0, -1.0]) * float(x.double() @ row.double())))
    bias = torch.full((E,), -0.25)
    bias[20] = 0.0
    bias[40] = float(np.float32(p[0] - p[1] + 1e-9))
    r, _ = check_route(T, len(x), E, 1, BF16, "sigmoid", bias, 1, 1, True, x=x.repeat(T, 1), w=w)
    assert int(r.topk_idx[0, 0]) == 40


@pytest.mark.parametrize("T", [1, 100, 900, 5300])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_groups_of_one_forced_expert(T, score):
    """A group with one expert of bias +inf and all others at -inf holds fewer than two that can be chosen: its score is
    -inf, and exactly `keep` groups stay."""
    need_gpu()
    say("route forced", T, score)
    H, E, inf = 128, 64, float("inf")
    bias = rnd(131, E, std=0.01)
    bias[8:16] = -inf
    bias[11] = inf
    bias[40:48] = -inf                             # nothing left
    bias[50:56] = -inf                             # two left
    x, w = rnd(132, T, H, dtype=BF16), rnd(133, E, H, std=H ** -0.5)
    with np.errstate(invalid="ignore"):
        r, _ = check_route(T, H, E, 8, BF16, score, bias, 8, 3, True, x=x, w=w)
    group = r.topk_idx.cpu().numpy() // 8
    assert not np.isin(group, [1, 5]).any() and all(len(set(g)) <= 3 for g in group)


# ------------------------------------------------------------------ rows to int8
def exact_swiglu(x):
    a, b = x.double().chunk(2, 1)
    return a / (1 + torch.exp(-a)) * b


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("K", [64, 200, 1003])
def test_swiglu_of_large_gates(xt, K):
    """Finite gates up to the type's largest, either sign, with `up` from small to as large as the product allows."""
    need_gpu()
    say("swiglu large", xt, K)
    big = float(torch.finfo(xt).max)
    rows = [(lo, hi, up) for lo, hi, up in (
        (80.0, 90.0, 1.0), (100.0, 200.0, 1e-3), (1e4, 2e4, 1.0), (1e31, 2e31, 1.0), (1e38, 2e38, 0.25), (2.4e38, 3.3e38, 1e-5),
        (big, big, 0.125), (-85.0, -80.0, 1.0), (-89.5, -86.0, 1e20), (-95.0, -87.0, 1e30), (-130.0, -100.0, 1e35),
        (-160.0, -140.0, 1e38), (-175.0, -165.0, 1e38), (-300.0, -200.0, 1e38), (-1.1e4, -1e4, 1.0), (-2e31, -1e31, 1e30),
        (-2e38, -1e38, 1.0), (-big, -big, 1e38), (-big, -big, 1.0))]
    g = torch.Generator().manual_seed(141)
    x = torch.empty((len(rows), 2 * K), dtype=xt)
    for i, (lo, hi, up) in enumerate(rows):
        x[i, :K] = (lo + (hi - lo) * torch.rand(K, generator=g)).clamp(-big, big).to(xt)
        x[i, K:] = (torch.rand(K, generator=g) * 2 - 1).mul(up).to(xt)
    q, qs = M.empty_i8(len(rows), K), torch.empty(len(rows), device="cuda")
    M.quant_i8(x.cuda(), q, qs, True)
    v = exact_swiglu(x)
    assert v.abs().max() < 3e38
    qs, q = qs.cpu().double(), q.cpu().double()
    amax = v.abs().amax(1)
    for i, r in enumerate(rows):                   # the quantizer's rule: rows below 2^-100 are zero
        if amax[i] < 2.0 ** -100 * (1 - 2.0 ** -20):
            assert float(qs[i]) == 0 and int(q[i].abs().max()) == 0, r
        elif amax[i] > 2.0 ** -100 * (1 + 2.0 ** -20):
            # as test_quant_i8: seven half units for the value, two roundings of the scale, three of the code
            assert abs(float(qs[i]) - float(amax[i]) / 127) <= 9.01 * H24 * float(amax[i]) / 127, r
            assert float((q[i] - v[i] * (127 / amax[i])).abs().max()) <= 0.5 + 127 * (14.02 + 3) * H24, r


def test_swiglu_marks_infinite_gates():
    need_gpu()
    say("swiglu marks")
    x = rnd(142, 7, 128)
    inf, nan = float("inf"), float("nan")
    x[0, 3], x[1, 3], x[2, 3], x[3, 64 + 3], x[4, 64 + 3] = inf, -inf, nan, inf, nan
    x[5, 3], x[5, 64 + 3] = -1e38, inf             # -0 * inf
    q, qs = M.empty_i8(7, 64), torch.empty(7, device="cuda")
    M.quant_i8(x.cuda(), q, qs, True)
    assert torch.isnan(qs[:6]).all() and int(q[:6].abs().max()) == 0 and torch.isfinite(qs[6])


# ------------------------------------------------------------------ int8 linear
@pytest.mark.parametrize("T,N,K,yt,bias,add,pad", [
    (1, 4096, 1024, F32, True, False, 0), (7, 1003, 600, F32, True, True, 1), (16, 512, 512, BF16, True, True, 0),
    (32, 512, 8192, F32, True, False, 0), (40, 1003, 8192, F32, True, True, 1), (32, 7168, 2048, F32, True, True, 0),
    (333, 1003, 1111, F32, True, False, 0), (300, 512, 640, BF16, True, True, 0), (2048, 2048, 512, F32, True, False, 0),
    (2100, 1101, 700, F32, True, True, 3), (4096, 4096, 384, F32, True, False, 0), (4096, 4095, 384, F32, True, True, 0),
    (2048, 7168, 512, BF16, True, False, 0), (128, 256, 100, F32, False, True, 0)])
def test_linear_rounds_as_stated(T, N, K, yt, bias, add, pad):
    """The scales' product, the sum's product with it, the bias and the addition each round to fp32, in every kernel:
    the same bits as these operations one after another."""
    need_gpu()
    say("linear bits", T, N, K, yt, bias, add, pad)
    g = torch.Generator(device="cuda").manual_seed(151)

    def codes(rows):
        return torch.randint(-128, 128, (rows, (K + 15) // 16 * 16), generator=g, device="cuda", dtype=torch.int8)[:, :K]

    x, w = codes(T), codes(N)
    xs, ws = (torch.rand(n, generator=g, device="cuda") * 0.01 for n in (T, N))
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    a = torch.randn((T, N), generator=g, device="cuda").to(yt) if add else None
    lin = M.LinearI8(w, ws, b)
    y = torch.empty((T, N + pad), dtype=yt, device="cuda")[:, :N]
    M.linear_i8(lin, x, xs, y, a, lin.workspace(T))
    v = torch.mm(x.double().contiguous(), w.double().t().contiguous()).float() * (xs[:, None] * ws[None, :])
    if bias:
        v = v + b
    if add:
        v = v + a.float()
    assert torch.equal(y, v.to(yt))


# ------------------------------------------------------------------ one workspace for all batches
def test_linear_workspace_of_the_largest_batch():
    need_gpu()
    say("linear workspace")
    N, K, most = 256, 7168, 2000
    g = torch.Generator(device="cuda").manual_seed(161)
    x, w = (torch.randint(-128, 128, (n, K), generator=g, device="cuda", dtype=torch.int8) for n in (most, N))
    lin = M.LinearI8(w, torch.ones(N, device="cuda"))
    ws, ones = lin.workspace(most), torch.ones(most, device="cuda")
    want = torch.mm(x.double(), w.double().t().contiguous())
    for T in (1, 17, 32, 64, 100, 300, 512, 1000, 1999, 2000):
        ws.fill_(0x55)
        y = torch.empty((T, N), device="cuda")
        M.linear_i8(lin, x[:T], ones[:T], y, ws=ws)
        assert torch.equal(y, want[:T].float()), T


@pytest.mark.parametrize("xt,score", [(BF16, "sigmoid"), (F32, "sigmoid"), (BF16, "softmax")])
def test_router_workspace_of_the_largest_batch(xt, score):
    need_gpu()
    say("router workspace", xt, score)
    H, E, k, most = 512, 256, 4, 4200
    x, w = rnd(171, most, H, dtype=xt), rnd(172, E, H, std=H ** -0.5)
    R = M.RouterWeights(w.cuda(), k, score)
    ws, xd = R.workspace(most), x.cuda()
    idx, _ = plain_route(x.float().numpy(), w.numpy(), k, score, None, 1, 1, True, 1.0)
    for T in (1, 128, 129, 320, 640, 641, 1152, 1153, 1984, 2688, 4033, 4200):
        ws.fill_(0x55)
        r = M.Routing(T, k, E)
        M.route_scored(R, xd[:T], r, ws)
        assert np.array_equal(r.topk_idx.cpu().numpy(), idx[:T]), T
