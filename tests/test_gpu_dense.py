"""The operators around the routed experts against 64-bit implementations.

Tolerances count roundings: one to type t is off by at most h(t) =
finfo(t).eps / 2 relative to its value (fp32 2^-24, bf16 2^-8).
"""
import numpy as np
import pytest
import torch

import bit_quantized_routed_amd as M
from gpu_common import need_gpu

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
H24 = 2.0 ** -24


def h(t):
    return torch.finfo(t).eps / 2


def rnd(seed, *shape, std=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def strided(t, pad, off=0):
    """t on the GPU as a view of rows `pad` elements longer, starting `off` elements in."""
    base = torch.full((t.shape[0], t.shape[1] + pad + off), 77, dtype=t.dtype, device="cuda")
    v = base[:, off:off + t.shape[1]]
    v.copy_(t)
    return v


def say(*a):
    print("[dense]", *a, flush=True)


# ------------------------------------------------------------------ rows to int8
def check_codes(v, q, qs, more):
    """Codes and scales of rows whose exact values are v (fp64), computed within `more` relative."""
    amax = v.abs().amax(1)
    scale = amax / 127
    qs, q = qs.double().cpu(), q.double().cpu()
    assert torch.all((qs - scale).abs() <= (more + 2 * H24) * scale)
    # v * (127 / amax): the value, amax, and two operations, then rint
    at = v * torch.where(amax > 0, 127 / amax, 0.0)[:, None]
    assert torch.all((q - at).abs() <= 0.5 + 127 * (2 * more + 3 * H24))
    assert q.abs().max() <= 127


NORM_CASES = [  # T, H, x, residual, out, codes, row padding, offset
    (1, 7168, F32, BF16, BF16, True, 0, 0),
    (3, 1, F32, None, F32, True, 0, 0),
    (5, 7, BF16, BF16, F32, True, 0, 0),
    (2, 64, F32, F32, F32, False, 0, 0),
    (33, 513, F32, BF16, BF16, True, 3, 1),
    (17, 1112, BF16, F32, F32, True, 0, 0),
    (65, 1024, BF16, None, BF16, True, 8, 8),
    (9, 2048, F32, F32, None, True, 0, 0),
    (300, 7168, F32, BF16, BF16, True, 16, 8),
    (4, 8192, BF16, BF16, BF16, True, 8, 4),
    (2, 16384, F32, BF16, F32, True, 0, 0),
    (2, 30001, BF16, BF16, F32, True, 0, 0),
    (3, 65536, F32, None, BF16, True, 0, 0),
]


@pytest.mark.parametrize("T,H,xt,rt,ot,codes,pad,off", NORM_CASES)
def test_residual_norm(T, H, xt, rt, ot, codes, pad, off):
    need_gpu()
    say("norm", T, H, xt, rt, ot, codes, pad, off)
    x, g = rnd(1, T, H, std=0.5, dtype=xt), 1 + rnd(2, H, std=0.2)
    res = None if rt is None else rnd(3, T, H, std=2.0, dtype=rt)
    xd, rd = strided(x, pad, off), None if res is None else strided(res, pad, off)
    n = M.NormWeights(g.cuda(), 1e-5)
    for inplace in (False, True) if rd is not None else (False,):
        total = None if rd is None else rd if inplace else strided(torch.zeros_like(res), pad, off)
        out = None if ot is None else strided(torch.zeros((T, H), dtype=ot), pad, off)
        q, qs = (strided(torch.zeros((T, H), dtype=torch.int8), pad, off), torch.zeros(T, device="cuda")) if codes else (None, None)
        M.residual_norm(n, xd, rd, total, out, q, qs)
        torch.cuda.synchronize()
        s = x.float()
        if res is not None:
            s = (s + res.float()).to(rt)
            assert torch.equal(total.cpu(), s)
        s = s.double()
        v = s / torch.sqrt((s * s).mean(1, keepdim=True) + float(np.float32(1e-5))) * g.double()
        # r, s * r and (s * r) * g round to fp32 (and fp64's roundings, far below)
        more = 3.01 * H24
        if out is not None:
            assert torch.all((out.double().cpu() - v).abs() <= (more + (h(ot) if ot != F32 else 0)) * 1.01 * v.abs() + 1e-37)
        if codes:
            check_codes(v, q, qs, more)
        for view in (total, out, q):
            if view is not None and pad:            # nothing outside the columns
                base = view._base if view._base is not None else view
                assert torch.all(base[:, off + H:] == 77) and torch.all(base[:, :off] == 77)


def test_norm_odd_rows():
    """Zero rows, tiny and huge rows, and rows that hold an infinity or a NaN."""
    need_gpu()
    say("norm odd rows")
    H = 264
    x = rnd(5, 8, H)
    x[1] = 0
    x[2] *= 1e-30
    x[3] *= 1e30
    x[4, 7] = float("inf")
    x[5, 9] = float("nan")
    x[6] = 0
    x[6, 263] = -3.0
    n = M.NormWeights(torch.ones(H, device="cuda"), 0.0)
    out, q, qs = torch.empty((8, H), device="cuda"), M.empty_i8(8, H), torch.empty(8, device="cuda")
    M.residual_norm(n, x.cuda(), out=out, q=q, q_scale=qs)
    torch.cuda.synchronize()
    out, q, qs = out.cpu(), q.cpu(), qs.cpu()
    fine = [0, 2, 3, 6]
    d = x[fine].double()
    v = d / torch.sqrt((d * d).mean(1, keepdim=True))
    assert torch.all((out[fine].double() - v).abs() <= 3.02 * H24 * v.abs())
    check_codes(v, q[fine], qs[fine], 3.01 * H24)
    # eps = 0: a zero row is 0 * inf = NaN, as the formula says; its codes are marked
    for r in (1, 4, 5):
        assert torch.isnan(qs[r]) and torch.all(q[r] == 0)
    assert torch.isnan(out[4, 7]) and torch.isnan(out[5]).all()
    n = M.NormWeights(torch.ones(H, device="cuda"), 1e-6)
    M.residual_norm(n, x.cuda(), out=torch.empty((8, H), device="cuda"), q=(q2 := M.empty_i8(8, H)), q_scale=(s2 := torch.empty(8, device="cuda")))
    assert float(s2[1]) == 0 and int(q2[1].abs().max()) == 0


@pytest.mark.parametrize("T,K,xt,swiglu,pad,off", [
    (1, 2048, F32, True, 0, 0), (1, 1, F32, False, 0, 0), (7, 33, BF16, True, 0, 0), (5, 130, F32, True, 2, 1),
    (64, 2048, BF16, True, 0, 0), (33, 4096, BF16, False, 8, 8), (3, 7168, F32, False, 0, 0), (2, 65536, BF16, True, 0, 0),
    (257, 1000, BF16, True, 0, 0), (9, 9001, F32, False, 0, 0)])
def test_quant_i8(T, K, xt, swiglu, pad, off):
    need_gpu()
    say("quant", T, K, xt, swiglu, pad, off)
    x = rnd(11, T, K * (2 if swiglu else 1), dtype=xt)
    if T > 2:
        x[1] = 0
        x[2, 0] = -60.0
    q, qs = strided(torch.zeros((T, K), dtype=torch.int8), pad, off), torch.zeros(T, device="cuda")
    M.quant_i8(strided(x, pad, off), q, qs, swiglu)
    torch.cuda.synchronize()
    d = x.double()
    if swiglu:
        a, b = d[:, :K], d[:, K:]
        d = a / (1 + torch.exp(-a)) * b
    # exp to two units in the last place (4 halves), and a sum, a quotient and a product
    check_codes(d, q, qs, 7.01 * H24 if swiglu else 0.0)
    if pad:
        assert torch.all(q._base[:, off + K:] == 77) and torch.all(q._base[:, :off] == 77)


def test_quant_marks_rows_that_are_not_finite():
    need_gpu()
    say("quant marks")
    x = rnd(12, 6, 200)
    x[1, 3], x[2, 199], x[3, 0] = float("inf"), float("nan"), -float("inf")
    x[4] = 2.0 ** -120
    q, qs = M.empty_i8(6, 200), torch.empty(6, device="cuda")
    M.quant_i8(x.cuda(), q, qs)
    qs = qs.cpu()
    assert torch.isnan(qs[1:4]).all() and int(q[1:5].abs().max()) == 0 and float(qs[4]) == 0
    check_codes(x[[0, 5]].double(), q.cpu()[[0, 5]], qs[[0, 5]], 0.0)


# ------------------------------------------------------------------ int8 linear
def codes(seed, rows, K, pad=0, extreme=False):
    """int8 rows at a stride of a multiple of 16, garbage behind the columns."""
    g = torch.Generator().manual_seed(seed)
    base = torch.randint(-128, 128, (rows, (K + 15) // 16 * 16 + 16 * pad), generator=g, dtype=torch.int8)
    if extreme:
        base[:] = -128
    return base.cuda()[:, :K]


def check_linear(x, xs, w, ws, bias, add, y):
    p = (x.cpu().double() @ w.cpu().double().t())              # exact: below 2^53
    p = p * xs.cpu().double()[:, None] * ws.cpu().double()[None, :]
    b = 0 * p if bias is None else bias.cpu().double().expand_as(p)
    a = 0 * p if add is None else add.cpu().double()
    # the sum to fp32, the scales' product and their product; then each addition
    tol = H24 * (3.01 * p.abs() + (0 if bias is None else 1.01) * (p + b).abs() + (0 if add is None else 1.01) * (p + b + a).abs())
    t = y.dtype
    ref = p + b + a
    tol = tol + (h(t) * 1.001 * (ref.abs() + tol) if t != F32 else 0) + 1e-38
    err = (y.cpu().double() - ref).abs()
    assert torch.all(err <= tol), float((err / tol).max())


LINEAR_CASES = [  # T, N, K, y, bias, add, padding of y
    (1, 1, 1, F32, False, False, 0), (1, 4096, 7168, F32, False, False, 0), (2, 17, 15, BF16, True, True, 0),
    (1, 100, 8192, F32, True, False, 3), (3, 7168, 2048, F32, False, True, 0), (4, 33, 16, F32, True, False, 0),
    (7, 256, 4097, BF16, True, True, 8), (15, 1000, 300, BF16, False, False, 0), (16, 512, 1024, F32, False, True, 0),
    (17, 4096, 640, F32, True, False, 0), (32, 7168, 2048, F32, False, True, 0), (33, 65, 65, BF16, False, True, 5),
    (47, 128, 128, F32, False, False, 0), (64, 2048, 7168, BF16, False, False, 0), (65, 96, 1111, F32, True, True, 1),
    (100, 1003, 513, BF16, True, False, 0), (127, 64, 70000, F32, False, False, 0), (128, 300, 256, F32, False, False, 4),
    (129, 257, 129, BF16, True, True, 0), (255, 512, 2048, BF16, False, False, 0), (333, 1003, 1111, BF16, True, False, 0),
    (512, 4096, 1024, BF16, False, True, 0), (1000, 770, 2000, F32, True, True, 2), (1023, 1025, 384, BF16, False, False, 0),
    (2048, 2048, 2048, BF16, False, False, 0), (2100, 1100, 1400, F32, False, True, 0), (4097, 300, 272, BF16, True, False, 0),
]


@pytest.mark.parametrize("T,N,K,yt,bias,add,pad", LINEAR_CASES)
def test_linear_i8(T, N, K, yt, bias, add, pad):
    need_gpu()
    say("linear", T, N, K, yt, bias, add, pad)
    x, w = codes(21, T, K, pad=T % 2), codes(22, N, K, pad=N % 3)
    xs, ws = (rnd(23, T).abs() * 0.01).cuda(), (rnd(24, N).abs() * 0.01).cuda()
    b = rnd(25, N).cuda() if bias else None
    lin = M.LinearI8(w, ws, b)
    wk = lin.workspace(T)
    wk.fill_(0xEE)
    y = strided(torch.zeros((T, N), dtype=yt), pad)
    a = strided(rnd(26, T, N, dtype=yt), pad) if add else None
    M.linear_i8(lin, x, xs, y, a, wk)
    check_linear(x, xs, w, ws, b, a, y)
    if pad:
        assert torch.all(y._base[:, N:] == 77)
    if add:                                        # in place
        y.copy_(a)
        a2 = a.clone()
        wk.fill_(0x11)
        M.linear_i8(lin, x, xs, y, y, wk)
        check_linear(x, xs, w, ws, b, a2, y)
        if pad:
            assert torch.all(y._base[:, N:] == 77)


@pytest.mark.parametrize("T,N,K,yt,bias,add", [
    (4000, 4000, 1, F32, False, False), (4000, 4000, 100, BF16, True, False), (4000, 4000, 128, F32, False, True),
    (4000, 4000, 130, BF16, False, True), (4000, 4000, 256, BF16, True, True), (3850, 4091, 300, F32, True, False),
    (4096, 4096, 384, BF16, False, False), (4000, 4001, 513, BF16, True, True), (4096, 4096, 1024, F32, False, False),
    (2048, 7168, 1400, BF16, False, False), (8192, 4096, 640, BF16, False, False)])
def test_linear_large(T, N, K, yt, bias, add):
    """Sizes of the largest tiles, with no, one and several whole steps of K and with ragged ends; the reference is
    computed in fp64 on the device."""
    need_gpu()
    say("linear large", T, N, K, yt, bias, add)
    x, w = codes(91, T, K), codes(92, N, K)
    g = torch.Generator(device="cuda").manual_seed(93)
    xs, ws = (torch.rand(n, generator=g, device="cuda") * 0.01 for n in (T, N))
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    a = torch.randn((T, N), generator=g, device="cuda").to(yt) if add else None
    lin = M.LinearI8(w, ws, b)
    y = torch.empty((T, N), dtype=yt, device="cuda")
    M.linear_i8(lin, x, xs, y, a, lin.workspace(T))
    p = torch.mm(x.double().contiguous(), w.double().t().contiguous())
    p *= xs.double()[:, None] * ws.double()[None, :]
    s = p if b is None else p + b.double()
    ref = s if a is None else s + a.double()
    tol = H24 * (3.01 * p.abs() + (0 if b is None else 1.01) * s.abs() + (0 if a is None else 1.01) * ref.abs())
    tol += (h(yt) * 1.001 * (ref.abs() + tol) if yt != F32 else 0) + 1e-38
    assert torch.all((y.double() - ref).abs() <= tol)


@pytest.mark.parametrize("T,N", [(1, 32), (20, 40), (130, 70), (400, 300)])
def test_linear_largest_sums(T, N):
    """K = 131071 codes of -128: the sum is 2^14 * 131071, just below 2^31."""
    need_gpu()
    say("linear largest", T, N)
    K = 131071
    x, w = codes(1, T, K, extreme=True), codes(2, N, K, extreme=True)
    lin = M.LinearI8(w, torch.ones(N, device="cuda"))
    y = torch.empty((T, N), device="cuda")
    M.linear_i8(lin, x, torch.ones(T, device="cuda"), y, ws=lin.workspace(T))
    assert torch.all(y == float(np.float32(2 ** 14 * 131071)))


def test_linear_is_the_same_bits_each_time():
    need_gpu()
    say("linear repeat")
    for T, N, K in ((8, 200, 9000), (200, 200, 9000), (700, 600, 2000)):
        x, w = codes(31, T, K), codes(32, N, K)
        lin, wk = M.LinearI8(w, torch.ones(N, device="cuda")), None
        wk = lin.workspace(T)
        xs = torch.ones(T, device="cuda")
        ys = [torch.empty((T, N), device="cuda") for _ in range(3)]
        for y in ys:
            M.linear_i8(lin, x, xs, y, ws=wk)
        assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


def test_rows_far_apart():
    """Strides that put the last rows past 2^31 and 2^32 bytes."""
    need_gpu()
    say("far rows")
    far = 1_100_000_000 // 16 * 16
    base = torch.empty(5 * far, dtype=torch.int8, device="cuda")
    T, N, K, H = 5, 33, 200, 264

    def put(t, ld):
        v = torch.as_strided(base.view(t.dtype), t.shape, (ld, 1))
        v.copy_(t)
        return v

    x, w = codes(81, T, K).contiguous(), codes(82, N, K)
    xs, ws = (rnd(83, T).abs() * 0.01).cuda(), (rnd(84, N).abs() * 0.01).cuda()
    lin = M.LinearI8(w, ws)
    y = torch.empty((T, N), device="cuda")
    M.linear_i8(lin, put(x, far), xs, y, None, lin.workspace(T))
    check_linear(x, xs, w, ws, None, None, y)
    lin = M.LinearI8(put(x, far), xs)              # and as weights
    M.linear_i8(lin, w, ws, yt := torch.empty((N, T), device="cuda"), None, lin.workspace(N))
    check_linear(w, ws, x, xs, None, None, yt)
    rows = rnd(85, T, H, dtype=BF16)
    q, qs = M.empty_i8(T, H), torch.empty(T, device="cuda")
    M.quant_i8(put(rows.cuda(), far // 2), q, qs)
    check_codes(rows.double(), q, qs, 0.0)
    out = torch.empty((T, H), device="cuda")
    M.residual_norm(M.NormWeights(torch.ones(H, device="cuda"), 0.0), put(rows.cuda(), far // 2), out=out)
    d = rows.double()
    v = d / torch.sqrt((d * d).mean(1, keepdim=True))
    assert torch.all((out.double().cpu() - v).abs() <= 3.02 * H24 * v.abs())
    xr = rnd(86, T, 64, dtype=BF16)
    r = M.RouterWeights(rnd(87, 8, 64, std=0.125).cuda(), 2)
    a, b = M.Routing(T, 2, 8), M.Routing(T, 2, 8)
    M.route_scored(r, put(xr.cuda(), far // 2), a, r.workspace(T))
    M.route_scored(r, xr.cuda(), b, r.workspace(T))
    assert torch.equal(a.topk_idx, b.topk_idx) and torch.equal(a.topk_w, b.topk_w)


# ------------------------------------------------------------------ scored routing
def plain_route(x, w, k, score, bias, groups, keep, renorm, scale):
    """fp64, one token at a time."""
    l = x.astype(np.float64) @ w.astype(np.float64).T
    T, E = l.shape
    idx, wt = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        lt = np.where(np.isnan(l[t]), -np.inf, l[t])
        with np.errstate(over="ignore", invalid="ignore"):
            if score == "sigmoid":
                p = 1 / (1 + np.exp(-lt))
            else:
                top = lt.max()
                p = np.where(lt == -np.inf, 0.0, np.where(lt == top, 1.0, np.exp(lt - top)))
                p = p / p.sum() if p.sum() > 0 else p
        c = p + (0 if bias is None else bias.astype(np.float64))
        c = np.where(np.isnan(l[t]), -np.inf, c)
        if keep < groups:
            of = np.sort(c.reshape(groups, -1), axis=1)[:, ::-1]
            gs = of[:, :2].sum(1)
            kept = np.argsort(-gs, kind="stable")[:keep]
            ok = np.zeros(groups, bool)
            ok[kept] = True
            c = np.where(np.repeat(ok, E // groups), c, -np.inf)
        at = np.argsort(-c, kind="stable")[:k]
        pw = np.where(c[at] == -np.inf, 0.0, p[at])
        if renorm:
            pw = pw / pw.sum() if pw.sum() > 0 else pw
        idx[t], wt[t] = at, pw * float(np.float32(scale))
    return idx, wt


def check_route(T, H, E, k, xt, score, bias, groups, keep, renorm, seed=41, x=None, w=None, pad=0):
    x = rnd(seed, T, H, dtype=xt) if x is None else x
    w = rnd(seed + 1, E, H, std=H ** -0.5) if w is None else w
    b = None if bias is None else bias if isinstance(bias, torch.Tensor) else rnd(seed + 2, E, std=bias)
    R = M.RouterWeights(w.cuda(), k, score, None if b is None else b.cuda(), groups, keep, renorm, 2.5)
    r, ws = M.Routing(T, k, E), R.workspace(T)
    ws.fill_(0xFF)
    M.route_scored(R, strided(x, pad), r, ws)
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        idx, wt = plain_route(x.float().numpy(), w.numpy(), k, score, None if b is None else b.numpy(), groups, keep, renorm, 2.5)
    got = r.topk_idx.cpu().numpy()
    assert np.array_equal(got, idx)
    # A weight is a smooth function of the logits, |d ln p / d l| <= 1 (sigmoid) or <= 2 times the largest logit's
    # (softmax), once more through the sum of the weights; a logit is off by at most 2^-20 |x| |w_e| (fp32 sums of
    # short stretches where many tokens share the matrix instructions).  One rounding to fp32 at the end.
    xn = np.linalg.norm(np.nan_to_num(x.double().numpy(), posinf=0, neginf=0), axis=1, keepdims=True)
    d = 2.0 ** -20 * xn * np.linalg.norm(w.numpy(), axis=1).max()
    gw = r.topk_w.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(gw - wt) <= wt * (1.01 * H24 + 4 * d) + 1e-44)
    flat = got.reshape(-1)
    perm = np.argsort(flat, kind="stable")
    assert np.array_equal(r.perm.cpu().numpy(), perm)
    inv = np.empty_like(perm)
    inv[perm] = np.arange(T * k)
    assert np.array_equal(r.inv.cpu().numpy(), inv)
    assert np.array_equal(r.offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))]))
    return r, wt


ROUTE_CASES = [  # T, H, E, k, x, score, bias, groups, keep, renorm, padding
    (1, 7168, 256, 8, BF16, "sigmoid", 0.05, 8, 4, True, 0), (1, 8, 1, 1, F32, "softmax", None, 1, 1, True, 0),
    (1, 512, 1024, 64, BF16, "softmax", 0.001, 16, 5, False, 0), (2, 64, 6, 3, F32, "sigmoid", None, 3, 2, False, 0),
    (5, 1112, 160, 6, F32, "softmax", 0.001, 8, 3, True, 8), (32, 7168, 256, 8, BF16, "sigmoid", 0.05, 8, 4, True, 0),
    (63, 128, 64, 8, BF16, "sigmoid", 0.1, 64, 8, True, 0), (64, 264, 100, 7, F32, "softmax", None, 1, 1, False, 0),
    (65, 264, 100, 7, BF16, "sigmoid", 0.05, 1, 1, False, 8), (100, 1024, 256, 8, BF16, "sigmoid", None, 8, 4, True, 16),
    (130, 72, 32, 4, F32, "sigmoid", 0.05, 4, 2, True, 0), (333, 1112, 160, 6, F32, "softmax", 0.001, 1, 1, False, 0),
    (500, 2048, 512, 10, BF16, "sigmoid", 0.02, 32, 8, True, 0), (257, 512, 1000, 16, BF16, "sigmoid", 0.02, 10, 9, True, 0),
    (1025, 1024, 256, 8, BF16, "softmax", None, 8, 4, True, 0), (2048, 7168, 256, 8, BF16, "sigmoid", 0.05, 8, 4, True, 0),
    (3000, 256, 128, 8, BF16, "sigmoid", 0.05, 1, 1, True, 0), (700, 7168, 256, 8, BF16, "sigmoid", 0.05, 8, 4, True, 8),
    (1300, 1112, 160, 64, BF16, "sigmoid", 0.05, 4, 3, False, 0), (4200, 520, 40, 5, BF16, "sigmoid", None, 20, 7, True, 0),
    (2600, 8, 64, 3, BF16, "sigmoid", 0.01, 16, 2, True, 0), (200, 4096, 1024, 8, BF16, "sigmoid", 0.02, 64, 60, True, 0),
]


@pytest.mark.parametrize("T,H,E,k,xt,score,bias,groups,keep,renorm,pad", ROUTE_CASES)
def test_route_scored(T, H, E, k, xt, score, bias, groups, keep, renorm, pad):
    need_gpu()
    say("route", T, H, E, k, xt, score, bias, groups, keep, renorm, pad)
    check_route(T, H, E, k, xt, score, bias, groups, keep, renorm, pad=pad)


@pytest.mark.parametrize("T", [1, 3, 40, 200, 2700])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_ties(T, score):
    """Equal router rows give equal scores: the lower expert and the lower group win."""
    need_gpu()
    say("route ties", T, score)
    H, E = 128, 64
    w = rnd(51, 8, H, std=H ** -0.5).repeat(E // 8, 1)
    check_route(T, H, E, 8, BF16, score, None, 8, 4, True, x=rnd(52, T, H, dtype=BF16), w=w)
    check_route(T, H, E, 8, BF16, score, None, 1, 1, True, x=torch.zeros((T, H), dtype=BF16), w=w)


@pytest.mark.parametrize("T", [70, 1500])
def test_route_near_ties(T):
    """Rows one unit in the last place apart: scores that only 64 bits tell apart."""
    need_gpu()
    say("route near ties", T)
    H, E = 1024, 128
    w = rnd(53, E, H, std=H ** -0.5)
    for e in range(1, E, 2):                       # odd rows follow the even ones, a few values nudged
        w[e] = w[e - 1]
        w[e, e] = torch.nextafter(w[e, e], torch.tensor(10.0))
    for groups, keep in ((1, 1), (8, 4)):
        check_route(T, H, E, 8, BF16, "sigmoid", None, groups, keep, True, x=rnd(54, T, H, dtype=BF16), w=w)


@pytest.mark.parametrize("T", [80, 2000, 2700])
def test_route_scores_on_the_border(T):
    """Biases that bring every expert's selection value to within 1e-7 of 1 for one token's scores, so that the order
    turns on bits that fp32 sums do not have; groups as close."""
    need_gpu()
    say("route border", T)
    H, E = 7168, 64
    w = rnd(58, E, H, std=H ** -0.5)
    x = rnd(59, 1, H, dtype=BF16)
    p = 1 / (1 + np.exp(-(x.double().numpy() @ w.double().numpy().T)))[0]
    bias = torch.from_numpy((1.0 - p + np.random.default_rng(3).uniform(-1e-7, 1e-7, E)).astype(np.float32))
    xs = x.repeat(T, 1)
    xs[1::2] = rnd(60, T // 2, H, dtype=BF16)
    for groups, keep in ((1, 1), (8, 4)):
        check_route(T, H, E, 8, BF16, "sigmoid", bias, groups, keep, True, x=xs, w=w)


@pytest.mark.parametrize("T,std", [(3000, 60.0), (3000, 1e-4), (2800, 1e30), (60, 60.0)])
def test_route_large_and_small_logits(T, std):
    """Logits far from the sigmoid's slope on both sides, with saturated scores that tie, and nearly equal ones."""
    need_gpu()
    say("route scale", T, std)
    x = rnd(63, T, 128, std=std, dtype=BF16)
    for groups, keep in ((1, 1), (8, 4)):
        check_route(T, 128, 64, 8, BF16, "sigmoid", None, groups, keep, False, x=x)
    check_route(T, 128, 64, 64, BF16, "sigmoid", 0.05, 1, 1, True, x=x)


@pytest.mark.parametrize("T", [1, 5, 300, 5300])
def test_route_masked_experts(T):
    """Experts masked by a bias of -inf, down to fewer than k and to none; NaN rows of x; very large scores."""
    need_gpu()
    say("route masks", T)
    H, E, k = 128, 32, 4
    inf = float("inf")
    for left in (20, 3, 0):
        bias = torch.zeros(E)
        bias[left:] = -inf
        for groups, keep in ((1, 1), (8, 4)):
            for score in ("sigmoid", "softmax"):
                r, wt = check_route(T, H, E, k, BF16, score, bias, groups, keep, True, x=rnd(55, T, H, dtype=BF16))
                assert np.isfinite(r.topk_w.cpu().numpy()).all()
    x = rnd(56, T, H, dtype=BF16)
    x[0, 5] = float("nan")
    for score in ("sigmoid", "softmax"):
        r, _ = check_route(T, H, E, k, BF16, score, None, 1, 1, True, x=x)
        assert torch.all(r.topk_w[0] == 0) and r.topk_idx[0].tolist() == [0, 1, 2, 3]
        check_route(T, H, E, k, F32, score, None, 4, 2, False, x=rnd(57, T, H) * 3000)


# ------------------------------------------------------------------ streams, graphs, profiles
def _block(seed=61, T=48, H=512, I=256, E=32):
    """Everything of one step on the device, and the calls that make it."""
    x, res = rnd(seed, T, H).cuda(), rnd(seed + 1, T, H, dtype=BF16).cuda()
    n = M.NormWeights((1 + rnd(seed + 2, H, std=0.1)).cuda())
    up = M.LinearI8.quantize(rnd(seed + 3, 2 * I, H, std=0.05).cuda())
    down = M.LinearI8.quantize(rnd(seed + 4, H, I, std=0.05, dtype=BF16).cuda())
    R = M.RouterWeights(rnd(seed + 5, E, H, std=H ** -0.5).cuda(), 4, "sigmoid", rnd(seed + 6, E, std=0.05).cuda(), 4, 2)
    b = dict(out=torch.empty((T, H), dtype=BF16, device="cuda"), q=M.empty_i8(T, H), qs=torch.empty(T, device="cuda"),
             gu=torch.empty((T, 2 * I), device="cuda"), hq=M.empty_i8(T, I), hs=torch.empty(T, device="cuda"),
             y=torch.empty((T, H), device="cuda"), total=torch.empty_like(res), r=M.Routing(T, 4, E))
    w1, w2, w3 = up.workspace(T), down.workspace(T), R.workspace(T)

    def step(stream=None):
        M.residual_norm(n, x, res, b["total"], b["out"], b["q"], b["qs"], stream)
        M.route_scored(R, b["out"], b["r"], w3, stream)
        M.linear_i8(up, b["q"], b["qs"], b["gu"], None, w1, stream)
        M.quant_i8(b["gu"], b["hq"], b["hs"], True, stream)
        M.linear_i8(down, b["hq"], b["hs"], b["y"], x, w2, stream)

    def outputs():
        torch.cuda.synchronize()
        return [t.clone() for t in (b["total"], b["out"], b["q"], b["qs"], b["gu"], b["hq"], b["y"], b["r"].topk_idx,
                                    b["r"].topk_w, b["r"].offsets, b["r"].perm, b["r"].inv)]

    def clear():
        for t in b.values():
            for u in ([t.topk_idx, t.topk_w, t.offsets, t.perm, t.inv] if isinstance(t, M.Routing) else [t]):
                u.zero_()
        torch.cuda.synchronize()
    return step, outputs, clear


@pytest.mark.parametrize("T", [1, 48, 200])
def test_graph_and_streams(T):
    need_gpu()
    say("graph", T)
    step, outputs, clear = _block(T=T)
    step()
    want = outputs()
    side = torch.cuda.Stream()
    clear()
    step(side)
    assert all(torch.equal(a, b) for a, b in zip(want, outputs()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        clear()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, outputs()))
        clear()
        step()
        assert all(torch.equal(a, b) for a, b in zip(want, outputs()))


def test_profile_names():
    need_gpu()
    say("profile")
    T, N, K = 16, 64, 256
    lin = M.LinearI8(codes(1, N, K), torch.ones(N, device="cuda"))
    y = torch.empty((T, N), device="cuda")
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record(), b.record()
    prof = M.Profile(0, 0, a.cuda_event, b.cuda_event, None)
    M.linear_i8(lin, codes(2, T, K), torch.ones(T, device="cuda"), y, ws=lin.workspace(T), prof=prof)
    torch.cuda.synchronize()
    assert prof.name == b"linear_i8" and prof.n_launches >= 1 and a.elapsed_time(b) > 0


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("T", [5000, 4096, 1400])
def test_route_few_experts_many_tokens(T):
    need_gpu()
    say("route few experts", T)
    check_route(T, 64, 3, 2, BF16, "sigmoid", None, 1, 1, True)
    check_route(T, 64, 1, 1, F32, "softmax", None, 1, 1, True)


@pytest.mark.parametrize("T", [1, 32, 200])
def test_moe_block(T):
    """The block of bit_quantized_routed_amd.block: its routing from its own norm, the routed experts against the
    oracle, the shared expert from its codes."""
    import os
    import sys
    need_gpu()
    say("block", T)
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_block as B
    import synthetic as S
    from gpu_common import oracle_experts, rel_l2
    from oracle import moe_ref as R
    H, I, E = 512, 256, 16
    block, gate_up, down = B.make(H, I, E)
    b = B.BlockBuffers(block, T)
    x, res = rnd(71, T, H).cuda(), rnd(72, T, H, dtype=BF16).cuda()
    before = res.clone()
    y = block(x, res, b)
    torch.cuda.synchronize()
    assert torch.equal(res, (x + before.float()).bfloat16())
    n = b.n.float().cpu().numpy()
    idx, w = plain_route(n, block.router.w_router.cpu().numpy(), 4, "sigmoid", block.router.bias.cpu().numpy(), 4, 2, True, 2.5)
    assert np.array_equal(b.routing.topk_idx.cpu().numpy(), idx)
    cfg = dict(hidden=H, inter=I, n_experts=E, top_k=4, fmt_gate_up=S.FMT_CB2, fmt_down=S.FMT_Q2K, sh_inter=0, seed=0)
    want = R.moe_layer(n, idx, w, oracle_experts(cfg, range(E)), None)
    d = lambda t: t.double().cpu()                                     # noqa: E731
    (wu, su, _), (wd, sd, _) = block.gate_up.tensors, block.down.tensors
    gu = (d(b.q) * d(b.q_scale)[:, None]) @ (d(wu) * d(su)[:, None]).t()
    # gate and up to fp32 (3 roundings), then silu: the codes as in test_quant_i8 on top
    assert rel_l2(b.gate_up.cpu(), gu) < 4 * H24
    check_codes(d(b.gate_up)[:, :I] * torch.sigmoid(d(b.gate_up)[:, :I]) * d(b.gate_up)[:, I:], b.h, b.h_scale, 7.01 * H24)
    want = want + ((d(b.h) * d(b.h_scale)[:, None]) @ (d(wd) * d(sd)[:, None]).t()).numpy()
    assert rel_l2(y.cpu(), want) < (1e-4 if T <= 64 else 5e-3)


def test_moe_block_example():
    import os
    import sys
    need_gpu()
    say("block example")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_block as B
    # three quantizations to 8 bits (x, h and the weights): about 1% in all, far below 5%
    assert B.main(["--tokens", "20", "--hidden", "512", "--inter", "256"]) < 0.05


def test_moe_block_refusals():
    import os
    import sys
    need_gpu()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_block as B
    block, _, _ = B.make(512, 256, 16)
    with pytest.raises(ValueError):
        B.MoeBlock(block.norm, block.router, block.layer, block.down, block.gate_up)
