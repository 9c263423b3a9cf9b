"""The operators for a few tokens of many requests against 64 bits: the MoE block in two kernels, the plan of a batch's
adapters, and low-rank adapters beside a projection.

Tolerances count roundings: one to type t is off by at most finfo(t).eps / 2 relative to its value (fp32 2^-24, bf16 2^-8).
"""
import numpy as np
import pytest
import torch

import bit_quantized_routed_amd as M
from gpu_common import need_gpu
from test_gpu_dense import plain_route, rnd, strided

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
H24 = 2.0 ** -24


def say(*a):
    print("[few]", *a, flush=True)


# ------------------------------------------------------------------ block
class Block:
    """A block on random packed weights, and its reference in 64 bits with a bound on the kernels' roundings."""

    def __init__(self, H, I, E, k, sh, act=BF16, score="sigmoid", groups=1, keep=1, renorm=True, bias=True, sh_bias=False, seed=0):
        self.g = torch.Generator().manual_seed(seed)
        self.H, self.I, self.E, self.k, self.sh, self.act = H, I, E, k, sh, act
        nb, nbi = (H + 255) // 256, (I + 255) // 256
        self.codebook = (torch.randint(0, 4, (256, 8), generator=self.g) * 2 - 3).to(torch.int8).cuda()
        self.gate, self.up = (self._cb2(E, I, nb, H) for _ in range(2))
        self.down = self._q2k(E, H, nbi, I)
        self.norm_w = (1 + self._n(H, std=0.2)).cuda()
        self.router_w = self._n(E, H, std=H ** -0.5).cuda()
        self.bias = self._n(E, std=0.05).cuda() if bias else None
        self.norm = M.NormWeights(self.norm_w, 1e-5)
        self.router = M.RouterWeights(self.router_w, k, score, self.bias, groups, keep, renorm, 2.5)
        self.layer = M.DeviceLayer(H, I, E, k, M.FMT_CB2, M.FMT_Q2K, self.gate, self.up, self.down, self.codebook, self.router_w)
        self.gate_up = self.shared_down = None
        if sh:
            b = [self._n(n, std=0.1).cuda() if sh_bias else None for n in (2 * sh, H)]
            self.gate_up, self.shared_down = (M.LinearI8(*self._i8(n, K), b[i]) for i, (n, K) in enumerate(((2 * sh, H), (H, sh))))
        self.w = M.BlockWeights(self.norm, self.router, self.layer, self.gate_up, self.shared_down, act)
        self.route = (score, groups, keep, renorm)

    def _n(self, *shape, std=1.0):
        return torch.randn(shape, generator=self.g) * std

    def _bytes(self, E, rows, nb, size):
        return torch.randint(0, 256, (E, rows, nb, size), generator=self.g, dtype=torch.uint8)

    def _half(self, w, at, v):
        w[..., at:at + 2] = v.to(torch.float16)[..., None].view(torch.uint8)

    def _cb2(self, E, rows, nb, K):
        w = self._bytes(E, rows, nb, 38)
        self._half(w, 0, 0.0007 + 0.0006 * torch.rand(w.shape[:3], generator=self.g))
        return w.cuda()

    def _q2k(self, E, rows, nb, K):
        w = self._bytes(E, rows, nb, 84)
        d = 0.0015 + 0.001 * torch.rand(w.shape[:3], generator=self.g)
        self._half(w, 0, d)
        self._half(w, 2, 1.5 * d)
        return w.cuda()

    def _i8(self, N, K):
        """Codes in rows of whole 16 bytes whose end holds anything, and scales."""
        w = torch.randint(-128, 128, (N, (K + 15) // 16 * 16), generator=self.g, dtype=torch.int8)
        w[:, :K] = torch.clamp(torch.round(self._n(N, K) * 35), -127, 127).to(torch.int8)
        return w.cuda()[:, :K], (0.5 + torch.rand(N, generator=self.g)).cuda() * (0.02 / 35)

    def unpack(self, fmt, w, rows, K):
        out = torch.empty((rows, K), device="cuda")
        M.q2_unpack(fmt, w.contiguous(), rows, K, self.codebook, out)
        return out.double()

    @staticmethod
    def spread(v, size):
        """The largest magnitude of each `size` neighbours, in their places."""
        T, n = v.shape
        p = torch.zeros((T, (n + size - 1) // size * size), dtype=v.dtype, device=v.device)
        p[:, :n] = v.abs()
        return p.view(T, -1, size).amax(2, keepdim=True).expand(-1, -1, size).reshape(T, -1)[:, :n]

    def reference(self, x, res):
        """(sum, n, idx, weights, y, bound on |kernel's y - y|), from the stated roundings of n on in 64 bits."""
        H, I, k = self.H, self.I, self.k
        s, total = x.float(), None
        if res is not None:
            total = (s + res.float()).to(res.dtype)
            s = total.float()
        r = (1 / torch.sqrt((s.double() ** 2).mean(1, keepdim=True) + float(np.float32(1e-5)))).float()
        n = ((s * r) * self.norm_w).to(self.act).float()
        score, groups, keep, renorm = self.route
        idx, wt = plain_route(n.cpu().numpy(), self.router_w.cpu().numpy(), k, score,
                              np.zeros(self.E, np.float32) if self.bias is None else self.bias.cpu().numpy(), groups, keep, renorm, 2.5)
        idx, wt = torch.from_numpy(np.asarray(idx)).cuda().long(), torch.from_numpy(np.asarray(wt)).double().cuda()
        n = n.double()
        # an activation is off by a rounding of its quotient and one of its integer, with the reciprocal's: 1.5 units of a
        # block's largest value / (127 * 2^16), and the block's scale by 2 roundings
        unit = 1.5 / (127 * 2.0 ** 16)

        def linear(v, ev, size, w, parts, adds):
            """v w^T and the bound: v's own error ev and its digits, the scales' roundings (5) and `adds` fp32 additions of parts
            whose magnitudes add up to |v| |w parts|."""
            y = v @ w.t()
            mag = v.abs() @ parts.t()
            return y, ev @ w.abs().t() + unit * (self.spread(v, size) + ev) @ w.abs().t() + (adds + 5) * H24 * mag

        def expert(v, gate, up, down, parts, adds, size):
            a, ea = linear(v, torch.zeros_like(v), 256, gate, gate.abs(), adds)
            u, eu = linear(v, torch.zeros_like(v), 256, up, up.abs(), adds)
            silu = a * torch.sigmoid(a)
            # silu' is at most 1.1; exp, sum, quotient and two products round (8 in all with exp's own)
            h, eh = silu * u, 1.1 * ea * (u.abs() + eu) + silu.abs() * eu + 8 * H24 * (silu * u).abs()
            return linear(h, eh, size, down, parts, adds)

        y = torch.zeros((x.shape[0], H), dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(y)
        mag = torch.zeros_like(y)
        none = self.down.clone()
        none[..., 20:] = 0                       # codes 0: only the mins are left
        adds = (max(H, I, self.sh) + 255) // 256 + 24          # blocks, lanes, waves, and 16 sums within a block's min term
        for e in idx.unique().tolist():
            t, j = torch.nonzero(idx == e, as_tuple=True)
            w = self.unpack(M.FMT_Q2K, self.down[e], H, I)
            m = self.unpack(M.FMT_Q2K, none[e], H, I)
            o, eo = expert(n[t], self.unpack(M.FMT_CB2, self.gate[e], I, H), self.unpack(M.FMT_CB2, self.up[e], I, H), w,
                           (w - m).abs() + m.abs(), adds, 64)
            y.index_add_(0, t, o * wt[t, j][:, None])
            bound.index_add_(0, t, (eo + 4 * H24 * o.abs()) * wt[t, j][:, None].abs())     # the weight's roundings, the product's
            mag.index_add_(0, t, (o * wt[t, j][:, None]).abs())
        if self.sh:
            (wu, su, bu), (wd, sd, bd) = self.gate_up.tensors, self.shared_down.tensors
            gu = wu.double() * su.double()[:, None]
            v, w = n, wd.double() * sd.double()[:, None]
            if bu is None:
                o, eo = expert(v, gu[:self.sh], gu[self.sh:], w, w.abs(), adds, 256)
            else:
                a, ea = linear(v, torch.zeros_like(v), 256, gu, gu.abs(), adds)
                a, ea = a + bu.double(), ea + H24 * (a.abs() + bu.double().abs())
                a, u, ea, eu = a[:, :self.sh], a[:, self.sh:], ea[:, :self.sh], ea[:, self.sh:]
                silu = a * torch.sigmoid(a)
                o, eo = linear(silu * u, 1.1 * ea * (u.abs() + eu) + silu.abs() * eu + 8 * H24 * (silu * u).abs(), 256, w, w.abs(), adds)
                o, eo = o + bd.double(), eo + 2 * H24 * bd.double().abs()
            y, bound, mag = y + o, bound + eo, mag + o.abs()
        # the waves' sums and the bias
        return total, n, idx.int(), wt, y, bound + 20 * H24 * mag + 1e-30

    def run(self, x, res, T=None, ws=None, y=None, stream=None, total=None):
        T = x.shape[0]
        r = M.Routing(T, self.k, self.E)
        y = torch.full((T, self.H), 77.0, device="cuda") if y is None else y
        ws = self.w.workspace(T) if ws is None else ws
        M.block_decode(self.w, x, res, total, y, r, ws, stream)
        return y, r


def check_block(b, T, xt=F32, rt=BF16, seed=1, pad=0):
    x = rnd(seed, T, b.H, std=0.5, dtype=xt)
    res = None if rt is None else rnd(seed + 1, T, b.H, std=2.0, dtype=rt)
    xd = strided(x, pad, 8) if pad else x.cuda()
    rd = None if res is None else strided(res, pad, 8) if pad else res.cuda()
    out = strided(torch.zeros(T, b.H), pad, 4) if pad else None
    total = None if res is None else strided(torch.zeros_like(res), pad, 8) if pad else torch.empty_like(rd)
    want_total, n, idx, wt, want, bound = b.reference(xd, rd)
    y, r = b.run(xd, rd, y=out, total=total)
    torch.cuda.synchronize()
    if res is not None:
        assert torch.equal(total, want_total)
    assert torch.equal(r.topk_idx, idx)
    assert torch.all((r.topk_w.double() - wt).abs() <= 3 * H24 * wt.abs())
    flat = idx.cpu().reshape(-1)
    perm = torch.sort(flat, stable=True).indices
    assert torch.equal(r.perm.cpu().long(), perm)
    assert torch.equal(r.inv.cpu().long(), torch.argsort(perm))
    assert torch.equal(r.offsets.cpu().long(), torch.searchsorted(flat[perm], torch.arange(b.E + 1).int()))
    off = (y.double() - want).abs()
    worst = float((off / bound).max())
    say("  worst error of its bound %.3f, relative %.2e" % (worst, float(off.norm() / want.norm())))
    assert worst <= 1
    assert off.norm() <= 3e-6 * want.norm()      # what the bound's sums of magnitudes hide
    if pad:
        for v, o in ((y, 4), (total, 8)):
            if v is not None:
                base = v._base
                assert torch.all(base[:, o + b.H:] == 77) and torch.all(base[:, :o] == 77)
    return y


BLOCKS = [  # T, H, I, E, k, shared, act, x, residual, score, groups, keep
    (1, 7168, 2048, 24, 8, 2048, BF16, F32, BF16, "sigmoid", 8, 4),
    (4, 7168, 2048, 16, 8, 2048, BF16, F32, BF16, "sigmoid", 4, 2),
    (1, 8, 8, 1, 1, 0, F32, F32, None, "softmax", 1, 1),
    (3, 8, 16, 2, 2, 1, BF16, BF16, BF16, "sigmoid", 1, 1),
    (2, 256, 256, 8, 2, 0, F32, F32, F32, "sigmoid", 1, 1),
    (3, 264, 264, 9, 3, 17, F32, BF16, F32, "softmax", 3, 1),
    (5, 520, 264, 16, 4, 300, BF16, F32, None, "sigmoid", 1, 1),
    (7, 1112, 712, 24, 5, 0, F32, F32, F32, "softmax", 1, 1),
    (2, 1032, 1032, 12, 4, 260, BF16, BF16, BF16, "sigmoid", 4, 3),
    (8, 2048, 768, 64, 6, 1408, BF16, F32, BF16, "sigmoid", 8, 3),
    (16, 1024, 512, 64, 16, 512, BF16, F32, BF16, "sigmoid", 1, 1),
    (16, 512, 128, 3, 3, 64, F32, F32, F32, "softmax", 1, 1),          # every expert has every token
    (13, 264, 72, 512, 7, 33, BF16, F32, BF16, "sigmoid", 64, 9),
    (6, 300 // 4 * 8, 2056, 10, 2, 8, F32, F32, None, "sigmoid", 1, 1),
    (9, 8192, 64, 5, 2, 24, BF16, F32, BF16, "softmax", 5, 2),
    (4, 8192, 264, 6, 3, 40, F32, F32, F32, "sigmoid", 1, 1),
    (2, 72, 8192, 4, 2, 8192, BF16, F32, BF16, "sigmoid", 1, 1),
    (10, 6152, 1000, 40, 8, 700, BF16, F32, BF16, "sigmoid", 1, 1),
]


@pytest.mark.parametrize("T,H,I,E,k,sh,act,xt,rt,score,groups,keep", BLOCKS)
def test_block(T, H, I, E, k, sh, act, xt, rt, score, groups, keep):
    need_gpu()
    say("block", T, H, I, E, k, sh, act, xt, rt, score, groups, keep)
    b = Block(H, I, E, k, sh, act, score, groups, keep, seed=T + H)
    check_block(b, T, xt, rt)
    check_block(b, T, xt, rt, seed=5, pad=16)


@pytest.mark.parametrize("T", range(1, 17))
def test_block_every_batch(T):
    need_gpu()
    say("block batch", T)
    check_block(Block(776, 328, 20, 4, 200, sh_bias=True, renorm=T % 2 == 0, bias=T % 3 != 0, seed=T), T)


def test_block_few_experts_left():
    """Biases of -inf that leave fewer experts than k, or none: weights 0, and the shared expert alone where nothing is left."""
    need_gpu()
    say("block masks")
    b = Block(256, 128, 8, 4, 64, groups=1, keep=1)
    b.bias[:] = -float("inf")
    x, res = rnd(3, 3, 256).cuda(), rnd(4, 3, 256).cuda()
    y, r = b.run(x, res)
    torch.cuda.synchronize()
    assert torch.all(r.topk_w == 0) and torch.equal(r.topk_idx.cpu(), torch.arange(4).int().expand(3, 4))
    only = Block(256, 128, 8, 4, 64)
    only.bias[:] = -float("inf")
    b.bias[5] = 0.1
    y2, r2 = b.run(x, res)
    torch.cuda.synchronize()
    assert torch.all(r2.topk_idx[:, 0] == 5) and torch.all(r2.topk_w[:, 1:] == 0) and torch.all((r2.topk_w[:, 0] - 2.5).abs() < 1e-6)
    assert torch.isfinite(y).all() and torch.isfinite(y2).all()


def test_block_odd_rows():
    """Zero rows, tiny and large ones; a row with a NaN or an infinity is NaN and leaves the others as they are."""
    need_gpu()
    say("block odd rows")
    b = Block(512, 256, 12, 3, 128, act=F32)
    x = rnd(9, 6, 512)
    x[1] = 0
    x[2] *= 1e-20
    x[3] *= 1e15
    good, _ = b.run(x.cuda(), None)
    bad = x.clone()
    bad[4, 7] = float("nan")
    bad[5, 300] = float("inf")
    y, r = b.run(bad.cuda(), None)
    torch.cuda.synchronize()
    assert torch.isfinite(good).all()
    # the others' sums may meet the waves in another order
    off = (y[:4] - good[:4]).abs().amax(1)
    assert torch.all(off <= 1e-5 * good[:4].abs().amax(1) + 1e-30)
    assert torch.isnan(y[4:]).any(1).all()
    assert torch.all((r.topk_idx >= 0) & (r.topk_idx < 12))
    want = b.reference(x.cuda(), None)
    assert torch.all((good.double() - want[4]).abs() <= want[5])


def test_block_in_place_and_repeated():
    """sum = residual, y = x, one workspace for several batches one after another, and the same bits every time."""
    need_gpu()
    say("block in place")
    b = Block(1024, 512, 32, 4, 256)
    ws = b.w.workspace(16)
    for T in (16, 1, 5, 2, 16):
        x, res = rnd(T, T, 1024).cuda(), rnd(T + 1, T, 1024, dtype=BF16).cuda()
        total, n, idx, wt, want, bound = b.reference(x, res)
        y, _ = b.run(x, res, ws=ws)
        again = x.clone()
        keep = res.clone()
        z, r = b.run(again, keep, ws=ws, y=again, total=keep)
        torch.cuda.synchronize()
        assert z is again and torch.equal(y, z) and torch.equal(keep, total) and torch.equal(r.topk_idx, idx)
        assert torch.all((y.double() - want).abs() <= bound)


def test_block_streams_and_graph():
    """Two calls at once on two streams with a workspace each; a captured call replayed between eager ones."""
    need_gpu()
    say("block streams")
    a, b = Block(2048, 512, 48, 6, 512, seed=1), Block(1536, 768, 32, 4, 0, seed=2)
    xa, ra, xb, rb = rnd(1, 4, 2048).cuda(), rnd(2, 4, 2048, dtype=BF16).cuda(), rnd(3, 7, 1536).cuda(), rnd(4, 7, 1536).cuda()
    ya, _ = a.run(xa, ra)
    yb, _ = b.run(xb, rb)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    ws = [a.w.workspace(4), b.w.workspace(7)]
    oa, ob = torch.empty_like(ya), torch.empty_like(yb)
    qa, qb = M.Routing(4, 6, 48), M.Routing(7, 4, 32)
    torch.cuda.synchronize()
    for _ in range(20):
        M.block_decode(a.w, xa, ra, None, oa, qa, ws[0], s)
        M.block_decode(b.w, xb, rb, None, ob, qb, ws[1], t)
    torch.cuda.synchronize()
    assert torch.equal(oa, ya) and torch.equal(ob, yb)
    say("block graph")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        M.block_decode(a.w, xa, ra, None, oa, qa, ws[0], s)
    for i in range(4):
        x = rnd(30 + i, 4, 2048)
        xa.copy_(x)
        oa.zero_()
        g.replay()
        want, _ = a.run(xa, ra)                  # eager, a workspace of its own
        torch.cuda.synchronize()
        assert torch.equal(oa, want)


def test_block_far_rows():
    """Rows of x, residual, sum and y more than 2^31 bytes apart."""
    need_gpu()
    say("block far rows")
    b = Block(64, 32, 4, 2, 16, act=F32)
    x, res = rnd(1, 2, 64), rnd(2, 2, 64)
    far = (1 << 29) + 64
    wide = lambda v: torch.empty(far + 64, device="cuda").as_strided((2, 64), (far, 1)).copy_(v)  # noqa: E731
    xd, rd, yd, sd = wide(x), wide(res), wide(x * 0), wide(x * 0)
    want = b.reference(x.cuda(), res.cuda())
    b.run(xd, rd, y=yd, total=sd)
    torch.cuda.synchronize()
    assert torch.equal(sd, want[0]) and torch.all((yd.double() - want[4]).abs() <= want[5])


def test_block_against_the_operators():
    """MoeBlock.decode and the operators one after another: the same routing and residual, y within the codes' rounding;
    the oracle's packed weights."""
    import os
    import sys
    need_gpu()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_block as B
    import synthetic as S
    from gpu_common import oracle_experts, rel_l2
    from oracle import moe_ref as R
    H, I, E = 512, 256, 16
    block, _, _ = B.make(H, I, E)
    for T in (1, 3, 16):
        say("block and operators", T)
        one, other = B.BlockBuffers(block, T), B.BlockBuffers(block, T)
        x, res = rnd(71, T, H).cuda(), rnd(72, T, H, dtype=BF16).cuda()
        first, second = res.clone(), res.clone()
        y = block.decode(x, first, one)
        z = block(x, second, other)
        torch.cuda.synchronize()
        assert torch.equal(first, second)
        for name in ("topk_idx", "topk_w", "offsets", "perm", "inv"):
            assert torch.equal(getattr(one.routing, name), getattr(other.routing, name))
        n = other.n.float().cpu().numpy()
        cfg = dict(hidden=H, inter=I, n_experts=E, top_k=4, fmt_gate_up=S.FMT_CB2, fmt_down=S.FMT_Q2K, sh_inter=0, seed=0)
        want = R.moe_layer(n, other.routing.topk_idx.cpu().numpy(), other.routing.topk_w.double().cpu().numpy(), oracle_experts(cfg, range(E)), None)
        (wu, su, _), (wd, sd, _) = block.gate_up.tensors, block.down.tensors
        d = lambda t: t.double().cpu()                                 # noqa: E731
        a, u = (d(other.n) @ (d(wu) * d(su)[:, None]).t()).chunk(2, 1)
        shared = (a * torch.sigmoid(a) * u) @ (d(wd) * d(sd)[:, None]).t()
        assert rel_l2(y.cpu(), want + shared.numpy()) < 3e-6
        # two roundings to 8 bits in the other, each evenly spread over a step of largest / 127, 1 / sqrt(12) of it in the mean square:
        # n, whose largest of 512 normal values is up to 4 times their rms, is off by 0.9%, and so are gate and up (1.3% of their
        # product); h, products of two normal values, has a largest of up to 12 times its rms: 2.8%.  Together 3.1%
        off = float((y - z).double().norm() / shared.norm())
        assert off < 0.031
    with pytest.raises(ValueError):
        block.decode(rnd(1, 17, H).cuda(), rnd(2, 17, H, dtype=BF16).cuda(), B.BlockBuffers(block, 17))
    assert B.main(["--tokens", "5", "--hidden", "512", "--inter", "256"]) < 0.05


def test_block_refusals():
    need_gpu()
    b = Block(256, 128, 8, 2, 0)
    x, y, r, ws = rnd(1, 2, 256).cuda(), torch.empty((2, 256), device="cuda"), M.Routing(2, 2, 8), b.w.workspace(2)
    res = rnd(2, 2, 256).cuda()
    for bad in (dict(x=x[:, :255]), dict(x=x.double()), dict(y=y.bfloat16()), dict(y=y[:1]), dict(total=res), dict(r=M.Routing(3, 2, 8)),
                dict(residual=res, total=res.bfloat16())):
        kw = dict(x=x, residual=None, total=None, y=y, r=r)
        kw.update(bad)
        with pytest.raises(ValueError):
            M.block_decode(b.w, kw["x"], kw["residual"], kw["total"], kw["y"], kw["r"], ws)
    with pytest.raises(ValueError):
        b.w.workspace(17)


# ------------------------------------------------------------------ plan
def check_plan(ids, n):
    T = ids.shape[0]
    plan = M.AdapterPlan(T, n)
    plan.tiles.fill_(77)
    M.adapter_plan(ids.cuda(), plan)
    torch.cuda.synchronize()
    key = torch.where((ids >= 0) & (ids < n), ids, n).long()
    order = torch.sort(key, stable=True).indices
    assert torch.equal(plan.order.cpu().long(), order)
    offsets = torch.searchsorted(key[order], torch.arange(n + 1))
    assert torch.equal(plan.offsets.cpu().long(), offsets)
    # the tiles cover every token once, each of one adapter
    size, seen = 16 if T <= 512 else 64, torch.zeros(T, dtype=torch.int32)
    ends = torch.cat([offsets[1:], torch.tensor([T])])
    for a, at in plan.tiles.cpu().tolist():
        assert -2 <= a < n
        if a == -2:
            continue
        bin_ = a if a >= 0 else n
        assert offsets[bin_] <= at < ends[bin_]
        seen[at:min(at + size, int(ends[bin_]))] += 1
    assert torch.all(seen == 1)
    return plan


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 333, 512, 513, 1000, 1024, 1025, 4097, 8192, 70001])
def test_plan(T):
    need_gpu()
    say("plan", T)
    g = torch.Generator().manual_seed(T)
    for n in (1, 2, 3, 31, 32, 100, 1024):
        check_plan(torch.randint(-1, n, (T,), generator=g).int(), n)
        check_plan(torch.sort(torch.randint(-2, n + 3, (T,), generator=g)).values.flip(0).int(), n)
    check_plan(torch.full((T,), -1).int(), 5)
    check_plan(torch.full((T,), 4).int(), 5)
    check_plan(torch.full((T,), 2 ** 31 - 1).int(), 1024)
    check_plan(torch.full((T,), -2 ** 31).int(), 1)


# ------------------------------------------------------------------ adapters
def make_adapters(seed, n, K, N, r, parts):
    a, b = rnd(seed, n, parts * r, K, std=K ** -0.5, dtype=BF16), rnd(seed + 1, n, N, r, std=r ** -0.5, dtype=BF16)
    return a, b, 0.5 + rnd(seed + 2, n).abs()


def adapters_reference(a, b, scale, parts, ids, x, add, yt):
    """y in 64 bits and the bound on the kernels' roundings."""
    T, N = add.shape
    n, r = b.shape[0], b.shape[2]
    x, want = x.double(), add.double()
    bound, wide = torch.zeros_like(want), N // parts
    K = x.shape[1]
    for q in range(n):
        t = torch.nonzero(ids == q)[:, 0]
        if not len(t):
            continue
        low, mag = x[t] @ a[q].double().t(), x[t].abs() @ a[q].double().abs().t()
        # a matrix instruction of 32 products is off by at most 12 units of 2^-24 of its running sum's magnitude; then the parts' and
        # waves' additions (fewer than the steps), the factors' two products and the terms' split
        elow = (12 * (K / 32 + 2) + 80) * H24 * mag
        for p in range(parts):
            bb = b[q, p * wide:(p + 1) * wide].double()
            cols = slice(p * wide, (p + 1) * wide)
            want[t, cols] += float(scale[q]) * (low[:, p * r:(p + 1) * r] @ bb.t())
            # three terms of each value, two steps of 32
            bound[t, cols] += float(scale[q]) * (elow[:, p * r:(p + 1) * r] + 80 * H24 * low[:, p * r:(p + 1) * r].abs()) @ bb.abs().t()
    rest = 2 * H24 * want.abs() + bound
    return want, rest + (2.0 ** -8 * (want.abs() + rest) if yt == BF16 else 0)


def check_adapters(seed, T, K, N, r, parts, n, kind, yt, pad=0, off=0, ids=None, inplace=False):
    a, b, scale = make_adapters(seed, n, K, N, r, parts)
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(-1, n, (T,), generator=g).int() if ids is None else ids
    xs = None
    if kind == "i8":
        x = torch.randint(-127, 128, (T, K), generator=g, dtype=torch.int8)
        xs = 0.01 + 0.01 * torch.rand(T, generator=g)
        value = x.double() * xs.double()[:, None]
    else:
        x = rnd(seed + 5, T, K, dtype=kind)
        value = x.double()
    add = rnd(seed + 6, T, N, dtype=yt)
    put = (lambda v: strided(v, pad, off)) if pad or off else (lambda v: v.cuda())  # noqa: E731
    w = M.AdapterWeights(a.cuda(), b.cuda(), scale.cuda(), parts)
    plan = M.AdapterPlan(T, n)
    M.adapter_plan(ids.cuda(), plan)
    xd, addd = put(x), put(add)
    y = addd if inplace else put(torch.zeros_like(add))
    M.adapters(w, plan, xd, None if xs is None else xs.cuda(), y, None if inplace else addd, w.workspace(T))
    torch.cuda.synchronize()
    want, bound = adapters_reference(a, b, scale, parts, ids, value, add, yt)
    got = y.double().cpu()
    worst = float(((got - want).abs() / (bound + 1e-30)).max())
    say("  worst error of its bound %.3f" % worst)
    assert worst <= 1
    if yt == F32:                                # roundings of 2^-24 meet in the mean square; with a term less they would be 2^-17
        assert float((got - want).norm()) <= 2.0 ** -21 * float((want - add.double()).norm() + add.double().norm())
    none = (ids < 0) | (ids >= n)
    assert torch.equal(y.cpu()[none], add[none])
    if pad:
        for v in (y, addd):
            base = v._base
            assert torch.all(base[:, off + N:] == 77) and torch.all(base[:, :off] == 77)


ADAPTERS = [  # T, K, N, rank, parts, adapters, x, y, pad, offset
    (1, 7168, 4096, 16, 2, 16, BF16, F32, 0, 0),
    (1, 1, 1, 1, 1, 1, F32, F32, 0, 0),
    (2, 7, 5, 3, 1, 2, BF16, BF16, 3, 1),
    (5, 64, 64, 8, 2, 3, "i8", F32, 0, 0),
    (17, 100, 66, 5, 3, 4, "i8", BF16, 5, 3),
    (33, 520, 260, 16, 2, 40, F32, BF16, 0, 0),
    (64, 2048, 768, 64, 4, 6, BF16, F32, 8, 8),
    (64, 1111, 1003, 13, 1, 1024, F32, F32, 0, 0),
    (333, 1000, 1002, 33, 1, 5, BF16, BF16, 1, 1),
    (512, 256, 512, 64, 2, 3, "i8", F32, 0, 0),
    (513, 264, 192, 32, 1, 3, BF16, BF16, 0, 0),
    (700, 1031, 130, 64, 2, 9, F32, BF16, 4, 2),
    (1000, 2000, 512, 48, 2, 2, F32, F32, 0, 0),
    (1500, 96, 1024, 64, 4, 20, BF16, F32, 0, 0),
    (2048, 500, 320, 4, 1, 300, "i8", BF16, 0, 0),
    (4000, 320, 96, 17, 1, 1, BF16, BF16, 16, 8),
]


@pytest.mark.parametrize("T,K,N,r,parts,n,kind,yt,pad,off", ADAPTERS)
def test_adapters(T, K, N, r, parts, n, kind, yt, pad, off):
    need_gpu()
    say("adapters", T, K, N, r, parts, n, kind, yt, pad, off)
    check_adapters(T, T, K, N, r, parts, n, kind, yt, pad, off)
    check_adapters(T + 1, T, K, N, r, parts, n, kind, yt, pad, off, inplace=True)
    check_adapters(T + 2, T, K, N, r, parts, n, kind, yt, ids=torch.full((T,), n - 1).int())
    check_adapters(T + 3, T, K, N, r, parts, n, kind, yt, ids=torch.full((T,), -1).int())


def test_adapters_streams_and_graph():
    """A captured plan and its projections replayed on new ids and inputs, between eager calls on another stream."""
    need_gpu()
    say("adapters graph")
    T, K, N, n = 48, 512, 384, 7
    a, b, scale = make_adapters(3, n, K, N, 16, 2)
    w = M.AdapterWeights(a.cuda(), b.cuda(), scale.cuda(), 2)
    plan, ws, s = M.AdapterPlan(T, n), w.workspace(T), torch.cuda.Stream()
    ids, x, add = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros(T, K, device="cuda"), rnd(4, T, N).cuda()
    y = torch.empty_like(add)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        M.adapter_plan(ids, plan)
        M.adapters(w, plan, x, None, y, add, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        M.adapter_plan(ids, plan)
        M.adapters(w, plan, x, None, y, add, ws)
    gen = torch.Generator().manual_seed(0)
    for i in range(4):
        new = torch.randint(-1, n, (T,), generator=gen).int()
        xi = rnd(50 + i, T, K)
        ids.copy_(new)
        x.copy_(xi)
        y.zero_()
        g.replay()
        other, ws2, y2 = M.AdapterPlan(T, n), w.workspace(T), torch.empty_like(add)
        M.adapter_plan(ids, other)
        M.adapters(w, other, x, None, y2, add, ws2)
        torch.cuda.synchronize()
        assert torch.equal(y, y2)
        want, bound = adapters_reference(a, b, scale, 2, new, xi.double(), add.cpu(), F32)
        assert torch.all((y.double().cpu() - want).abs() <= bound)


def test_adapters_do_not_touch_each_other():
    """A NaN or an infinity in one token, or in an adapter that one token has, stays there."""
    need_gpu()
    say("adapters nan")
    T, K, N, n = 40, 256, 128, 4
    a, b, scale = make_adapters(3, n, K, N, 8, 1)
    x, add = rnd(4, T, K), rnd(5, T, N)
    ids = (torch.arange(T) % 3).int()
    ids[7] = 3
    a[3, 2, 9] = float("nan")
    x[11, 5] = float("inf")
    x[12, 250] = float("nan")
    w = M.AdapterWeights(a.cuda(), b.cuda(), scale.cuda())
    plan, y = M.AdapterPlan(T, n), torch.empty((T, N), device="cuda")
    M.adapter_plan(ids.cuda(), plan)
    M.adapters(w, plan, x.cuda(), None, y, add.cuda(), w.workspace(T))
    torch.cuda.synchronize()
    bad = torch.zeros(T, dtype=torch.bool)
    bad[[7, 11, 12]] = True
    assert torch.isfinite(y.cpu()[~bad]).all() and torch.isnan(y.cpu()[bad]).all(1).all()


def test_adapters_far_rows():
    need_gpu()
    say("adapters far rows")
    K, N, far = 64, 64, (1 << 30) + 64
    a, b, scale = make_adapters(1, 2, K, N, 8, 1)
    w = M.AdapterWeights(a.cuda(), b.cuda(), scale.cuda())
    x, add = rnd(1, 3, K, dtype=BF16), rnd(2, 3, N, dtype=BF16)
    wide = lambda v: torch.empty(2 * far + 64, dtype=BF16, device="cuda").as_strided((3, 64), (far, 1)).copy_(v)  # noqa: E731
    xd, yd = wide(x), wide(add)
    ids = torch.tensor([1, 0, 1]).int()
    plan = M.AdapterPlan(3, 2)
    M.adapter_plan(ids.cuda(), plan)
    M.adapters(w, plan, xd, None, yd, None, w.workspace(3))
    torch.cuda.synchronize()
    want, bound = adapters_reference(a, b, scale, 1, ids, x.double(), add, BF16)
    assert torch.all((yd.double().cpu() - want).abs() <= bound)


def test_adapters_refusals():
    need_gpu()
    a, b, scale = (t.cuda() for t in make_adapters(1, 3, 64, 32, 8, 2))
    w, plan, x, y = M.AdapterWeights(a, b, scale, 2), M.AdapterPlan(4, 3), rnd(1, 4, 64).cuda(), rnd(2, 4, 32).cuda()
    ws = w.workspace(4)
    for bad in ((a.float(), b, scale, 2), (a, b[:2], scale, 2), (a, b, scale, 1), (a, b, scale[:2], 2)):
        with pytest.raises(ValueError):
            M.AdapterWeights(*bad)
    for ids in (torch.zeros(5, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)):
        with pytest.raises(ValueError):
            M.adapter_plan(ids.cuda(), plan)
    with pytest.raises(ValueError):
        M.adapters(w, M.AdapterPlan(4, 4), x, None, y, None, ws)
    with pytest.raises(ValueError):
        M.adapters(w, plan, x[:3], None, y, None, ws)
    with pytest.raises(ValueError):
        M.adapters(w, plan, x, None, y, y.bfloat16(), ws)
    with pytest.raises(M.MoeError):
        M.adapters(w, plan, x, None, y, None, None)
    with pytest.raises(ValueError):
        M.AdapterPlan(4, 2000)


# ------------------------------------------------------------------ together
def test_block_step_with_adapters():
    """A step of a batch through the block with its requests' adapters on the shared expert: one plan, both projections; and
    the tokens without an adapter as without any."""
    import os
    import sys
    need_gpu()
    say("step with adapters")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_block as B
    from bit_quantized_routed_amd.block import StepAdapters
    H, I, T, n = 512, 256, 24, 5
    block, _, _ = B.make(H, I, 16)
    up, down = make_adapters(11, n, H, 2 * I, 8, 2), make_adapters(21, n, I, H, 8, 1)
    ids = (torch.arange(T) % (n + 1) - 1).int()
    plan = M.AdapterPlan(T, n)
    M.adapter_plan(ids.cuda(), plan)
    step = StepAdapters(plan, M.AdapterWeights(*(t.cuda() for t in up), 2), M.AdapterWeights(*(t.cuda() for t in down)))
    x, res = rnd(71, T, H).cuda(), rnd(72, T, H, dtype=BF16).cuda()
    b, plain = B.BlockBuffers(block, T), B.BlockBuffers(block, T)
    y = block(x, res.clone(), b, adapters=step)
    z = block(x, res.clone(), plain)
    routed = torch.empty_like(y)
    M.ffn_decode(block.layer, b.n, M.ACT_BF16, T, b.routing, routed, b.ws_ffn)
    torch.cuda.synchronize()
    none = ids < 0
    assert torch.equal(y.cpu()[none], z.cpu()[none]) and not torch.equal(y.cpu()[~none], z.cpu()[~none])
    d = lambda t: t.double().cpu()                                     # noqa: E731
    # gate and up rows: the int8 layer's output, then the adapters
    want, bound = adapters_reference(*up, 2, ids, d(b.n), d(plain.gate_up), F32)
    assert torch.all((d(b.gate_up) - want).abs() <= bound)
    # the down rows on the codes of what they became
    (wd, sd, _) = block.down.tensors
    h = d(b.h) * d(b.h_scale)[:, None]
    base = d(routed) + h @ (d(wd) * d(sd)[:, None]).t()
    want, bound = adapters_reference(*down, 1, ids, h, base, F32)
    assert torch.all((d(y) - want).abs() <= bound + 8 * H24 * (base.abs() + d(routed).abs()))
