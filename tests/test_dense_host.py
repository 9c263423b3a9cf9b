"""Refusals of the operators around the routed experts (no GPU needed): every
bad argument returns its documented status before any HIP call."""
import ctypes

import pytest

import bit_quantized_routed_amd as M

FAKE = 0x1000            # never dereferenced: every call below fails validation first or has T == 0
BIG = 1 << 40


def _err():
    return M.lib().moe_last_error().decode()


# ------------------------------------------------------------------ scored routing
def _router(**kw):
    base = dict(hidden=256, n_experts=16, top_k=2, score=0, n_groups=4, keep_groups=2, flags=1, scale=1.0,
                w_router=FAKE, bias=None)
    base.update(kw)
    return M.RouterC(**base)


def _route(R, x=FAKE, act=1, ldx=256, T=4, out=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return M.lib().moe_route_scored(None if R is None else ctypes.byref(R), x, act, ldx, T, out, out, out, out, out,
                                    ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw", [
    dict(hidden=0), dict(hidden=100), dict(n_experts=0), dict(n_experts=1025, n_groups=1, keep_groups=1), dict(score=2),
    dict(n_groups=0), dict(n_groups=3), dict(n_experts=256, n_groups=128, keep_groups=100), dict(keep_groups=0), dict(keep_groups=5), dict(top_k=0), dict(top_k=9),
    dict(n_experts=128, n_groups=1, keep_groups=1, top_k=65), dict(flags=2), dict(w_router=None),
    dict(w_router=FAKE + 4), dict(bias=FAKE + 2)])
def test_router_refusals(kw):
    assert _route(_router(**kw)) == -1 and _err()
    assert M.lib().moe_route_scored_workspace_bytes(ctypes.byref(_router(**kw)), 4) == 0


def test_route_scored_call_refusals():
    R = _router()
    assert _route(None) == -1
    for kw in (dict(T=-1), dict(act=2), dict(x=None), dict(x=FAKE + 8), dict(ldx=252), dict(ldx=248), dict(out=None),
               dict(ws=None), dict(ws=FAKE + 8), dict(T=1 << 30)):
        assert _route(R, **kw) == -1, kw
    assert _route(R, ws_bytes=64) == -3
    assert _route(R, T=1 << 22) == -2
    assert _route(R, T=0, x=None, out=None, ws=None) == 0
    a, b = (M.lib().moe_route_scored_workspace_bytes(ctypes.byref(R), T) for T in (4, 4000))
    assert 0 < a < b


# ------------------------------------------------------------------ norm
def _norm(N=None, T=4, x=FAKE, ax=1, ldx=64, res=FAKE, ar=1, ldr=64, total=FAKE, lds=64, out=FAKE, ao=1, ldo=64, q=FAKE,
          ldq=64, qs=FAKE):
    N = M.NormC(64, 1e-6, FAKE) if N is None else N
    return M.lib().moe_residual_norm(ctypes.byref(N), T, x, ax, ldx, res, ar, ldr, total, lds, out, ao, ldo, q, ldq, qs,
                                     None, None)


def test_norm_refusals():
    for N in (M.NormC(0, 1e-6, FAKE), M.NormC(65537, 1e-6, FAKE), M.NormC(64, -1.0, FAKE), M.NormC(64, float("nan"), FAKE),
              M.NormC(64, 1e-6, None), M.NormC(64, 1e-6, FAKE + 2)):
        assert _norm(N) == -1 and _err()
    assert M.lib().moe_residual_norm(None, 4, *([FAKE, 1, 64] * 2), FAKE, 64, FAKE, 1, 64, FAKE, 64, FAKE, None, None) == -1
    for kw in (dict(T=-1), dict(x=None), dict(x=FAKE + 1), dict(ax=5), dict(ar=5), dict(ao=-1), dict(ldx=63), dict(ldr=63),
               dict(lds=10), dict(ldo=63), dict(ldq=63), dict(res=None), dict(out=None, q=None, qs=None), dict(q=None),
               dict(qs=None), dict(qs=FAKE + 2), dict(ar=0, res=FAKE + 2), dict(ldx=-64), dict(ldx=BIG + 1)):
        assert _norm(**kw) == -1, kw
    assert _norm(T=1 << 22) == -2
    assert _norm(T=0, x=None, out=None, q=None, qs=None) == 0


# ------------------------------------------------------------------ quant
def _quant(x=FAKE, act=1, ldx=128, T=4, K=64, flags=1, q=FAKE, ldq=64, qs=FAKE):
    return M.lib().moe_quant_i8(x, act, ldx, T, K, flags, q, ldq, qs, None, None)


def test_quant_refusals():
    for kw in (dict(K=0), dict(K=65537), dict(T=-1), dict(act=2), dict(flags=2), dict(x=None), dict(x=FAKE + 1), dict(ldx=127),
               dict(q=None), dict(ldq=63), dict(qs=None), dict(qs=FAKE + 1)):
        assert _quant(**kw) == -1, kw
        assert _err()
    assert _quant(T=1 << 22) == -2 and "rows" in _err()
    assert _quant(T=0, x=None, q=None, qs=None) == 0


# ------------------------------------------------------------------ linear
def _linear(W=None, T=4, x=FAKE, ldx=64, xs=FAKE, add=None, lda=0, y=FAKE, ay=0, ldy=32, ws=FAKE, ws_bytes=1 << 40):
    W = M.LinearC(64, 32, 64, FAKE, FAKE, None) if W is None else W
    return M.lib().moe_linear_i8(ctypes.byref(W), T, x, ldx, xs, add, lda, y, ay, ldy, ws, ws_bytes, None, None)


def test_linear_refusals():
    for W in (M.LinearC(0, 32, 64, FAKE, FAKE, None), M.LinearC(131072, 32, 131072, FAKE, FAKE, None),
              M.LinearC(64, 0, 64, FAKE, FAKE, None), M.LinearC(64, 32, 64, None, FAKE, None),
              M.LinearC(64, 32, 64, FAKE, None, None), M.LinearC(64, 32, 64, FAKE + 8, FAKE, None),
              M.LinearC(64, 32, 72, FAKE, FAKE, None), M.LinearC(64, 32, 48, FAKE, FAKE, None),
              M.LinearC(64, 32, 64, FAKE, FAKE + 2, None), M.LinearC(64, 32, 64, FAKE, FAKE, FAKE + 2)):
        assert _linear(W) == -1 and _err()
        assert M.lib().moe_linear_i8_workspace_bytes(ctypes.byref(W), 4) == 0
    assert M.lib().moe_linear_i8(None, 4, FAKE, 64, FAKE, None, 0, FAKE, 0, 32, FAKE, 1 << 40, None, None) == -1
    for kw in (dict(T=-1), dict(x=None), dict(x=FAKE + 8), dict(ldx=72), dict(ldx=48), dict(xs=None), dict(xs=FAKE + 2),
               dict(y=None), dict(y=FAKE + 2), dict(ay=3), dict(ldy=31), dict(add=FAKE, lda=31), dict(add=FAKE + 1, lda=32),
               dict(ws=FAKE + 8)):
        assert _linear(**kw) == -1, kw
    assert _linear(M.LinearC(64, 2 ** 31 - 1, 64, FAKE, FAKE, None), T=2 ** 31 - 1, ldy=2 ** 31) == -2
    assert _linear(M.LinearC(64, 1 << 26, 64, FAKE, FAKE, None), T=1, ldy=1 << 26) == -2
    assert _linear(T=0, x=None, xs=None, y=None, ws=None) == 0


def test_linear_workspace_is_checked():
    """Where a shape needs a workspace, a missing or short one is refused."""
    for T, N, K in ((1, 64, 8192), (32, 64, 65536), (300, 128, 100000), (64, 7168, 2048)):
        W = M.LinearC(K, N, K, FAKE, FAKE, None)
        need = M.lib().moe_linear_i8_workspace_bytes(ctypes.byref(W), T)
        if need:
            assert _linear(W, T=T, ldx=K, ldy=N, ws=None, ws_bytes=0) == -1
            assert _linear(W, T=T, ldx=K, ldy=N, ws_bytes=need - 1) == -3


# ------------------------------------------------------------------ the Python entry points
def test_python_refusals():
    torch = pytest.importorskip("torch")
    f = lambda *s: torch.zeros(s)                                      # noqa: E731
    n = M.NormWeights(f(64))
    with pytest.raises(ValueError):
        M.residual_norm(n, f(4, 63), out=f(4, 63))
    with pytest.raises(ValueError):
        M.residual_norm(n, f(64, 4).t(), out=f(4, 64))                 # columns, not rows
    with pytest.raises(ValueError):
        M.residual_norm(n, f(4, 64).double(), out=f(4, 64))
    with pytest.raises(ValueError):
        M.residual_norm(n, f(4, 64), f(4, 64), f(4, 64).bfloat16(), f(4, 64))
    with pytest.raises(ValueError):
        M.residual_norm(n, f(4, 64), out=f(4, 64), q=f(4, 64), q_scale=f(4))
    with pytest.raises(ValueError):
        M.quant_i8(f(4, 64), M.empty_i8(4, 64, "cpu"), f(4), swiglu=True)
    with pytest.raises(ValueError):
        M.LinearI8(torch.zeros((4, 30), dtype=torch.int8), f(4))       # the last row ends inside its 16 bytes
    with pytest.raises(ValueError):
        M.LinearI8(M.empty_i8(4, 30, "cpu"), f(5))
    with pytest.raises(M.MoeError) as e:
        M.linear_i8(M.LinearI8(M.empty_i8(4, 32, "cpu"), f(4)), torch.zeros((2, 40), dtype=torch.int8)[:, :32], f(2), f(2, 4), stream=0)
    assert e.value.status == -1
    with pytest.raises(KeyError):
        M.RouterWeights(f(8, 64), 2, score="relu")
