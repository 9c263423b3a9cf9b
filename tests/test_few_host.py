"""Refusals of the operators for a few tokens of many requests (no GPU needed): every bad argument returns its documented
status before any HIP call."""
import ctypes

import pytest

import bit_quantized_routed_amd as M

FAKE = 0x1000            # never dereferenced: every call below fails validation first or has T == 0


def _err():
    return M.lib().moe_last_error().decode()


# ------------------------------------------------------------------ block
class Parts:
    """A valid block of H = 64, I = 32, E = 8, k = 2 and 16 shared features, with fields replaced."""

    def __init__(self, norm=None, router=None, layer=None, gate_up=None, down=None, act_n=1, without=()):
        n = dict(hidden=64, eps=1e-6, weight=FAKE)
        r = dict(hidden=64, n_experts=8, top_k=2, score=0, n_groups=1, keep_groups=1, flags=1, scale=1.0, w_router=FAKE, bias=None)
        y = dict(hidden=64, inter=32, n_experts=8, top_k=2, fmt_gate_up=M.FMT_CB2, fmt_down=M.FMT_Q2K, sh_inter=0, flags=0, w_gate=FAKE,
                 w_up=FAKE, w_down=FAKE, codebook=FAKE, sh_gate=None, sh_up=None, sh_down=None, w_router=None, expert_slot=None)
        u = dict(in_features=64, out_features=32, ldw=64, w=FAKE, w_scale=FAKE, bias=None)
        d = dict(in_features=16, out_features=64, ldw=16, w=FAKE, w_scale=FAKE, bias=None)
        c = []
        for name, cls, base, more in (("norm", M.NormC, n, norm), ("router", M.RouterC, r, router), ("layer", M.Layer, y, layer),
                                      ("gate_up", M.LinearC, u, gate_up), ("down", M.LinearC, d, down)):
            base.update(more or {})
            c.append(None if name in without else ctypes.pointer(cls(**base)))
        self.keep = c
        self.c = M.BlockC(*c, act_n)


def _block(B=None, T=4, x=FAKE, ax=0, ldx=64, res=FAKE, ar=1, ldr=64, total=FAKE, lds=64, y=FAKE, ldy=64, out=FAKE, ws=FAKE,
           ws_bytes=1 << 40):
    B = Parts() if B is None else B
    return M.lib().moe_block_decode(ctypes.byref(B.c), T, x, ax, ldx, res, ar, ldr, total, lds, y, ldy, out, out, out, out, out, ws,
                                    ws_bytes, None, None)


BAD = [dict(norm=dict(hidden=0)), dict(norm=dict(eps=-1.0)), dict(norm=dict(weight=None)), dict(norm=dict(weight=FAKE + 4)),
       dict(norm=dict(hidden=72)), dict(router=dict(hidden=72)), dict(router=dict(n_experts=16)), dict(router=dict(top_k=3)),
       dict(router=dict(score=2)), dict(router=dict(flags=2)), dict(router=dict(w_router=None)), dict(layer=dict(inter=0)),
       dict(layer=dict(inter=36)), dict(layer=dict(w_gate=None)), dict(layer=dict(w_down=FAKE + 8)), dict(layer=dict(codebook=None)),
       dict(layer=dict(hidden=72)), dict(gate_up=dict(in_features=72, ldw=80)), dict(gate_up=dict(out_features=34)),
       dict(gate_up=dict(ldw=72)), dict(gate_up=dict(w=None)), dict(down=dict(out_features=72)), dict(down=dict(in_features=24, ldw=32)),
       dict(down=dict(w_scale=None)), dict(act_n=2), dict(without=("norm",)), dict(without=("router",)), dict(without=("layer",)),
       dict(without=("gate_up",)), dict(without=("down",))]


@pytest.mark.parametrize("kw", BAD, ids=[str(i) for i in range(len(BAD))])
def test_block_refusals(kw):
    B = Parts(**kw)
    assert _block(B) == -1 and _err()
    assert M.lib().moe_block_decode_workspace_bytes(ctypes.byref(B.c), 4) == 0


@pytest.mark.parametrize("kw", [
    dict(layer=dict(fmt_gate_up=M.FMT_Q4K)), dict(layer=dict(fmt_down=M.FMT_Q4K)), dict(layer=dict(fmt_gate_up=M.FMT_CB2S)),
    dict(layer=dict(sh_inter=256)), dict(layer=dict(flags=1)), dict(layer=dict(expert_slot=FAKE)), dict(layer=dict(inter=8200)),
    dict(layer=dict(n_experts=520), router=dict(n_experts=520)), dict(layer=dict(top_k=17, n_experts=32), router=dict(top_k=17, n_experts=32)),
    dict(gate_up=dict(out_features=2 * 8200), down=dict(in_features=8200, ldw=8208))])
def test_block_unsupported(kw):
    assert _block(Parts(**kw)) == -2 and _err()


def test_block_call_refusals():
    assert M.lib().moe_block_decode(None, 4, FAKE, 0, 64, FAKE, 1, 64, FAKE, 64, FAKE, 64, *([FAKE] * 5), FAKE, 1 << 40, None, None) == -1
    for kw in (dict(T=-1), dict(x=None), dict(x=FAKE + 8), dict(ax=2), dict(ar=7), dict(ldx=63), dict(ldx=68), dict(res=FAKE + 2),
               dict(ldr=60), dict(ldr=68), dict(total=FAKE + 8), dict(lds=60), dict(res=None), dict(y=None), dict(y=FAKE + 2), dict(ldy=63),
               dict(out=None), dict(ws=None), dict(ws=FAKE + 8)):
        assert _block(**kw) == -1, kw
        assert _err()
    assert _block(T=17) == -2
    assert _block(ws_bytes=1000) == -3
    assert _block(T=0, x=None, y=None, out=None, ws=None) == 0
    assert _block(Parts(without=("gate_up", "down")), T=0) == 0


def test_block_workspace_serves_smaller_batches():
    for kw in (dict(), dict(without=("gate_up", "down")), dict(layer=dict(inter=8192)),
               dict(norm=dict(hidden=8192), router=dict(hidden=8192), layer=dict(hidden=8192), without=("gate_up", "down"))):
        B = Parts(**kw)
        need = [M.lib().moe_block_decode_workspace_bytes(ctypes.byref(B.c), T) for T in range(1, 17)]
        assert all(a <= b for a, b in zip(need, need[1:])) and need[0] > 0
        assert M.lib().moe_block_decode_workspace_bytes(ctypes.byref(B.c), 17) == 0


# ------------------------------------------------------------------ plan
def _plan(ids=FAKE, T=4, n=3, order=FAKE, offsets=FAKE, tiles=FAKE):
    return M.lib().moe_adapter_plan(ids, T, n, order, offsets, tiles, None, None)


def test_plan_refusals():
    for kw in (dict(T=-1), dict(n=0), dict(n=1025), dict(ids=None), dict(order=None), dict(offsets=None), dict(tiles=None),
               dict(ids=FAKE + 2), dict(order=FAKE + 1), dict(tiles=FAKE + 4)):
        assert _plan(**kw) == -1, kw
        assert _err()
    assert _plan(T=(1 << 20) + 1) == -2
    assert _plan(T=0, ids=None, order=None, offsets=None, tiles=None) == 0


def test_tiles_hold_every_batch():
    """Tiles of one adapter each: the count for any split of T tokens into n adapters and those without."""
    import random
    rng = random.Random(0)
    for _ in range(300):
        T, n = rng.choice([1, 2, 15, 16, 17, 64, 500, 512, 513, 576, 2000]), rng.choice([1, 2, 3, 17, 100, 1024])
        tile, left, used = (16 if T <= 512 else 64), T, 0
        for b in range(n + 1):
            c = left if b == n else rng.randint(0, min(left, rng.choice([1, 2, tile, 5 * tile])))
            used += -(-c // tile)
            left -= c
        assert used <= M.lib().moe_adapter_tiles(T, n), (T, n)
    assert M.lib().moe_adapter_tiles(0, 4) == M.lib().moe_adapter_tiles(4, 0) == M.lib().moe_adapter_tiles((1 << 20) + 1, 4) == 0


# ------------------------------------------------------------------ adapters
def _set(**kw):
    base = dict(in_features=64, out_features=32, n_adapters=3, rank=8, parts=2, lda=64, ldb=8, a=FAKE, b=FAKE, scale=FAKE)
    base.update(kw)
    return M.AdapterSetC(**base)


def _adapters(W=None, T=4, order=FAKE, offsets=FAKE, tiles=FAKE, x=FAKE, kind=1, ldx=64, xs=None, add=FAKE, lda=32, y=FAKE, ay=0,
              ldy=32, ws=FAKE, ws_bytes=1 << 40):
    W = _set() if W is None else W
    return M.lib().moe_adapters(ctypes.byref(W), T, order, offsets, tiles, x, kind, ldx, xs, add, lda, y, ay, ldy, ws, ws_bytes, None,
                                None)


@pytest.mark.parametrize("kw", [
    dict(in_features=0), dict(out_features=0), dict(n_adapters=0), dict(n_adapters=1025), dict(rank=0), dict(rank=65), dict(parts=0),
    dict(parts=3), dict(out_features=64, parts=64), dict(a=None), dict(b=None), dict(scale=None), dict(a=FAKE + 8), dict(b=FAKE + 2),
    dict(scale=FAKE + 1), dict(lda=68), dict(lda=56), dict(ldb=4), dict(rank=9), dict(in_features=(1 << 24) + 1, lda=1 << 25)])
def test_adapter_set_refusals(kw):
    assert _adapters(_set(**kw)) == -1 and _err()
    assert M.lib().moe_adapters_workspace_bytes(ctypes.byref(_set(**kw)), 4) == 0


def test_adapters_call_refusals():
    assert M.lib().moe_adapters(None, 4, FAKE, FAKE, FAKE, FAKE, 1, 64, None, FAKE, 32, FAKE, 0, 32, FAKE, 1 << 40, None, None) == -1
    for kw in (dict(T=-1), dict(order=None), dict(offsets=None), dict(tiles=None), dict(tiles=FAKE + 4), dict(x=None), dict(x=FAKE + 1),
               dict(kind=3), dict(kind=-1), dict(ldx=63), dict(xs=FAKE), dict(kind=2), dict(kind=2, xs=FAKE + 2), dict(add=None),
               dict(add=FAKE + 2), dict(lda=31), dict(y=None), dict(ldy=31), dict(ay=2), dict(ws=None), dict(ws=FAKE + 8)):
        assert _adapters(**kw) == -1, kw
        assert _err()
    assert _adapters(T=(1 << 20) + 1) == -2
    assert _adapters(ws_bytes=16) == -3
    assert _adapters(T=0, order=None, x=None, add=None, y=None, ws=None) == 0


def test_adapters_workspace_serves_smaller_batches():
    """What a call of t tokens asks for is there in a workspace sized for T >= t, and no byte too few is taken."""
    def call(W, t, nbytes):                      # never launched: x is not aligned to its elements
        return _adapters(W, T=t, ldx=1 << 20, x=FAKE + 1, ws_bytes=nbytes)

    for kw in (dict(), dict(in_features=7168, lda=7168), dict(in_features=7168, lda=7168, n_adapters=100), dict(rank=64, ldb=64, parts=1)):
        W = _set(**kw)
        last = 0
        for T in (1, 2, 3, 15, 16, 17, 31, 33, 64, 100, 256, 511, 512, 513, 576, 577, 1000, 4096, 8192, 40000):
            have = M.lib().moe_adapters_workspace_bytes(ctypes.byref(W), T)
            assert have >= last
            last = have
            for t in {1, 2, max(1, T // 3), max(1, T - 1), min(T, 512), min(T, 513), T}:
                if t <= T:
                    assert call(W, t, have) == -1
        assert call(W, 512, 512 * 4 - 1) == -3
