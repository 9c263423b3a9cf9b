"""A workspace that was sized for a batch serves every smaller one (no GPU needed)."""
import ctypes

import pytest

import bit_quantized_routed_amd as M

FAKE = 0x1000            # never dereferenced: only sizes are asked for


def check_grows(size, counts):
    last = 0
    for T in counts:
        n = size(T)
        assert n >= last, (T, n, last)
        last = n


@pytest.mark.parametrize("N,K", [(4096, 7168), (7168, 2048), (64, 131071), (1003, 1111), (128, 100000), (2048, 7168), (16384, 8192),
                                 (16385, 8192), (300, 3500), (300, 3600), (1, 1)])
def test_linear_workspace_grows(N, K):
    W = M.LinearC(K, N, (K + 15) // 16 * 16, FAKE, FAKE, None)
    check_grows(lambda T: M.lib().moe_linear_i8_workspace_bytes(ctypes.byref(W), T),
                list(range(1, 700)) + list(range(700, 20000, 37)))


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E,H", [(256, 7168), (64, 128), (160, 1112), (1024, 512), (7, 8), (1, 4096), (1000, 7168), (32, 200)])
def test_router_workspace_grows(E, H, score):
    R = M.RouterC(hidden=H, n_experts=E, top_k=1, score=score, n_groups=1, keep_groups=1, flags=1, scale=1.0, w_router=FAKE, bias=None)
    near = [t for b in range(64, 41000, 64) for t in (b - 1, b, b + 1)]
    start = 640 * 256 // E
    check_grows(lambda T: M.lib().moe_route_scored_workspace_bytes(ctypes.byref(R), T),
                sorted(set(list(range(1, 200)) + near[::5] + list(range(start - 3, start + 4)) + [1 << 18, 1 << 20, (1 << 22) - 1])))
