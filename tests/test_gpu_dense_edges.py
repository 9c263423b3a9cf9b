"""The operators around the routed experts at the edges of what they take.

Tolerances count roundings: one to fp32 is off by at most 2^-24 relative to its value.
"""
import numpy as np
import pytest
import torch

from gpu_common import need_gpu
from test_gpu_dense import BF16, check_route, rnd

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
