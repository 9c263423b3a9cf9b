"""Edges of the operators for a few tokens that need no GPU: what is checked, kept or sized before any launch."""
import ctypes

import bit_quantized_routed_amd as M
from test_few_host import FAKE, Parts, _block


def test_block_workspace_at_any_offset():
    """The block lays its workspace out from a multiple of 256 on, wherever the caller's begins (a reader's cached line may hold
    nothing that another work-group writes later): the size that the library names has room for that, and a smaller one is
    refused where the gap takes what the call needs."""
    for T in (1, 4, 16):
        B = Parts()
        have = M.lib().moe_block_decode_workspace_bytes(ctypes.byref(B.c), T)
        need = have - 240                        # at a multiple of 256
        assert need % 256 == 0
        for at in range(0, 256, 16):
            gap = -at % 256
            # never launched
            assert _block(B, T=T, ws=FAKE + at, ws_bytes=need + gap - 1) == -3, (T, at)
