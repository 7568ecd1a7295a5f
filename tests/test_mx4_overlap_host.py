"""The bf16 weights that MXFP4 tiles are turned back into are outputs: they may not overlap
one another. CPU only (no call here launches)."""
import ctypes

import pytest

from route_permute_grouped_gb300 import build as B
from route_permute_grouped_gb300 import ops

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    B.build()
    return ops.lib()


@pytest.mark.parametrize("Fs", [0, 128])
def test_weights_written_back_may_not_overlap(lib, Fs):
    # order: W1 W3 W2 Ws1 Ws3 Ws2
    cfg = ops.make_config(1, 256, 3, 1, 128, F_shared=Fs)
    sizes = [2 * 3 * 256 * 128] * 3 + [2 * 256 * Fs] * 3
    tiles = ctypes.byref(ops.MoeMx4Weights(*[(10 + j) << 24 for j in range(4)]))
    n = 6 if Fs else 3
    for i in range(n):
        for j in range(n):
            if i == j:
                continue
            for at in (0, sizes[j] - 16, 16 - sizes[i]):  # all of it, the last bytes, the first
                p = [(k + 1) << 24 for k in range(6)]
                p[i] = p[j] + at
                st = lib.moe_mx4_dequantize_weights(ctypes.byref(cfg), tiles, *[P(v) for v in p], None)
                assert st == ops.MOE_ERR_INVALID_ARG, (i, j, at)
