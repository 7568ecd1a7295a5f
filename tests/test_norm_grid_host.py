"""The norms' backward is launched with the blocks that an SM holds at once, by threads and by
the two rows that each has on its way in shared memory: its workspace says how many.
CPU only."""
import ctypes

import pytest

from route_permute_grouped_gb300 import build as B
from route_permute_grouped_gb300 import ops


def _blocks(lib, H, residual_fp32, out_fp32, T=1 << 24):
    cfg = ops.make_norm_config(T, H, residual_fp32=residual_fp32, out_fp32=out_fp32)
    return (lib.moe_norm_workspace_bytes(ctypes.byref(cfg)) - 256) // (16 * H)


# 1024 threads an SM, H / 8 a block; 228 KB of shared memory, 8 to 16 bytes a column and row
@pytest.mark.parametrize("H,residual_fp32,out_fp32,blocks", [
    (64, True, True, 16), (1024, False, False, 8), (1024, True, False, 8), (1024, True, True, 6), (2048, False, False, 4),
    (2048, True, True, 3), (4096, False, False, 2), (4096, True, False, 2), (4096, True, True, 1), (7168, True, True, 1),
    (8192, True, True, 1), (16384, True, True, 1)])
def test_blocks_an_sm(H, residual_fp32, out_fp32, blocks):
    B.build()
    lib = ops.lib()
    sms = _blocks(lib, 8192, False, False)
    assert _blocks(lib, H, residual_fp32, out_fp32) == blocks * sms
    assert _blocks(lib, H, residual_fp32, out_fp32, T=1) == 1
