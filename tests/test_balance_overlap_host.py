"""The gradient of the logits over other arguments of its call: in place or
apart. CPU only (no call here launches)."""
import ctypes

import pytest

from route_permute_grouped_gb300 import build as B
from route_permute_grouped_gb300 import ops

P = ctypes.c_void_p
T, E = 64, 8
NBYTES, STATS = 4 * T * E, 4 * (E + 2)
LOGITS, APART = 1 << 20, 1 << 24


@pytest.fixture(scope="module")
def lib():
    B.build()
    return ops.lib()


@pytest.mark.parametrize("dlogits,stats", [(LOGITS + 16, APART), (LOGITS - 16, APART), (LOGITS + NBYTES - 16, APART),
                                           (APART, APART), (APART, APART + NBYTES - 16), (APART + 16, APART)])
def test_shifted_overlap_is_refused(lib, dlogits, stats):
    cfg = ops.make_balance_config(T, E, 2)
    assert lib.moe_balance_loss_bwd(ctypes.byref(cfg), P(LOGITS), P(stats), None, None, None, P(dlogits), None) == \
        ops.MOE_ERR_INVALID_ARG
