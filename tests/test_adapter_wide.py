"""Adapters beside projections so wide that one run of rows fills the machine:
no partial weight gradients, and no workspace for them."""
import pytest

from route_permute_grouped_gb300 import ops
from tests.test_adapter_gpu import _compare, _idx, _inputs


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


@pytest.mark.parametrize("T,K,N,r", [(2100, 1 << 20, 64, 128), (2100, 64, 1 << 20, 128), (3000, 1 << 19, 1 << 19, 16)])
def test_workspace_holds_what_is_used(T, K, N, r):
    # parts of u: at most 8 of [T, r padded] fp32; du: three of [T, r] bf16; no partials of dA and dB beside one run
    cfg = ops.make_adapter_config(T, K, N, 3, r)
    assert ops._size("moe_adapter_workspace_bytes", cfg, 1) <= T * r * (8 * 4 + 3 * 2) + (1 << 16)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,L,r", [(2100, 19464, 64, 5, 64), (2049, 64, 9736, 3, 72), (2500, 20000, 40, 2100 // 3, 16)])
def test_gradients_of_one_run(T, K, N, L, r):
    _compare(_inputs(T, K, N, L, r, T), _idx(T, L, T))
