"""The few-token layer's kernel when a wait runs out at the blocks' first barrier, with weights
on their way into shared memory: it ends with an error status, and what runs right
behind it is right."""
import pytest
import torch

from route_permute_grouped_gb300 import ops
from tests.test_few_gpu import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


@pytest.mark.parametrize("form", [dict(), dict(out_fp32=True), dict(mxfp4=True), dict(mxfp4=True, out_fp32=True)])
@pytest.mark.parametrize("T,Fs", [(1, 0), (9, 384), (64, 1024)])
def test_what_runs_behind_a_call_that_gave_up(form, T, Fs):
    # with a shared expert its weights are on their way before the barrier (phase 0), one to four stages of them
    L = Layer(T, 2048, 8, 2, 512, Fs=Fs, **form)
    ws, other = (ops.few_workspace(L.cfg, mxfp4=L.mx) for _ in range(2))
    want = [t.clone() for t in L.run(ws=ws)]
    norm = ops.make_norm_config(500, 4096, residual=False)
    y, w = torch.randn((500, 4096), device="cuda").to(torch.bfloat16), torch.ones(4096, device="cuda")
    h, n, st = ops.block_norm_fwd(norm, y, pre_weight=w)
    g = ops.block_norm_bwd(norm, y, y, st, pre_weight=w)
    torch.cuda.synchronize()
    ops.set_wait_limit_ns(1_000_000)
    try:
        for _ in range(5):
            ops.set_fault(1)
            L.run(ws=ws)
            ops.set_fault(0)
            got = L.run(ws=other)                                      # the same shared memory, right behind
            g2 = ops.block_norm_bwd(norm, y, y, st, pre_weight=w)
            assert all(torch.equal(a, b) for a, b in zip(want, got))
            assert all(torch.equal(g[k], g2[k]) for k in g)
            assert ops.device_status(ws) == ops.MOE_ERR_DEVICE_TIMEOUT and ops.device_status(other) == 0
            assert not ws[:256].any()
    finally:
        ops.set_fault(0)
        ops.set_wait_limit_ns(0)
    assert all(torch.equal(a, b) for a, b in zip(want, L.run(ws=ws)))
