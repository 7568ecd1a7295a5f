"""Clipping at the ends of its arguments' ranges."""
import pytest
import torch

from route_permute_grouped_gb300 import ops

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bad", [None, INF, -INF])
def test_an_infinite_threshold_scales_nothing(kind, dtype, bad):
    # the norm alone, as a training loop asks for it: also where the norm is infinite
    t = torch.linspace(-3, 3, 5001).to(dtype).cuda()
    if bad is not None:
        t[1234] = bad
    keep, out = t.clone(), torch.zeros_like(t)
    norm = ops.clip_grad_norm(ops.tensor_list([t], out=[out]), INF, kind)
    assert torch.equal(out, keep) and torch.equal(norm, ops.grad_norm([t], kind))
    assert (float(norm) == INF) == (bad is not None)
    ops.clip_grad_norm([t], INF, kind)
    assert torch.equal(t, keep)


@pytest.mark.parametrize("kind", ["l2", "max"])
def test_a_nan_reaches_every_gradient_whatever_the_threshold(kind):
    for limit in (0.0, 1.0, INF):
        ts = [torch.ones(100, device="cuda"), torch.ones(7, device="cuda")]
        ts[0][3] = float("nan")
        norm = ops.clip_grad_norm(ts, limit, kind)
        assert bool(torch.isnan(norm)) and all(bool(torch.isnan(t).all()) for t in ts)


def test_a_norm_beyond_fp32_counts_as_infinite():
    t = torch.full((1000,), 3e38, device="cuda")
    assert float(ops.clip_grad_norm([t], 1.0)) == INF and not t.any()
