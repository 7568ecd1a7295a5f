"""The norms around a block on rows far from 1, forward and backward, against the fp64
oracle: the squares of a row's values are the first that leave fp32, at 2^-63 and at
2^64 over the root of H. Bounds as in test_block_norm_gpu.py: every sum and product
there is relative to the magnitudes that meet in it, whatever the scale."""
import numpy as np
import pytest
import torch

from oracle import decode_oracle as DO
from route_permute_grouped_gb300 import ops
from tests.test_block_norm_gpu import BF, F32, _check, _f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


def _scaled(T, H, scale, gate="none", post=False, residual_fp32=False, out_fp32=False, dh_none=False, residual=True, pre=True):
    """h of the scale's size in every row (a gate of that size where u is normalised), its gradient of the
    inverse's, so that both terms of the norm's gradient count."""
    g = torch.Generator("cuda").manual_seed(T * 31 + H)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    stream, io = F32 if residual_fp32 else BF, F32 if out_fp32 else BF
    y = (scale * r(T, H)).to(io)
    gv = {"none": None, "channel": r(H), "token": r(T)}[gate]
    if post and gv is not None:
        gv = gv * (scale if isinstance(scale, float) else scale[:, 0])
    kw = {"residual": (scale * r(T, H)).to(stream) if residual else None, "post_weight": 1 + 0.3 * r(H) if post else None,
          "gate": gv, "pre_weight": 1 + 0.3 * r(H) if pre else None}
    dh, dn = None if dh_none else (r(T, H) / scale).to(stream), r(T, H).to(io) if pre else None
    cfg = ops.make_norm_config(T, H, eps=0.0, residual=residual, residual_scale=0.8, gate=gate, post=post, pre=pre,
                               residual_fp32=residual_fp32, out_fp32=out_fp32)
    h, n, stats = ops.block_norm_fwd(cfg, y, **kw)
    got = {"h": h, "n": n, **ops.block_norm_bwd(cfg, dn, y, stats, dh=dh, **kw)}
    if not pre:
        assert got.pop("n") is None
    want, mag = DO.block_norm(_f64(y), _f64(kw["residual"]), 0.8, _f64(kw["post_weight"]), _f64(gv), _f64(kw["pre_weight"]),
                              eps=0.0, dh=_f64(dh), dn=_f64(dn))
    assert set(got) == set(want)
    for name, t in got.items():
        assert torch.isfinite(t.float()).all(), name
        _check(name, t, want[name], mag[name], 64 if name in "hn" else 192 if name in ("dpre", "dpost", "dgate") else 128)


SCALES = [2.0 ** e for e in (-55, -45, 45, 55)]


# one thread a column run, rows on their way in shared memory, two runs a thread straight from memory
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("H", [264, 4104, 8200])
@pytest.mark.parametrize("over", [dict(), dict(dh_none=True), dict(residual=False), dict(gate="token", post=True),
                                  dict(gate="channel", post=True, residual_fp32=True),
                                  dict(gate="channel", residual_fp32=True, out_fp32=True)])
def test_rows_far_from_one(scale, H, over):
    _scaled(5, H, scale, **over)


@pytest.mark.parametrize("over", [dict(), dict(gate="token", post=True), dict(gate="token", out_fp32=True, residual_fp32=True)])
def test_rows_of_unlike_sizes(over):
    # every row its own power of two: a row's factors are its own
    scale = torch.tensor(SCALES * 3, device="cuda")[:, None]
    _scaled(12, 512, scale, **over)


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_without_a_norm_no_square_is_taken(gate):
    _scaled(5, 264, 2.0 ** 90, gate=gate, pre=False)


def test_the_gradient_along_a_row_is_zero():
    # n does not change when h grows: with dn = n / w the gradient of h is 0 but for roundings, which is the
    # difference of two terms of the size dn / rms; either alone is as large as the whole
    H = 4096
    for scale in (2.0 ** -50, 1.0, 2.0 ** 50):
        y = scale * torch.randn((3, H), generator=torch.Generator("cuda").manual_seed(5), device="cuda")
        w = torch.ones(H, device="cuda")
        cfg = ops.make_norm_config(3, H, eps=0.0, residual=False, out_fp32=True)
        h, n, st = ops.block_norm_fwd(cfg, y, pre_weight=w)
        dn = y / y.square().mean(1, keepdim=True).sqrt()
        g = ops.block_norm_bwd(cfg, dn, y, st, pre_weight=w)
        # (bf16's 2^-8 of what is left, 128 half steps of fp32 of each of the two terms)
        assert (g["dy"].float().abs() * scale <= 2 * 128 * 2.0 ** -24 * dn.abs().clamp(min=1.0)).all()
