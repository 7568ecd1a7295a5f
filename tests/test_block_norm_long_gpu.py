"""Sums over more rows a block than are added in fp32 alone, where a block has several
warps: two floats in the workspace, read again and added to, for either order of a
thread's columns. The blocks are counted from the workspace."""
import pytest
import torch

from route_permute_grouped_gb300 import ops
from tests.test_block_norm_gpu import BF, F32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


def _blocks(H, **over):
    cfg = ops.make_norm_config(1 << 24, H, **over)
    return (ops.norm_workspace(cfg).numel() - 256) // (16 * H)


def _sums(cfg, y, kw, dh, dn, chunk):
    """dpre, dpost and dgate by the formulas in fp64, and the sums of their terms' magnitudes."""
    out, mag = {}, {}

    def add(name, v, m):
        out[name] = out.get(name, 0.0) + v.sum(0)
        mag[name] = mag.get(name, 0.0) + m.sum(0)

    rms = lambda v: torch.rsqrt(v.square().mean(1, keepdim=True) + cfg.eps)
    for i in range(0, y.shape[0], chunk):
        f = lambda t: t[i:i + chunk].double()
        yy = f(y)
        if cfg.post:
            yy = yy * rms(yy)
            u = yy * kw["post_weight"].double()
        else:
            u = yy
        g = kw["gate"].double() if cfg.gate else 1.0
        h, big = g * u, (g * u).abs()
        if cfg.residual:
            r = cfg.residual_scale * f(kw["residual"])
            h, big = h + r, big + r.abs()
        rh = rms(h)
        d, hh, bh = f(dn), h * rh, big * rh
        add("dpre", d * hh, d.abs() * bh)
        if cfg.post or cfg.gate:
            dw = d * kw["pre_weight"].double()
            dH = f(dh) + rh * (dw - hh * (dw * hh).mean(1, keepdim=True))
            mH = f(dh).abs() + rh * (dw.abs() + bh * (dw.abs() * bh).mean(1, keepdim=True) * (1 + 2 * bh.square().mean(1, keepdim=True)))
            add("dgate", dH * u, mH * u.abs())
            add("dpost", g * dH * yy, (g * yy).abs() * mH)
    return out, mag


# 66 rows a block and some: a second run of rows is added to what the first left. 64 threads, 544 (one block an SM,
# four columns in either half of an fp32 row) and 1024 of two runs
@pytest.mark.parametrize("H,over", [(512, dict(residual=False)), (4104, dict(gate="channel", post=True, residual_fp32=True)),
                                    (16384, dict(residual=False)), (1000, dict(gate="channel", post=True, residual_fp32=True, out_fp32=True))])
def test_more_rows_a_block_than_fp32_alone_adds(H, over):
    T = 66 * _blocks(H, **over) + 5
    g = torch.Generator("cuda").manual_seed(H)
    r = lambda *s, t=F32: torch.randn(s, generator=g, device="cuda", dtype=t)
    stream, io = F32 if over.get("residual_fp32") else BF, F32 if over.get("out_fp32") else BF
    cfg = ops.make_norm_config(T, H, **over)
    assert (ops.norm_workspace(cfg).numel() - 256) // (16 * H) * 64 < T
    y, dn = r(T, H, t=io), r(T, H, t=io)
    kw = {"residual": r(T, H, t=stream) if cfg.residual else None, "post_weight": 1 + 0.3 * r(H) if cfg.post else None,
          "gate": 0.5 + 0.2 * r(H) if cfg.gate else None, "pre_weight": 1 + 0.3 * r(H)}
    dh = r(T, H, t=stream)
    _, _, stats = ops.block_norm_fwd(cfg, y, **kw)
    got = ops.block_norm_bwd(cfg, dn, y, stats, dh=dh, **kw)
    want, mag = _sums(cfg, y, kw, dh, dn, 4096)
    assert {"dpre", "dpost", "dgate"} & set(got) == set(want)
    for name, v in want.items():
        # 192 half steps of fp32 as in test_block_norm_gpu.py, one more for the result
        err = (got[name].double() - v).abs()
        assert (err <= 2.0 ** -24 * (192 * mag[name] + v.abs())).all(), (name, float((err / mag[name]).max() * 2 ** 24))
