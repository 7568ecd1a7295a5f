"""Norms before and after a block, with gate and scaled residual, against the fp64
oracle, forward and backward.

Tolerances: every output is off by half a step of its type and by what its fp32
operations add to the magnitudes that meet in it (the oracle's `mag`). A sum of
squares over a row adds at most 16 squares in a chain and joins them in about 20
additions, halved by the root; a value then takes about a dozen roundings, the
backward twice that: 64 half steps of fp32 forward, 128 backward. A sum over rows
adds chains of at most 64 rows: 192."""
import numpy as np
import pytest
import torch

from oracle import decode_oracle as DO
from route_permute_grouped_gb300 import ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


def _f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def _inputs(T, H, gate="none", post=False, residual=True, pre=True, residual_fp32=False, out_fp32=False, seed=0):
    g = torch.Generator("cuda").manual_seed(seed + T * 31 + H)
    r = lambda *s, dt=F32: torch.randn(s, generator=g, device="cuda").to(dt)
    stream, io = F32 if residual_fp32 else BF, F32 if out_fp32 else BF
    kw = {"residual": r(T, H, dt=stream) if residual else None, "post_weight": 1 + 0.3 * r(H) if post else None,
          "gate": {"none": None, "channel": r(H), "token": r(T)}[gate], "pre_weight": 1 + 0.3 * r(H) if pre else None}
    return r(T, H, dt=io), kw, r(T, H, dt=stream), r(T, H, dt=io) if pre else None


def _check(name, t, want, mag, steps):
    err = np.abs(_f64(t) - want)
    lim = HALF[t.dtype] * np.abs(want) + steps * HALF[F32] * mag * (1 + HALF[t.dtype]) + 1e-37
    assert (err <= lim).all(), (name, float((err / lim).max()))


def _both(T, H, dh_none=False, scale=0.8, **over):
    y, kw, dh, dn = _inputs(T, H, **over)
    cfg = ops.make_norm_config(T, H, residual=kw["residual"] is not None, residual_scale=scale, gate=over.get("gate", "none"),
                               post=kw["post_weight"] is not None, pre=kw["pre_weight"] is not None,
                               residual_fp32=over.get("residual_fp32", False), out_fp32=over.get("out_fp32", False))
    h, n, stats = ops.block_norm_fwd(cfg, y, **kw)
    if dh_none:
        dh = None
    ws = ops.norm_workspace(cfg)
    ws[256:] = 0x5a
    g = ops.block_norm_bwd(cfg, dn, y, stats, dh=dh, ws=ws, **kw)
    want, mag = DO.block_norm(_f64(y), _f64(kw["residual"]), scale, _f64(kw["post_weight"]), _f64(kw["gate"]),
                              _f64(kw["pre_weight"]), dh=_f64(dh), dn=_f64(dn))
    _check("h", h, want["h"], mag["h"], 64)
    if n is not None:
        _check("n", n, want["n"], mag["n"], 64)
    assert (n is None) == (kw["pre_weight"] is None)
    assert {k for k in g if g[k] is not None} == {k for k in want if k.startswith("d")}
    for k, t in g.items():
        _check(k, t, want[k], mag[k], 192 if k in ("dpre", "dpost", "dgate") else 128)
    assert not ws[:256].any()
    return cfg, y, kw, dh, dn, (h, n, stats), g


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("types", [(False, False), (True, False), (False, True), (True, True)])
def test_every_form(gate, post, residual, pre, types):
    _both(37, 264, gate=gate, post=post, residual=residual, pre=pre, residual_fp32=types[0], out_fp32=types[1])


# both sides of each border of the thread counts, the rows on their way and the longest rows
@pytest.mark.parametrize("T,H", [(1, 8), (2, 16), (1, 1016), (5, 1032), (3, 4096), (3, 4104), (2, 7168), (3, 7176), (2, 8192),
                                 (2, 8200), (3, 16384), (700, 8), (400, 1024), (2000, 72)])
@pytest.mark.parametrize("over", [dict(), dict(gate="channel", post=True, residual_fp32=True),
                                  dict(gate="token", post=True, residual_fp32=True, out_fp32=True)])
def test_sizes(T, H, over):
    _both(T, H, **over)


def test_more_rows_than_are_added_in_fp32_alone():
    # 80 and 160 rows a block: two floats in the workspace take over after 64
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    _both(80 * 16 * sms, 64, gate="channel", post=True)
    _both(160 * 2 * sms, 512)


def test_long_sums_keep_their_bits():
    # dn h rh is 1 in one column of every row, 2^-20 in the next: sums that plain fp32 additions in a row would lose
    T, H = 1 << 20, 16
    y = torch.zeros((T, H), device="cuda", dtype=BF)
    y[:, 0] = 1.0
    cfg = ops.make_norm_config(T, H, residual=False, eps=0.0)
    w = torch.ones(H, device="cuda")
    h, n, st = ops.block_norm_fwd(cfg, y, pre_weight=w)
    assert (n[:, 0] == 4.0).all()
    dn = torch.zeros((T, H), device="cuda", dtype=BF)
    dn[:, 0] = 0.25
    dn[T // 2:, 0] = 2.0 ** -22
    g = ops.block_norm_bwd(cfg, dn, y, st, pre_weight=w)
    want = T / 2 + (T / 2) * 2.0 ** -20
    # each of the at most 16 blocks an SM has one run of 64 rows that holds both kinds, where a sum of up to 64 ones
    # takes none of up to 64 times 2^-20: 0.15 in all on 152 SMs, where plain additions would lose the whole half
    mixed = 16 * torch.cuda.get_device_properties(0).multi_processor_count * 64 * 2.0 ** -20
    lim = 2 * 2.0 ** -24 * want + mixed
    assert abs(float(g["dpre"][0]) - want) <= lim < want - T / 2


def test_without_a_gradient_of_h():
    _both(9, 512, dh_none=True, gate="channel", post=True)
    _both(9, 512, dh_none=True)


def test_rows_with_infinities_and_nans_stay_by_themselves():
    y, kw, dh, dn = _inputs(6, 256, gate="channel", post=True)
    cfg = ops.make_norm_config(6, 256, gate="channel", post=True)
    clean = ops.block_norm_fwd(cfg, y, **kw)
    z = y.clone()
    z[1, 3], z[4, 200] = float("nan"), float("inf")
    h, n, st = ops.block_norm_fwd(cfg, z, **kw)
    keep = [0, 2, 3, 5]
    assert torch.equal(h[keep], clean[0][keep]) and torch.equal(n[keep], clean[1][keep])
    assert torch.isnan(n[1].float()).any() and torch.isnan(n[4].float()).any()
    g = ops.block_norm_bwd(cfg, dn, z, st, dh=dh, **kw)
    good = ops.block_norm_bwd(cfg, dn, y, clean[2], dh=dh, **kw)
    assert torch.equal(g["dy"][keep], good["dy"][keep]) and torch.equal(g["dresidual"][keep], good["dresidual"][keep])


def test_rows_of_zeros():
    y, kw, dh, dn = _inputs(3, 128, post=True, residual=False)
    y.zero_()
    cfg = ops.make_norm_config(3, 128, post=True, residual=False)
    h, n, st = ops.block_norm_fwd(cfg, y, **kw)
    assert not h.any() and not n.any()
    g = ops.block_norm_bwd(cfg, dn, y, st, **kw)
    assert torch.isfinite(g["dy"].float()).all() and not g["dpost"].any() and not g["dpre"].any()


def test_in_place():
    cfg, y, kw, dh, dn, (h, n, st), g = _both(33, 512, gate="channel", post=True)
    res, yy = kw["residual"].clone(), y.clone()
    h2, n2, st2 = ops.block_norm_fwd(cfg, yy, **{**kw, "residual": res}, h=res, n=yy)
    assert torch.equal(h2, h) and torch.equal(n2, n) and torch.equal(st2, st) and h2 is res and n2 is yy
    out = ops.alloc_norm_grads(cfg)
    out["dresidual"], out["dy"] = dh.clone(), dn.clone()
    g2 = ops.block_norm_bwd(cfg, out["dy"], y, st, dh=out["dresidual"], grads=out, **kw)
    assert all(torch.equal(g[k], g2[k]) for k in g)


def test_the_same_bits_every_time_and_on_another_stream():
    cfg, y, kw, dh, dn, (h, n, st), g = _both(1000, 1536, gate="channel", post=True)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(3):
            h2, n2, st2 = ops.block_norm_fwd(cfg, y, **kw)
            g2 = ops.block_norm_bwd(cfg, dn, y, st2, dh=dh, **kw)
    s.synchronize()
    assert torch.equal(h, h2) and torch.equal(n, n2) and all(torch.equal(g[k], g2[k]) for k in g)


def test_captured_while_an_eager_result_lives():
    cfg, y, kw, dh, dn, (h, n, st), g = _both(64, 1024, gate="token", post=True)
    ws, st2 = ops.norm_workspace(cfg), torch.cuda.Stream()
    yy, keep = y.clone(), [t.clone() for t in g.values()]
    with torch.cuda.stream(st2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st2):
            hc, nc, sc = ops.block_norm_fwd(cfg, yy, **kw)
            gc = ops.block_norm_bwd(cfg, dn, yy, sc, dh=dh, ws=ws, **kw)
        yy.copy_(y * 2)
        graph.replay()
        yy.copy_(y)
        graph.replay()
    st2.synchronize()
    assert torch.equal(hc, h) and torch.equal(nc, n) and all(torch.equal(g[k], gc[k]) for k in g)
    assert all(torch.equal(a, b) for a, b in zip(keep, g.values()))


def test_offsets_beyond_32_bits():
    T, H = (1 << 32) // 16384 + 2, 16384
    y = torch.zeros((T, H), dtype=BF, device="cuda")
    y[-3:] = torch.randn((3, H), device="cuda").to(BF)
    w = torch.rand(H, device="cuda")
    cfg, small = ops.make_norm_config(T, H, residual=False), ops.make_norm_config(3, H, residual=False)
    h, n, st = ops.block_norm_fwd(cfg, y, pre_weight=w)
    tail = y[-3:].contiguous()
    h3, n3, st3 = ops.block_norm_fwd(small, tail, pre_weight=w)
    assert torch.equal(h[-3:], h3) and torch.equal(n[-3:], n3) and torch.equal(st[-3:], st3)
    g = ops.block_norm_bwd(cfg, y, y, st, pre_weight=w)  # dn = y
    g3 = ops.block_norm_bwd(small, tail, tail, st3, pre_weight=w)
    assert torch.equal(g["dy"][-3:], g3["dy"])
    assert torch.allclose(g["dpre"], g3["dpre"], rtol=1e-5, atol=1e-6)


def test_refusals():
    y, kw, dh, dn = _inputs(4, 64, gate="channel", post=True)
    cfg = ops.make_norm_config(4, 64, gate="channel", post=True)
    h, n, st = ops.block_norm_fwd(cfg, y, **kw)
    for over in (dict(residual=None), dict(post_weight=None), dict(gate=None), dict(pre_weight=None),
                 dict(residual=kw["residual"].float()), dict(gate=kw["gate"][:32].contiguous()), dict(post_weight=kw["post_weight"].cpu())):
        with pytest.raises(ops.MoeError):
            ops.block_norm_fwd(cfg, y, **{**kw, **over})
    with pytest.raises(ops.MoeError):
        ops.block_norm_fwd(cfg, y.float(), **kw)
    with pytest.raises(ops.MoeError):
        ops.block_norm_fwd(cfg, y[:, ::1][:3], **kw)
    with pytest.raises(ops.MoeError):
        ops.block_norm_bwd(cfg, None, y, st, dh=dh, **kw)
    with pytest.raises(ops.MoeError):
        ops.block_norm_bwd(cfg, dn, y, st, dh=dh, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"), **kw)
    for bad in (dict(H=12), dict(H=16392), dict(T=0), dict(gate=3), dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(ops.MoeError):
            ops.norm_workspace(ops.make_norm_config(**{**dict(T=4, H=64), **bad}))
