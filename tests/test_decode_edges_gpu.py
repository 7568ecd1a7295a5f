"""The few-token layer, MXFP4 and the block norms at the ends of what they take: one
workspace under two captured graphs, weights beyond 32-bit offsets, the most tokens,
experts and slots, and fp32 streams whose rows end inside a warp."""
import pytest
import torch

from route_permute_grouped_gb300 import ops
from tests.test_few_gpu import Layer

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


def test_two_captured_layers_share_a_workspace():
    a, b = Layer(5, 1024, 16, 4, 512, Fs=256), Layer(40, 512, 24, 3, 384, mxfp4=True)
    want = {n: [t.clone() for t in L.run()] for n, L in (("a", a), ("b", b))}
    size = max(ops.few_workspace(a.cfg).numel(), ops.few_workspace(b.cfg, mxfp4=True).numel())
    ws, st = torch.zeros(size, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        graphs, got = {}, {}
        for n, L in (("a", a), ("b", b)):
            graphs[n] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[n], stream=st):
                got[n] = L.run(ws=ws)
        for order in ("a", "b", "ab", "ba", "aabb"):
            for t in (*got["a"], *got["b"]):
                t.fill_(-1)
            for n in order:
                graphs[n].replay()
            st.synchronize()
            for n in set(order):
                assert all(torch.equal(x, y) for x, y in zip(got[n], want[n])), order
    assert ops.device_status(ws) == 0


def test_two_captured_norms_share_a_workspace():
    g = torch.Generator("cuda").manual_seed(3)
    r = lambda *s, t=BF: torch.randn(s, generator=g, device="cuda").to(t)
    cases = []
    for T, H, stream in ((700, 1032, torch.float32), (33, 4096, BF)):
        cfg = ops.make_norm_config(T, H, gate="channel", post=True, residual_fp32=stream == torch.float32)
        cases.append((cfg, r(T, H), r(T, H, t=stream), r(H, t=torch.float32), r(H, t=torch.float32), r(H, t=torch.float32),
                      r(T, H), r(T, H, t=stream)))

    def step(c, ws):
        cfg, y, res, wp, gate, wn, dn, dh = c
        kw = dict(residual=res, post_weight=wp, gate=gate, pre_weight=wn)
        h, n, stats = ops.block_norm_fwd(cfg, y, **kw)
        return [h, n, *ops.block_norm_bwd(cfg, dn, y, stats, dh=dh, ws=ws, **kw).values()]

    want = [[t.clone() for t in step(c, ops.norm_workspace(c[0]))] for c in cases]
    ws = torch.empty(max(ops.norm_workspace(c[0]).numel() for c in cases), dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        graphs = [torch.cuda.CUDAGraph() for _ in cases]
        got = []
        for graph, c in zip(graphs, cases):
            with torch.cuda.graph(graph, stream=st):
                got.append(step(c, ws))
        for i in (0, 1, 1, 0):
            graphs[i].replay()
            st.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got[i], want[i]))


def test_weights_beyond_32_bit_offsets():
    # 130 experts of 4096 x 4096: 2.2e9 elements a weight, 2.3e9 bytes of MXFP4 tiles. The tokens
    # go to the last two experts alone: the same units in the same order as a layer of these two
    E, H, F, T = 130, 4096, 4096, 3
    small = Layer(T, H, 2, 2, F)
    last = slice(E - 2, E)
    W = []
    for w in small.W:
        big = torch.zeros((E, *w.shape[1:]), dtype=BF, device="cuda")
        big[last] = w
        W.append(big)
    router = torch.zeros((E, H), dtype=BF, device="cuda")
    router[last] = small.router_w
    lb = torch.full((E,), -1e4, device="cuda")
    lb[last] = 0.0
    cfg = ops.make_config(T, H, E, 2, F)
    y, idx, gate = ops.layer_few_fwd(cfg, small.x, router, *W, logit_bias=lb)
    sy, sidx, sgate = small.run()
    assert torch.equal(idx, sidx + (E - 2)) and torch.equal(gate, sgate) and torch.equal(y, sy)
    q = ops.mx4_quantize_weights(cfg, *W)
    y, idx, gate = ops.layer_few_fwd_mxfp4(cfg, small.x, router, q, logit_bias=lb)
    sq = ops.mx4_quantize_weights(small.cfg, *small.W)
    sy, sidx, sgate = ops.layer_few_fwd_mxfp4(small.cfg, small.x, small.router_w, sq)
    assert torch.equal(idx, sidx + (E - 2)) and torch.equal(gate, sgate) and torch.equal(y, sy)
    back, sback = ops.mx4_dequantize_weights(cfg, q), ops.mx4_dequantize_weights(small.cfg, sq)
    for a, b in zip(back[:3], sback[:3]):
        assert torch.equal(a[last], b) and not a[0].any()


@pytest.mark.parametrize("form", [dict(), dict(mxfp4=True, out_fp32=True)])
@pytest.mark.parametrize("over", [dict(), dict(lbias=True), dict(force_balanced=True)])
def test_most_tokens_experts_and_slots(form, over):
    L = Layer(64, 256, 256, 16, 128, Fs=128, **form, **over)
    ws = ops.few_workspace(L.cfg, mxfp4=L.mx)
    L.check(L.run(ws=ws))
    assert ops.device_status(ws) == 0 and not ws[:256].any()


@pytest.mark.parametrize("mxfp4", [False, True])
def test_every_token_to_the_same_sixteen_experts(mxfp4):
    # rows of an expert in several entries under MXFP4 (26 rows an entry with fp32 results)
    L = Layer(64, 128, 256, 16, 128, mxfp4=mxfp4, out_fp32=True)
    L.lb = torch.zeros(256, device="cuda")
    L.lb[240:] = 100.0
    L.check(L.run())


@pytest.mark.parametrize("H", [8, 24, 264, 1000, 7160, 8200])
def test_norms_of_fp32_streams_at_odd_widths(H):
    T = 9
    g = torch.Generator("cuda").manual_seed(H)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    y, res, dh, dn = r(T, H).to(BF), r(T, H), r(T, H), r(T, H).to(BF)
    wp, gate, wn = 1 + 0.2 * r(H), 0.5 + 0.2 * r(H), 1 + 0.2 * r(H)
    cfg = ops.make_norm_config(T, H, gate="channel", post=True, residual_fp32=True, residual_scale=0.75)
    kw = dict(residual=res, post_weight=wp, gate=gate, pre_weight=wn)
    h, n, stats = ops.block_norm_fwd(cfg, y, **kw)
    grads = ops.block_norm_bwd(cfg, dn, y, stats, dh=dh, **kw)
    # differences: <dh, h> + <dn, n> along a direction of every input, in fp64 by the formula
    f = lambda t: t.double()

    def value(y, res, wp, gate, wn):
        rms = lambda v: torch.rsqrt(v.square().mean(1, keepdim=True) + cfg.eps)
        hh = 0.75 * res + gate * (y * rms(y) * wp)
        return (f(dh) * hh).sum() + (f(dn) * hh * rms(hh) * wn).sum()

    # the gradients' formulas with every term by its magnitude: what roundings are relative to
    rms = lambda v: torch.rsqrt(v.square().mean(1, keepdim=True) + cfg.eps)
    Y, ry = f(y), rms(f(y))
    hh = 0.75 * f(res) + f(gate) * (Y * ry * f(wp))
    rh, big = rms(hh), 0.75 * f(res).abs() + (f(gate) * Y * f(wp)).abs() * ry
    dnw = (f(dn) * f(wn)).abs()
    dH = f(dh).abs() + rh * dnw + big * rh ** 3 * (dnw * big).mean(1, keepdim=True)
    gw = (f(gate) * f(wp)).abs() * dH
    size = {"dy": ry * (gw + Y.abs() * ry ** 2 * (gw * Y.abs()).mean(1, keepdim=True)), "dresidual": 0.75 * dH,
            "dpost": ((f(gate) * Y).abs() * ry * dH).sum(0), "dgate": ((f(wp) * Y).abs() * ry * dH).sum(0),
            "dpre": ((f(dn) * big).abs() * rh).sum(0)}
    inputs = [f(t) for t in (y, res, wp, gate, wn)]
    for i, name in enumerate(("dy", "dresidual", "dpost", "dgate", "dpre")):
        v = torch.randn(inputs[i].shape, generator=g, device="cuda", dtype=torch.float64)
        step = 1e-5
        moved = [[t + s * step * v if j == i else t for j, t in enumerate(inputs)] for s in (1, -1)]
        want = (value(*moved[0]) - value(*moved[1])) / (2 * step)
        # a term passes at most 128 fp32 roundings (two row sums of 8 to 16 a thread and ten exchanges, each
        # in a root or a product, some ten products): 2^-17 of it; dy's last rounding is 2^-8 of the element;
        # the difference leaves step^2 / 6 of the third derivative, about 1e-10 of the terms, and 1e-11 of
        # fp64's roundings: 1e-7 holds both
        bound = ((2.0 ** -17 + 1e-7) * size[name] * v.abs()).sum()
        if name == "dy":
            bound += (2.0 ** -8 * f(grads[name]).abs() * v.abs()).sum()
        assert abs((f(grads[name]) * v).sum() - want) <= bound, name


@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(torch.float32).min, float("nan"), float("inf")])
@pytest.mark.parametrize("left", [0, 1, 2, 5])
@pytest.mark.parametrize("opts", [dict(), dict(score="sigmoid"), dict(score="sigmoid", n_groups=4, topk_groups=2), dict(bias=True),
                                  dict(force_balanced=True)])
def test_masked_experts_are_routed_as_in_the_layer(low, left, opts):
    # a logit bias that leaves `left` experts of 16 (none, fewer than k, k, more): the same experts and gates as
    # layer_fwd takes, whatever they are. Logits of either are off by at most 256 2^-24 sum |x w|, which is below 30
    # here: 4.6e-4, twice that in a gate's quotient of exponentials, for both 1.8e-3 < 2^-9
    L = Layer(5, 256, 16, 2, 128, **opts)
    L.lb = torch.full((16,), low, device="cuda")
    keep = torch.tensor([3, 4, 9, 12, 15][:left], dtype=torch.long, device="cuda")
    L.lb[keep] = 0.0
    y, idx, gate = L.run()
    saved = ops.alloc_saved(L.cfg)
    want = ops.layer_fwd(L.cfg, L.x, L.router_w, *L.W, expert_bias=L.eb, logit_bias=L.lb, saved=saved)
    assert torch.equal(idx, saved["topk_idx"].view_as(idx))
    assert torch.allclose(gate, saved["topk_gate"].view_as(gate), rtol=2.0 ** -9, atol=0, equal_nan=True)
    assert torch.equal(y.isnan(), want.isnan())
