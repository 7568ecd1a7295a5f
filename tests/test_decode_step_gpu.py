"""The norms, the few-token layer and the training layer together, as a model runs them."""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import decode_oracle as DO
from route_permute_grouped_gb300 import ops

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _rand(g, *s, std=1.0):
    return torch.randn(s, generator=g, device="cuda") * std


def _rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


@pytest.mark.parametrize("mxfp4", [False, True])
def test_decoding_steps_of_two_blocks(mxfp4):
    # norm -> layer -> gate, residual and the next block's norm -> layer -> residual, eager and as one graph
    T, H, E, k, F = 6, 512, 16, 4, 256
    g = torch.Generator("cuda").manual_seed(3)
    cfg = ops.make_config(T, H, E, k, F)
    blocks = []
    for _ in range(2):
        W = [_rand(g, E, H, F, std=H ** -0.5).to(BF), _rand(g, E, H, F, std=H ** -0.5).to(BF), _rand(g, E, F, H, std=F ** -0.5).to(BF)]
        blocks.append({"W": W, "r": _rand(g, E, H, std=1.5 * H ** -0.5).to(BF), "pre": 1 + 0.2 * _rand(g, H),
                       "post": 1 + 0.2 * _rand(g, H), "gate": 0.5 + 0.1 * _rand(g, H),
                       "q": ops.mx4_quantize_weights(cfg, *W) if mxfp4 else None})
    first = ops.make_norm_config(T, H, residual=False, residual_fp32=True)
    mid = ops.make_norm_config(T, H, gate="channel", post=True, residual_fp32=True, residual_scale=0.9)
    last = ops.make_norm_config(T, H, gate="channel", post=True, pre=False, residual_fp32=True, residual_scale=0.9)
    ws = ops.few_workspace(cfg, mxfp4=mxfp4)

    def layer(b, n):
        if mxfp4:
            return ops.layer_few_fwd_mxfp4(cfg, n, b["r"], b["q"], ws=ws)[0]
        return ops.layer_few_fwd(cfg, n, b["r"], *b["W"], ws=ws)[0]

    def step(x):
        h, n, _ = ops.block_norm_fwd(first, x, pre_weight=blocks[0]["pre"])
        b = blocks[0]
        h, n, _ = ops.block_norm_fwd(mid, layer(b, n), residual=h, post_weight=b["post"], gate=b["gate"], pre_weight=blocks[1]["pre"])
        b = blocks[1]
        return ops.block_norm_fwd(last, layer(b, n), residual=h, post_weight=b["post"], gate=b["gate"], h=h)[0]

    def oracle(x):
        f = lambda t: _f64(t)
        h = f(x)
        n = DO.block_norm(h, pre=f(blocks[0]["pre"]))[0]["n"]
        for i, b in enumerate(blocks):
            y = DO.few_layer(O.bf16_rne(n), f(b["r"]), *[f(w) for w in b["W"]], k, mxfp4=mxfp4)["y"]
            nxt = f(blocks[1]["pre"]) if i == 0 else None
            o = DO.block_norm(O.bf16_rne(y), h, 0.9, f(b["post"]), f(b["gate"]), nxt)[0]
            h, n = o["h"], o.get("n")
        return h

    xs = [_rand(g, T, H).to(BF) for _ in range(2)]
    want = [step(x).clone() for x in xs]
    # bf16 roundings of n and y along the way: half a step of 2^-8 of their own size, four times
    for x, w in zip(xs, want):
        assert _rel(_f64(w), oracle(x)) < 4 * 2.0 ** -8
    st, x = torch.cuda.Stream(), xs[0].clone()
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            out = step(x)
        for i in (0, 1):
            x.copy_(xs[i])
            graph.replay()
            st.synchronize()
            assert torch.equal(out, want[i])


def test_training_step_with_norms_and_clipping():
    # residual stream -> norm -> layer -> post norm, gate and residual; the backward through all of it
    T, H, E, k, F = 300, 256, 8, 2, 128
    g = torch.Generator("cuda").manual_seed(4)
    cfg = ops.make_config(T, H, E, k, F)
    W1, W3, W2 = (_rand(g, *s, std=s[1] ** -0.5).to(BF) for s in ((E, H, F), (E, H, F), (E, F, H)))
    wr, pre, post, gate = _rand(g, E, H, std=H ** -0.5).to(BF), 1 + 0.2 * _rand(g, H), 1 + 0.2 * _rand(g, H), 0.5 + 0.2 * _rand(g, H)
    x, dh = _rand(g, T, H).to(BF), _rand(g, T, H).to(BF)
    before = ops.make_norm_config(T, H, residual=False)
    after = ops.make_norm_config(T, H, gate="channel", post=True, pre=False)
    ws, saved = ops.workspace(cfg, True), ops.alloc_saved(cfg)

    def step(x):
        h0, n, s0 = ops.block_norm_fwd(before, x, pre_weight=pre)
        y = ops.layer_fwd(cfg, n, wr, W1, W3, W2, saved=saved, ws=ws)
        h, _, s1 = ops.block_norm_fwd(after, y, residual=h0, post_weight=post, gate=gate)
        g1 = ops.block_norm_bwd(after, None, y, s1, dh=dh, residual=h0, post_weight=post, gate=gate)
        gl = ops.layer_bwd(cfg, g1["dy"], n, wr, W1, W3, W2, saved, ws=ws)
        g0 = ops.block_norm_bwd(before, gl["dx"], x, s0, dh=g1["dresidual"], pre_weight=pre)
        norm = ops.clip_grad_norm([g0["dpre"], g1["dpost"], g1["dgate"], gl["dW_r"]], 1e9)
        return h, g0["dy"], g0["dpre"], g1["dpost"], g1["dgate"], norm

    f = _f64
    h, dx, dpre, dpost, dgate, norm = step(x)
    n = O.bf16_rne(DO.block_norm(f(x), pre=f(pre))[0]["n"])
    y = O.layer_fwd(n, f(wr), f(W1), f(W3), f(W2), k)["y"]
    o1, _ = DO.block_norm(y, f(x), 1.0, f(post), f(gate), dh=f(dh))
    gl = O.layer_bwd(n, f(wr), f(W1), f(W3), f(W2), O.bf16_rne(o1["dy"]), k)
    o0, _ = DO.block_norm(f(x), pre=f(pre), dh=o1["dresidual"], dn=gl["dx"])
    # values stored as bf16 between the operators: a few half steps of 2^-8 in the mean square
    for name, got, want in (("h", h, o1["h"]), ("dx", dx, o0["dy"]), ("dpre", dpre, o0["dpre"]), ("dpost", dpost, o1["dpost"]),
                            ("dgate", dgate, o1["dgate"])):
        assert _rel(f(got), want) < 3 * 2.0 ** -8, name
    assert float(norm) > 0 and ops.device_status(ws) == 0
    # a captured step beside the eager result that is still alive
    keep = [t.clone() for t in (h, dx, dpre, dpost, dgate, norm)]
    st, xx = torch.cuda.Stream(), x.clone()
    with torch.cuda.stream(st):
        step(xx)
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            out = step(xx)
        graph.replay()
        st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, keep))
