"""The training-step operators together with the layer, as a fine-tuning step
uses them: layer forward, adapters on the layer's output, router losses, their
gradients through the layer's backward, one norm over every gradient, clipping.
The layer's own terms are covered elsewhere; here the joints are."""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import train_oracle as TO
from route_permute_grouped_gb300 import ops, synth
from tests._util import assert_close, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


def _layer(T, prec="bf16", **over):
    ls = synth.shape("tiny", T=T, H=256, E=8, k=2, F=256, **over)
    d = synth.make_layer(ls, seed=5, device="cuda", training=True)
    cfg = ops.config_from_shape(ls, out_fp32=True)
    return ls, d, cfg


def _bwd(prec, cfg, d, saved_fwd=None):
    """(saved, call(dlogits) -> grads) after a training forward."""
    if prec == "bf16":
        saved, ws = ops.alloc_saved(cfg), ops.workspace(cfg, True)
        ops.layer_fwd(cfg, d["x"], d["router_w"], d["W1"], d["W3"], d["W2"], saved=saved, ws=ws)
        return saved, lambda dl: ops.layer_bwd(cfg, d["dO"], d["x"], d["router_w"], d["W1"], d["W3"], d["W2"], saved,
                                               ws=ws, dlogits=dl)
    if prec == "mxfp8":
        wf = ops.mx_quantize_weights(cfg, d["W1"], d["W3"], d["W2"])
        wb = ops.mx_quantize_bwd_weights(cfg, d["W1"], d["W3"], d["W2"])
        saved, ws = ops.alloc_saved_mxfp8(cfg), ops.mx_train_workspace(cfg)
        ops.layer_fwd_mxfp8_train(cfg, d["x"], d["router_w"], wf, saved, ws=ws)
        return saved, lambda dl: ops.layer_bwd_mxfp8(cfg, d["dO"], d["x"], d["router_w"], wb, saved, ws=ws, dlogits=dl)
    fw, bw = ops.nv_quantize_train_weights(cfg, d["W1"], d["W3"], d["W2"])
    saved, ws = ops.alloc_saved(cfg), ops.nv_train_workspace(cfg)
    ops.layer_fwd_nvfp4_train(cfg, d["x"], d["router_w"], fw, saved, ws=ws)
    return saved, lambda dl: ops.layer_bwd_nvfp4(cfg, d["dO"], d["x"], d["router_w"], bw, saved, ws=ws, dlogits=dl)


@pytest.mark.parametrize("prec", ["bf16", "mxfp8", "nvfp4"])
def test_outside_gradient_of_the_logits(prec):
    # dlogits adds dlogits W_r to dx and dlogits^T x to dW_r and leaves the rest as it is
    ls, d, cfg = _layer(300)
    _, call = _bwd(prec, cfg, d)
    plain = {k: v.clone() for k, v in call(None).items()}
    zero = {k: v.clone() for k, v in call(torch.zeros((300, 8), device="cuda")).items()}
    for k in plain:
        assert torch.equal(plain[k], zero[k]), k
    g = torch.Generator(device="cuda").manual_seed(1)
    dl = torch.randn((300, 8), generator=g, device="cuda")
    got = call(dl)
    for k in ("dW1", "dW3", "dW2"):
        assert torch.equal(plain[k], got[k]), k
    # the logits' gradient enters the router's GEMMs as two bf16 parts
    assert_close("dx", f64(got["dx"]) - f64(plain["dx"]), f64(dl) @ f64(d["router_w"]), rel=1e-4, atol=2e-4)
    assert_close("dW_r", f64(got["dW_r"]) - f64(plain["dW_r"]), f64(dl).T @ f64(d["x"]), rel=1e-4, atol=2e-3)


def test_balance_gradient_is_the_layers_aux_gradient():
    # one sequence and softmax: the loss outside the layer replaces aux_coeff
    ls, d, with_aux = _layer(500, aux_coeff=0.05)
    _, _, without = _layer(500, aux_coeff=0.0)
    saved, call = _bwd("bf16", with_aux, d)
    inside = call(None)
    saved, call = _bwd("bf16", without, d)
    bc = ops.make_balance_config(500, 8, 2, balance_coeff=0.05)
    losses, counts, stats = ops.balance_loss_fwd(bc, saved["logits"], saved["topk_idx"])
    outside = call(ops.balance_loss_bwd(bc, saved["logits"], stats))
    assert torch.equal(counts[0], saved["counts"])
    assert abs(float(losses[0]) - float(inside["aux_loss"])) <= 1e-5 * float(losses[0])
    for k in ("dx", "dW_r", "dW1"):
        # the same terms, summed in another order before two bf16 parts are taken
        assert_close(k, f64(outside[k]), f64(inside[k]), rel=1e-4, atol=1e-4)


def test_fine_tuning_step_and_its_graph():
    T = 700
    ls, d, cfg = _layer(T, aux_coeff=0.0)
    L, r = 5, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    bf = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(torch.bfloat16)
    A, B = bf(L, 256, r, std=1 / 16), bf(L, r, 256, std=0.25)
    scale = torch.linspace(0.5, 1.5, L, device="cuda")
    idx = torch.randint(-1, L, (T,), generator=g, device="cuda").to(torch.int32)
    off = torch.tensor([0, 250, 251, 690], dtype=torch.int32, device="cuda")
    mask = torch.rand(T, generator=g, device="cuda") > 0.1
    acfg = ops.make_adapter_config(T, 256, 256, L, r, out_fp32=True)
    bcfg = ops.make_balance_config(T, 8, 2, n_seqs=3, balance_coeff=0.5, z_coeff=0.1)
    ws, aws, bws, gws = (ops.workspace(cfg, True), ops.adapter_workspace(acfg, True), ops.balance_workspace(bcfg),
                         ops.grad_norm_workspace())
    saved, u, grads, ag = ops.alloc_saved(cfg), ops.alloc_adapter_saved(acfg), ops.alloc_grads(cfg), ops.alloc_adapter_grads(acfg)
    y = torch.empty((T, 256), device="cuda")
    plan = ops.adapter_plan(acfg, idx)
    raw = [grads["dW_r"], grads["dW1"], grads["dW3"], grads["dW2"], ag["dA"], ag["dB"]]
    clipped = [torch.empty_like(t) for t in raw]
    tl = ops.tensor_list(raw, out=clipped)

    def step():
        ops.layer_fwd(cfg, d["x"], d["router_w"], d["W1"], d["W3"], d["W2"], saved=saved, ws=ws, y=y)
        ops.adapter_plan(acfg, idx, plan=plan)
        ops.adapter_fwd(acfg, d["x"], A, B, scale, plan, base=y, y=y, u=u, ws=aws)
        losses, counts, stats = ops.balance_loss_fwd(bcfg, saved["logits"], saved["topk_idx"], off, mask, ws=bws)
        dl = ops.balance_loss_bwd(bcfg, saved["logits"], stats, None, off, mask)
        ops.layer_bwd(cfg, d["dO"], d["x"], d["router_w"], d["W1"], d["W3"], d["W2"], saved, ws=ws, grads=grads,
                      dlogits=dl)
        ops.adapter_bwd(acfg, d["dO"], d["x"], A, B, scale, plan, u, dx_base=grads["dx"],
                        grads={**ag, "dx": grads["dx"]}, ws=aws)
        return losses, ops.clip_grad_norm(tl, 0.5, ws=gws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        losses, norm = (t.clone() for t in step())
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for w in (ws, aws, bws, plan):
        assert ops.device_status(w) == 0

    # against the oracles
    ref = O.layer_bwd(f64(d["x"]), f64(d["router_w"]), f64(d["W1"]), f64(d["W3"]), f64(d["W2"]), f64(d["dO"]), 2)
    fw = O.layer_fwd(f64(d["x"]), f64(d["router_w"]), f64(d["W1"]), f64(d["W3"]), f64(d["W2"]), 2)
    logits = f64(d["x"]) @ f64(d["router_w"]).T
    bl, _, bd, _ = TO.balance(logits, ref["topk_idx"], 2, "softmax", 0.5, 0.1, off.tolist(), f64(mask))
    ad, _ = TO.adapter(f64(d["x"]), f64(A), f64(B), f64(scale), idx.cpu().numpy(), fw["y"], f64(d["dO"]),
                       ref["dx"] + bd @ f64(d["router_w"]))
    assert np.allclose(f64(losses), bl, rtol=1e-4)
    assert_close("y", f64(y), ad["y"])
    assert_close("dx", f64(grads["dx"]), ad["dx"])
    assert_close("dW_r", f64(grads["dW_r"]), ref["dW_r"] + bd.T @ f64(d["x"]), atol=5e-2)
    assert_close("dA", f64(ag["dA"]), ad["dA"])
    assert_close("dB", f64(ag["dB"]), ad["dB"])
    n, want = TO.clip([f64(t) for t in raw], 0.5)
    assert abs(float(norm) - n) <= 1e-6 * n
    for t, w in zip(clipped, want):
        assert np.max(np.abs(f64(t) - w)) <= 2e-6 * np.abs(w).max()

    # captured: the same bits
    eager = [t.clone() for t in (y, grads["dx"], *raw, *clipped)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        glosses, gnorm = step()
    for t in (y, *raw, *clipped):
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(glosses, losses) and torch.equal(gnorm, norm)
    for a, b in zip(eager, (y, grads["dx"], *raw, *clipped)):
        assert torch.equal(a, b)
