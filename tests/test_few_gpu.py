"""The whole layer for a few tokens, with bf16 and with MXFP4 weights, against the
fp64 oracle. The bounds are the oracle's: what the tensor cores' and the fp32 sums
and the activations' parts may add at most, and half a step of y's type."""
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


class Layer:
    """Inputs of one call and its config."""

    def __init__(self, T, H, E, k, F, Fs=0, mxfp4=False, bias=False, lbias=False, seed=0, **cfg):
        g = torch.Generator("cuda").manual_seed(seed * 7919 + T * 131 + H + E)
        r = lambda *s, std=1.0: torch.randn(s, generator=g, device="cuda") * std
        self.x = r(T, H).to(BF)
        self.router_w = r(E, H, std=1.5 * H ** -0.5).to(BF)
        self.W = [r(E, H, F, std=H ** -0.5).to(BF), r(E, H, F, std=H ** -0.5).to(BF), r(E, F, H, std=F ** -0.5).to(BF)]
        self.Ws = [r(H, Fs, std=H ** -0.5).to(BF), r(H, Fs, std=H ** -0.5).to(BF), r(Fs, H, std=Fs ** -0.5).to(BF)] if Fs else None
        self.eb = 0.2 * torch.rand(E, generator=g, device="cuda") - 0.1 if bias else None
        self.lb = r(E) if lbias else None
        self.mx = mxfp4
        self.cfg = ops.make_config(T, H, E, k, F, F_shared=Fs, **cfg)
        self.opts = {n: cfg[n] for n in ("score", "n_groups", "topk_groups", "gate_scale", "force_balanced") if n in cfg}
        self.out_fp32 = cfg.get("out_fp32", False)
        self.q = ops.mx4_quantize_weights(self.cfg, *self.W, Ws=self.Ws) if mxfp4 else None

    def run(self, x=None, ws=None, y=None):
        x = self.x if x is None else x
        ws = ops.few_workspace(self.cfg, mxfp4=self.mx) if ws is None else ws
        if self.mx:
            out = ops.layer_few_fwd_mxfp4(self.cfg, x, self.router_w, self.q, expert_bias=self.eb, logit_bias=self.lb, ws=ws, y=y)
        else:
            out = ops.layer_few_fwd(self.cfg, x, self.router_w, *self.W, expert_bias=self.eb, logit_bias=self.lb, Ws=self.Ws,
                                    ws=ws, y=y)
        return out

    def oracle(self, x=None):
        f = lambda ts: None if ts is None else [_f64(t) for t in ts]
        return DO.few_layer(_f64(self.x if x is None else x), _f64(self.router_w), *f(self.W), self.cfg.k, Ws=f(self.Ws),
                            out_fp32=self.out_fp32, mxfp4=self.mx, expert_bias=_f64(self.eb), logit_bias=_f64(self.lb), **self.opts)

    def check(self, out, want=None):
        y, idx, gate = out
        want = self.oracle() if want is None else want
        assert np.array_equal(idx.cpu().numpy(), want["topk_idx"])
        assert (np.abs(_f64(gate) - want["topk_gate"]) <= want["dgate"]).all()
        err, half = np.abs(_f64(y) - want["y"]), HALF[y.dtype]
        lim = want["dy"] * (1 + half) + half * np.abs(want["y"]) + 1e-37
        assert (err <= lim).all(), float((err / lim).max())


FORMS = [dict(), dict(mxfp4=True), dict(out_fp32=True), dict(mxfp4=True, out_fp32=True)]


def _run(form, T, H, E, k, F, **kw):
    d = {**form, **kw}
    L = Layer(T, H, E, k, F, **d)
    ws = ops.few_workspace(L.cfg, mxfp4=L.mx)
    ws[256:] = 0x7f                       # what an earlier user of the memory left
    L.check(L.run(ws=ws))
    assert ops.device_status(ws) == 0 and not ws[:256].any()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T", [1, 2, 3, 7, 8, 9, 16, 17, 33, 64])
def test_tokens(form, T):
    _run(form, T, 256, 8, 2, 256)


# one tile, odd tiles, tiles cut by many blocks, more tiles than blocks, k sub-blocks that end inside a stage
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,H,E,k,F", [(1, 128, 1, 1, 128), (4, 128, 4, 4, 128), (5, 384, 5, 3, 640), (2, 2048, 16, 4, 384),
                                       (3, 128, 3, 1, 4096), (2, 4096, 2, 2, 128), (61, 384, 33, 5, 384), (6, 256, 256, 8, 128),
                                       (64, 256, 40, 16, 256)])
def test_shapes(form, T, H, E, k, F):
    _run(form, T, H, E, k, F)


@pytest.mark.parametrize("T,H,E,k,F", [(1, 64, 2, 1, 64), (9, 192, 7, 3, 320), (64, 64, 4, 2, 64), (2, 1088, 12, 4, 192)])
def test_multiples_of_64(T, H, E, k, F):
    _run(dict(), T, H, E, k, F)
    _run(dict(out_fp32=True), T, H, E, k, F, Fs=192)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T", [1, 13, 64])
@pytest.mark.parametrize("Fs", [128, 640])
def test_shared_expert(form, T, Fs):
    _run(form, T, 256, 8, 2, 128, Fs=Fs)


@pytest.mark.parametrize("T", [2, 40])
@pytest.mark.parametrize("opts", [dict(score="sigmoid", bias=True, gate_scale=2.5), dict(score="softmax", bias=True, lbias=True),
                                  dict(score="sigmoid", n_groups=8, topk_groups=3, bias=True),
                                  dict(score="softmax", n_groups=4, topk_groups=2), dict(score="softmax", n_groups=32, topk_groups=9),
                                  dict(force_balanced=True, gate_scale=0.5), dict(score="sigmoid", force_balanced=True, lbias=True)])
def test_routers(T, opts):
    _run(dict(), T, 256, 32, 6, 128, **opts)


@pytest.mark.parametrize("form", FORMS)
def test_all_tokens_to_one_expert(form):
    # 64 rows of one expert: with MXFP4 more than an accumulator holds, so that the expert is taken in parts
    L = Layer(64, 256, 8, 1, 256, lbias=True, **form)
    L.lb.zero_()
    L.lb[5] = 50.0
    out = L.run()
    assert (out[1] == 5).all()
    L.check(out)


def test_ties_go_to_the_lower_expert():
    L = Layer(3, 128, 16, 4, 128)
    L.router_w[1::2] = L.router_w[0::2]
    out = L.run()
    L.check(out)
    L.router_w.zero_()
    out = L.run()
    assert (out[1].cpu() == torch.arange(4)).all() and torch.allclose(out[2], torch.full_like(out[2], 0.25))


@pytest.mark.parametrize("mxfp4", [False, True])
@pytest.mark.parametrize("T", [6, 30])
def test_infinities_and_nans_reach_their_own_rows_only(mxfp4, T):
    L = Layer(T, 256, 8, 2, 128, Fs=128, mxfp4=mxfp4)
    clean = L.run()
    x = L.x.clone()
    x[1, 7], x[4, 100] = float("nan"), float("inf")
    y, idx, gate = L.run(x=x)
    keep = [t for t in range(T) if t not in (1, 4)]
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(idx[keep], clean[1][keep]) and torch.equal(gate[keep], clean[2][keep])
    assert torch.isnan(y[1].float()).all() and not torch.isfinite(y[4].float()).all()
    assert int(idx.min()) >= 0 and int(idx.max()) < 8


def test_zero_tokens_rows():
    L = Layer(5, 256, 8, 2, 128, mxfp4=True)
    L.x[2] = 0
    out = L.run()
    assert not out[0][2].any()
    L.check(out)


@pytest.mark.parametrize("mxfp4", [False, True])
def test_large_and_small_values(mxfp4):
    for scale in (2.0 ** 40, 2.0 ** -60):
        L = Layer(4, 256, 8, 2, 256, mxfp4=mxfp4)
        x = L.x * scale
        L.router_w /= scale
        want = L.oracle(x=x)
        L.check(L.run(x=x), want)


@pytest.mark.parametrize("mxfp4", [False, True])
def test_y_over_x(mxfp4):
    L = Layer(20, 512, 8, 2, 256, Fs=128, mxfp4=mxfp4)
    want = L.run()
    x = L.x.clone()
    y, idx, gate = L.run(x=x, y=x)
    assert y is x and torch.equal(y, want[0]) and torch.equal(idx, want[1])


@pytest.mark.parametrize("form", FORMS)
def test_the_same_bits_every_time(form):
    L = Layer(27, 1024, 24, 4, 640, Fs=256, **form)
    ws = ops.few_workspace(L.cfg, mxfp4=L.mx)
    want = [t.clone() for t in L.run(ws=ws)]
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(want, L.run(ws=ws)))


def test_as_the_layer_of_any_length():
    # the same computation as layer_fwd, whose intermediates are bf16
    L = Layer(48, 512, 16, 4, 256, Fs=128, score="sigmoid", bias=True)
    y, idx, gate = L.run()
    ref = ops.layer_fwd(L.cfg, L.x, L.router_w, *L.W, expert_bias=L.eb, Ws=L.Ws)
    assert float((y.float() - ref.float()).norm() / ref.float().norm()) < 6e-3


def test_two_streams_two_workspaces():
    a, b = Layer(5, 1024, 16, 4, 512), Layer(9, 768, 8, 2, 384, mxfp4=True)
    wa, wb = a.run()[0].clone(), b.run()[0].clone()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    ws = [ops.few_workspace(a.cfg), ops.few_workspace(b.cfg, mxfp4=True)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        with torch.cuda.stream(sa):
            ya = a.run(ws=ws[0])[0]
        with torch.cuda.stream(sb):
            yb = b.run(ws=ws[1])[0]
        got.append((ya, yb))
    torch.cuda.synchronize()
    assert all(torch.equal(x, wa) and torch.equal(y, wb) for x, y in got)


@pytest.mark.parametrize("mxfp4", [False, True])
def test_captured_and_replayed_with_other_inputs(mxfp4):
    L = Layer(12, 512, 16, 4, 256, mxfp4=mxfp4)
    xs = [L.x.clone(), Layer(12, 512, 16, 4, 256, seed=5).x]
    want = [[t.clone() for t in L.run(x=x)] for x in xs]
    ws, st, x = ops.few_workspace(L.cfg, mxfp4=mxfp4), torch.cuda.Stream(), L.x.clone()
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            first = L.run(x=x, ws=ws)
            second = L.run(x=x, ws=ws)
        for i in (0, 1, 0):
            x.copy_(xs[i])
            graph.replay()
            st.synchronize()
            for out in (first, second):
                assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


def test_inputs_written_right_before_and_overwritten_right_after():
    L = Layer(3, 1024, 16, 4, 512)
    want = L.run()[0].clone()
    x, keep = torch.zeros_like(L.x), L.x.clone()
    ws = ops.few_workspace(L.cfg)
    for _ in range(5):
        x.copy_(keep)
        y = L.run(x=x, ws=ws)[0]
        x.fill_(float("nan"))
        assert torch.equal(y, want)


def test_scratch_lent_to_other_operators():
    L = Layer(10, 256, 8, 2, 128)
    want = L.run()[0].clone()
    n = max(ops.few_workspace(L.cfg).numel(), ops.grad_norm_workspace().numel(), ops.workspace(L.cfg).numel())
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    t = torch.randn(100000, device="cuda")
    norm = ops.grad_norm([t]).clone()
    for _ in range(3):
        assert torch.equal(L.run(ws=ws)[0], want) and not ws[:256].any()
        assert torch.equal(ops.grad_norm([t], ws=ws), norm)


@pytest.mark.parametrize("T,Fs,mxfp4", [(2, 0, False), (20, 256, False), (20, 256, True)])
def test_a_wait_that_runs_out_is_reported(T, Fs, mxfp4):
    L = Layer(T, 1024, 8, 2, 512, Fs=Fs, mxfp4=mxfp4)
    ws = ops.few_workspace(L.cfg, mxfp4=mxfp4)
    want = L.run(ws=ws)[0].clone()
    ops.set_wait_limit_ns(2_000_000)
    ops.set_fault(1)                      # the first block does not arrive: the others' waits end after 2 ms
    try:
        L.run(ws=ws)
        torch.cuda.synchronize()
    finally:
        ops.set_fault(0)
        ops.set_wait_limit_ns(0)
    assert ops.device_status(ws) == ops.MOE_ERR_DEVICE_TIMEOUT
    assert torch.equal(L.run(ws=ws)[0], want) and ops.device_status(ws) == 0 and not ws[:256].any()


def test_refusals():
    L = Layer(4, 128, 8, 2, 128, Fs=128)
    args = (L.cfg, L.x, L.router_w, *L.W)
    ws = ops.few_workspace(L.cfg)
    for over in (dict(T=65), dict(H=130), dict(F=96), dict(E=257), dict(k=17), dict(k=9, E=8)):
        d = {**dict(T=4, H=128, E=8, k=2, F=128), **over}
        with pytest.raises(ops.MoeError):
            ops.few_workspace(ops.make_config(**d))
    for d in (dict(T=4, H=192, E=8, k=2, F=128), dict(T=4, H=128, E=8, k=2, F=192), dict(T=4, H=128, E=8, k=2, F=128, F_shared=64)):
        ops.few_workspace(ops.make_config(**d))
        with pytest.raises(ops.MoeError):
            ops.few_workspace(ops.make_config(**d), mxfp4=True)
    bad = [(L.cfg, L.x[:3].contiguous(), *args[2:]), (L.cfg, L.x.float(), *args[2:]), (*args[:2], L.router_w.cpu(), *args[3:]),
           (*args[:3], L.W[0][:, :, ::2], *args[4:]), (*args[:5], L.W[0])]
    for a in bad[:4]:
        with pytest.raises(ops.MoeError):
            ops.layer_few_fwd(*a, Ws=L.Ws, ws=ws)
    with pytest.raises(ops.MoeError):
        ops.layer_few_fwd(*args, ws=ws)                  # no shared expert's weights
    with pytest.raises(ops.MoeError):
        ops.layer_few_fwd(*args, Ws=L.Ws, ws=ws[:-1])
    with pytest.raises(ops.MoeError):
        ops.layer_few_fwd(*args, Ws=L.Ws, ws=ws, y=torch.empty((4, 128), device="cuda"))
    q = ops.mx4_quantize_weights(L.cfg, *L.W, Ws=L.Ws)
    with pytest.raises(ops.MoeError):
        ops.layer_few_fwd_mxfp4(L.cfg, L.x, L.router_w, {n: q[n] for n in ("w13", "w2")})
    with pytest.raises(ops.MoeError):
        ops.layer_few_fwd_mxfp4(L.cfg, L.x, L.router_w, {**q, "w13": q["w13"][:-16]})
