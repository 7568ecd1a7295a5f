"""Calls at the ends of what the training-step operators accept: outputs over
their inputs, two streams with one plan, offsets beyond 32 bits, the most rows."""
import numpy as np
import pytest
import torch

from route_permute_grouped_gb300 import ops

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _adapters(T, K, N, L, r, seed, f32=False):
    g = _gen(seed)
    bf = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(torch.bfloat16)
    cfg = ops.make_adapter_config(T, K, N, L, r, out_fp32=f32)
    idx = torch.randint(-1, L, (T,), generator=g, device="cuda").to(torch.int32)
    return cfg, idx, bf(T, K), bf(L, K, r, std=K ** -0.5), bf(L, r, N, std=0.3), torch.rand(L, generator=g, device="cuda") + 0.5


@pytest.mark.parametrize("T", [1, 70, 2000, 2048, 5000])
def test_adapter_onto_its_own_input(T):
    # a residual stream that an adapter is added to in place: x is read before a column of y is written
    cfg, idx, x, A, B, scale = _adapters(T, 512, 512, 3, 16, T)
    plan, ws = ops.adapter_plan(cfg, idx), ops.adapter_workspace(cfg)
    want = ops.adapter_fwd(cfg, x, A, B, scale, plan, base=x, ws=ws)
    keep = x.clone()
    assert ops.adapter_fwd(cfg, x, A, B, scale, plan, base=x, y=x, ws=ws) is x
    assert torch.equal(x, want) and (T == 1 or not torch.equal(x, keep))
    over = keep.clone()                     # without a base: x is only overwritten
    none = ops.adapter_fwd(cfg, keep, A, B, scale, plan, ws=ws)
    ops.adapter_fwd(cfg, over, A, B, scale, plan, y=over, ws=ws)
    assert torch.equal(over, none)


@pytest.mark.parametrize("E", [7, 64, 256])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_over_the_logits(E, score):
    T = 9000
    cfg = ops.make_balance_config(T, E, 2, n_seqs=3, score=score, z_coeff=1e-3)
    g = _gen(E)
    logits = torch.randn((T, E), generator=g, device="cuda") * 2
    idx = torch.randint(0, E, (T, 2), generator=g, device="cuda").to(torch.int32)
    off = torch.tensor([3, 4000, 4000, 8990], dtype=torch.int32, device="cuda")
    mask = torch.rand(T, generator=g, device="cuda") > 0.2
    stats = ops.balance_loss_fwd(cfg, logits, idx, off, mask)[2]
    want = ops.balance_loss_bwd(cfg, logits, stats, None, off, mask)
    assert ops.balance_loss_bwd(cfg, logits, stats, None, off, mask, dlogits=logits) is logits
    assert torch.equal(logits, want)


def test_one_plan_on_two_streams():
    T = 6000
    cfg, idx, x, A, B, scale = _adapters(T, 256, 512, 5, 32, 1)
    plan = ops.adapter_plan(cfg, idx)
    xs = [x, x.flip(0).contiguous()]
    dy = torch.randn((T, 512), generator=_gen(2), device="cuda").to(torch.bfloat16)
    u = [ops.alloc_adapter_saved(cfg) for _ in xs]
    ws = [ops.adapter_workspace(cfg, True) for _ in xs]

    def step(i):
        y = ops.adapter_fwd(cfg, xs[i], A, B, scale, plan, u=u[i], ws=ws[i])
        return [y, *ops.adapter_bwd(cfg, dy, xs[i], A, B, scale, plan, u[i], ws=ws[i]).values()]

    want = [[t.clone() for t in step(i)] for i in range(2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = step(i)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_two_graphs_with_one_workspace():
    # replayed in turn in one stream
    T = 3000
    cfg, idx, x, A, B, scale = _adapters(T, 256, 320, 4, 16, 3)
    ws, s, graphs = ops.adapter_workspace(cfg, True), torch.cuda.Stream(), []
    dy = torch.randn((T, 320), generator=_gen(4), device="cuda").to(torch.bfloat16)
    for k in range(2):
        ix, xx = (idx, x) if k == 0 else (idx.flip(0).contiguous(), x.flip(0).contiguous())
        plan, u = ops.adapter_plan(cfg, ix), ops.alloc_adapter_saved(cfg)

        def step():
            ops.adapter_plan(cfg, ix, plan=plan)
            y = ops.adapter_fwd(cfg, xx, A, B, scale, plan, u=u, ws=ws)
            g = ops.adapter_bwd(cfg, dy, xx, A, B, scale, plan, u, ws=ws)
            return [y, ops.grad_norm([g["dA"], g["dB"]], ws=norm_ws), *g.values()]

        norm_ws = ops.grad_norm_workspace() if k == 0 else norm_ws
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = step()
        graphs.append((graph, out, want))
    with torch.cuda.stream(s):
        for _ in range(5):
            for graph, _, _ in graphs:
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("L", [1, 3, 1024])
def test_the_most_rows(L):
    T = 1 << 21
    cfg = ops.make_adapter_config(T, 8, 8, L, 8, out_fp32=True)
    idx = torch.randint(-1, L, (T,), generator=_gen(L), device="cuda").to(torch.int32)
    one = torch.zeros((T, 8), dtype=torch.bfloat16, device="cuda")
    one[:, 0] = 1
    A = torch.zeros((L, 8, 8), dtype=torch.bfloat16, device="cuda")
    A[:, 0, 0] = 1
    B = torch.zeros((L, 8, 8), dtype=torch.bfloat16, device="cuda")
    at = torch.arange(L, device="cuda")
    B[:, 0, 0], B[:, 0, 1] = (at % 32 + 1).to(torch.bfloat16), (at // 32 + 1).to(torch.bfloat16)
    sc, plan, u = torch.ones(L, device="cuda"), ops.adapter_plan(cfg, idx), ops.alloc_adapter_saved(cfg)
    ws = ops.adapter_workspace(cfg, True)
    y = ops.adapter_fwd(cfg, one, A, B, sc, plan, u=u, ws=ws)
    live = (idx >= 0).float()
    assert torch.equal(y[:, 0], live * (idx % 32 + 1)) and torch.equal(y[:, 1], live * (idx // 32 + 1)) and not y[:, 2:].any()
    g = ops.adapter_bwd(cfg, one, one, A, B, sc, plan, u, ws=ws)
    count = torch.bincount(idx[idx >= 0].long(), minlength=L).float()
    assert torch.equal(g["dB"][:, 0, 0], count) and int(g["dB"].double().sum()) == int(count.double().sum())
    assert torch.equal(g["dA"][:, 0, 0], count * (at % 32 + 1)) and torch.equal(g["dx"][:, 0], y[:, 0])
    assert ops.device_status(plan) == 0 and ops.device_status(ws) == 0


def test_adapter_rows_beyond_32_bit_offsets():
    T, K, N, L, r = 560_001, 4096, 4096, 5, 16      # 2.3e9 elements in x, base, y and dx
    g = _gen(7)
    x, base = (torch.empty((T, 4096), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (x, base):
        for c in t.split(70_000):
            c.copy_(torch.randn(c.shape, generator=g, device="cuda"))
    cfg, idx, _, A, B, scale = _adapters(8, K, N, L, r, 5)
    cfg.T = T
    idx = torch.randint(-1, L, (T,), generator=g, device="cuda").to(torch.int32)
    plan, u, ws = ops.adapter_plan(cfg, idx), ops.alloc_adapter_saved(cfg), ops.adapter_workspace(cfg, True)
    y = ops.adapter_fwd(cfg, x, A, B, scale, plan, base=base, u=u, ws=ws)
    grads = ops.adapter_bwd(cfg, base, x, A, B, scale, plan, u, ws=ws)
    pick = torch.cat([torch.arange(40, device="cuda"), torch.randint(0, T, (80,), generator=g, device="cuda"),
                      torch.arange(T - 40, T, device="cuda")])
    for t in pick.tolist():
        a = int(idx[t])
        if a < 0:
            assert torch.equal(y[t], base[t]) and not grads["dx"][t].any()
            continue
        c = scale[a].double()
        up = c * (x[t].double() @ A[a].double())
        want = base[t].double() + up @ B[a].double()
        dwant = (c * (base[t].double() @ B[a].double().t())) @ A[a].double().t()
        # the stored bf16's half step, and 2^-8 of the row's scale for the sums ahead of it
        for got, ref in ((y[t], want), (grads["dx"][t], dwant)):
            assert bool(((got.double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + 2.0 ** -6 * ref.abs().max())).all())
    # column sums of the weight gradients against the same rows' products, one adapter
    q = torch.nonzero(idx == 2)[:, 0]
    du = scale[2].double() * torch.cat([base[p].double() @ B[2].double().t() for p in q.split(20_000)])
    dA = sum(x[p].double().t() @ d for p, d in zip(q.split(20_000), du.split(20_000)))
    # sums of 93000 products of both signs: fp32 runs and their joins, 2^-16 of the largest covers 256 half steps
    assert bool(((grads["dA"][2].double() - dA).abs() <= 2.0 ** -16 * dA.abs().max()).all())
    assert ops.device_status(ws) == 0


def test_balance_rows_beyond_32_bit_offsets():
    T, E = (1 << 23) + 3001, 256                     # 2.15e9 logits
    g = _gen(9)
    logits = torch.empty((T, E), device="cuda")
    for c in logits.split(1 << 20):
        c.copy_(torch.randn(c.shape, generator=g, device="cuda"))
    idx = torch.randint(0, E, (T, 2), generator=g, device="cuda").to(torch.int32)
    off = torch.tensor([0, 1 << 22, T - 100, T], dtype=torch.int32, device="cuda")
    cfg = ops.make_balance_config(T, E, 2, n_seqs=3, balance_coeff=1.0, z_coeff=1.0)
    losses, counts, stats = ops.balance_loss_fwd(cfg, logits, idx, off)
    d = ops.balance_loss_bwd(cfg, logits, stats, None, off)
    z, balance = 0.0, 0.0
    for s, (a, b) in enumerate(zip(off.tolist()[:-1], off.tolist()[1:])):
        c = torch.bincount(idx[a:b].reshape(-1).long(), minlength=E)
        assert torch.equal(counts[s].long(), c)
        P = torch.zeros(E, dtype=torch.float64, device="cuda")
        for part in logits[a:b].split(1 << 18):
            l = part.double()
            z += float((torch.logsumexp(l, 1) ** 2).sum())
            P += torch.softmax(l, 1).sum(0)
        f = c.double() * E / (2 * (b - a))
        balance += float((f * P / (b - a)).sum()) / 3
        for t in (a, a + 1, (a + b) // 2, b - 1):
            l = logits[t].double()
            p, w = torch.softmax(l, 0), f / (3 * (b - a))
            lz = 2 / T * torch.logsumexp(l, 0)
            ref = p * (w - (p * w).sum()) + lz * p
            size = p * (w + (p * w).sum()) + lz.abs() * p
            assert bool(((d[t].double() - ref).abs() <= 128 * HALF * size).all())
    assert abs(float(losses[1]) - z / T) <= 160 * HALF * z / T and abs(float(losses[0]) - balance) <= 160 * HALF * balance


def test_gradients_beyond_32_bit_offsets():
    n = (1 << 31) + 4097
    t = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    g = _gen(11)
    for c in t.split(1 << 26):
        c.copy_(torch.randn(c.shape, generator=g, device="cuda"))
    want = float(torch.stack([c.double().square().sum() for c in t.split(1 << 26)]).sum().sqrt())
    ends = [t[:5000].clone(), t[-5000:].clone()]
    norm = ops.clip_grad_norm([t[1:]], 1e9)
    first = float(t[0]) ** 2
    assert abs(float(norm) ** 2 + first - want ** 2) <= 40 * HALF * want ** 2
    norm = ops.clip_grad_norm([t], 10.0)
    assert abs(float(norm) - want) <= 18 * HALF * want
    for got, was in zip((t[:5000], t[-5000:]), ends):
        ref = was.double() * (10.0 / (want + 1e-6))
        assert bool(((got.double() - ref).abs() <= (24 * HALF + 2.0 ** -8) * ref.abs()).all())
