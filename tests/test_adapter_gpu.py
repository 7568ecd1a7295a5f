"""Low-rank adapters of many requests against the fp64 oracle, element by
element.

Tolerances. bf16 products are exact in fp32. A sum of n of them is joined from
blocks of 64: inside a block the tensor cores may cut each of the (at most 64)
additions at the last fp32 bit of the running sum (2^-23 of it), the blocks and
the split parts are added in fp32: (64 + n / 64 + 32) * 2^-23 of the sum of
magnitudes. u and du enter their second product as two bf16 parts, 2^-17 of
them at most. The stored result is off by half a step more: bf16 2^-8, fp32
2^-24."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as TO
from route_permute_grouped_gb300 import ops

pytestmark = pytest.mark.gpu
STEP, SPLIT = 2.0 ** -23, 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


def _bf(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _inputs(T, K, N, L, r, seed, f32=False):
    rng = np.random.default_rng(seed)
    d = {"x": _bf(rng.normal(size=(T, K))), "A": _bf(rng.normal(size=(L, K, r)) * K ** -0.5),
         "B": _bf(rng.normal(size=(L, r, N)) * r ** -0.5), "dy": _bf(rng.normal(size=(T, N))),
         "scale": torch.from_numpy(rng.uniform(0.5, 2, L).astype(np.float32)),
         "base": torch.from_numpy(rng.normal(size=(T, N)).astype(np.float32)),
         "dx_base": torch.from_numpy(rng.normal(size=(T, K)).astype(np.float32))}
    if not f32:
        d["base"], d["dx_base"] = d["base"].to(torch.bfloat16), d["dx_base"].to(torch.bfloat16)
    return d


def _sum_err(n):
    return (64 + n / 64 + 32) * STEP


def _check(name, got, want, err):
    bad = np.abs(got - want) > err
    assert not bad.any(), (name, int(bad.sum()), float(np.max(np.abs(got - want) / np.maximum(err, 1e-300))))


def _compare(d, idx, f32=False, cfg=None, train=True):
    T, K = d["x"].shape
    L, r, N = d["B"].shape
    cfg = ops.make_adapter_config(T, K, N, L, r, out_fp32=f32)
    c = {k: v.cuda() for k, v in d.items()}
    ix = torch.from_numpy(np.asarray(idx, np.int32)).cuda()
    ws = ops.adapter_workspace(cfg, training=train)
    plan = ops.adapter_plan(cfg, ix)
    u = ops.alloc_adapter_saved(cfg) if train else None
    y = ops.adapter_fwd(cfg, c["x"], c["A"], c["B"], c["scale"], plan, base=c["base"], u=u, ws=ws)
    h = {k: _f64(v) for k, v in d.items()}
    ref, size = TO.adapter(h["x"], h["A"], h["B"], h["scale"], np.asarray(idx), h["base"],
                           h["dy"] if train else None, h["dx_base"] if train else None)
    out = 2.0 ** -24 if f32 else 2.0 ** -8
    a = np.asarray(idx)
    live = (a >= 0) & (a < L)
    Bm, Am = np.abs(h["B"])[np.where(live, a, 0)], np.abs(h["A"])[np.where(live, a, 0)]
    e_u = size["u"] * _sum_err(K)                       # zero rows where no adapter is
    e_y = np.einsum("tr,trn->tn", e_u + size["us"] * (SPLIT + _sum_err(r)), Bm) * (1 + STEP)
    _check("y", _f64(y), ref["y"], e_y * (1 + out) + out * np.abs(ref["y"]) + 2 * STEP * np.abs(h["base"]) * live[:, None])
    assert np.array_equal(_f64(y)[~live], h["base"][~live])
    if train:
        g = ops.adapter_bwd(cfg, c["dy"], c["x"], c["A"], c["B"], c["scale"], plan, u, dx_base=c["dx_base"], ws=ws)
        e_du = size["du"] * _sum_err(N)
        e_dx = np.einsum("tr,tkr->tk", e_du + size["dus"] * (SPLIT + _sum_err(r)), Am) * (1 + STEP)
        _check("dx", _f64(g["dx"]), ref["dx"],
               e_dx * (1 + out) + out * np.abs(ref["dx"]) + 2 * STEP * np.abs(h["dx_base"]) * live[:, None])
        assert np.array_equal(_f64(g["dx"])[~live], h["dx_base"][~live])
        for l in range(L):
            q = np.nonzero(a == l)[0]
            n = len(q)
            e_a = np.abs(h["x"][q]).T @ (e_du[q] + size["dus"][q] * (SPLIT + _sum_err(n)))
            e_b = (e_u[q] + size["us"][q] * (SPLIT + _sum_err(n))).T @ np.abs(h["dy"][q])
            _check(f"dA[{l}]", _f64(g["dA"][l]), ref["dA"][l], e_a + 2.0 ** -24 * np.abs(ref["dA"][l]))
            _check(f"dB[{l}]", _f64(g["dB"][l]), ref["dB"][l], e_b + 2.0 ** -24 * np.abs(ref["dB"][l]))
    assert ops.device_status(plan) == 0 and ops.device_status(ws) == 0


def _idx(T, L, seed, none=0.1):
    rng = np.random.default_rng(seed)
    return np.where(rng.random(T) < none, -1 - rng.integers(0, 5, T), rng.integers(0, L, T))


@pytest.mark.parametrize("r", [8, 16, 24, 32, 48, 64, 72, 128])
def test_ranks(r):
    _compare(_inputs(150, 136, 200, 3, r, r), _idx(150, 3, r))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 96, 128])
def test_ranks_of_larger_batches(r, f32):
    _compare(_inputs(2100, 200, 328, 3, r, r, f32), _idx(2100, 3, r), f32)


@pytest.mark.parametrize("T,K,N,L,r", [(513, 1160, 648, 2, 16), (2500, 136, 2056, 1, 64), (3000, 72, 88, 700, 8),
                                       (5000, 264, 40, 2, 32), (2050, 2056, 1032, 5, 128), (2300, 1160, 136, 1024, 24)])
def test_long_axes_and_many_segments(T, K, N, L, r):
    # sums longer than an accumulator's turn, several runs of rows for an adapter, adapters of a few rows
    _compare(_inputs(T, K, N, L, r, T), _idx(T, L, T, none=0.02))


@pytest.mark.parametrize("T", [1023, 1024, 1025, 2047, 2048, 2049])
def test_both_forms_agree_at_their_border(T):
    idx = np.sort(_idx(T, 3, T, none=0.0))
    _compare(_inputs(T, 128, 128, 3, 16, T), idx)
    _compare(_inputs(T, 128, 128, 3, 16, T), np.full(T, 2))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,K,N,L", [(1, 8, 8, 1), (1, 1024, 136, 5), (2, 64, 64, 1), (15, 72, 88, 40), (64, 128, 256, 1),
                                     (65, 264, 120, 2), (130, 520, 504, 200), (700, 200, 328, 4), (1024, 64, 64, 1024),
                                     (1025, 72, 64, 33), (2500, 256, 192, 3)])
def test_sizes(T, K, N, L, f32):
    _compare(_inputs(T, K, N, L, 16, T + K, f32), _idx(T, L, T), f32)


@pytest.mark.parametrize("idx", [[0] * 200, [-1] * 200, [2] * 100 + [-1] * 100, list(range(3)) * 66 + [0, 1],
                                 [1] * 64 + [0] * 65 + [-5] * 7 + [2] * 64])
def test_distributions(idx):
    _compare(_inputs(200, 96, 80, 3, 32, 1), idx)


def test_serving_form_without_saved_state():
    _compare(_inputs(33, 640, 256, 9, 16, 2), _idx(33, 9, 3), train=False)


def test_in_place_and_without_a_base():
    d = _inputs(90, 128, 136, 4, 16, 7)
    c = {k: v.cuda() for k, v in d.items()}
    idx = torch.from_numpy(_idx(90, 4, 1, none=0.3).astype(np.int32)).cuda()
    cfg = ops.make_adapter_config(90, 128, 136, 4, 16)
    plan, u = ops.adapter_plan(cfg, idx), ops.alloc_adapter_saved(cfg)
    y = ops.adapter_fwd(cfg, c["x"], c["A"], c["B"], c["scale"], plan, base=c["base"], u=u)
    inp = c["base"].clone()
    assert ops.adapter_fwd(cfg, c["x"], c["A"], c["B"], c["scale"], plan, base=inp, y=inp) is inp
    assert torch.equal(inp, y)
    zero = ops.adapter_fwd(cfg, c["x"], c["A"], c["B"], c["scale"], plan, base=torch.zeros_like(inp))
    none = ops.adapter_fwd(cfg, c["x"], c["A"], c["B"], c["scale"], plan)
    assert torch.equal(zero, none) and not none[idx < 0].any()
    g = ops.adapter_bwd(cfg, c["dy"], c["x"], c["A"], c["B"], c["scale"], plan, u, dx_base=c["dx_base"])
    grads = ops.alloc_adapter_grads(cfg)
    grads["dx"].copy_(c["dx_base"])
    ops.adapter_bwd(cfg, c["dy"], c["x"], c["A"], c["B"], c["scale"], plan, u, dx_base=grads["dx"], grads=grads)
    for k in g:
        assert torch.equal(g[k], grads[k])


def test_rows_do_not_leak_into_each_other():
    # a row of NaN or infinities touches its own results and its adapter's
    # gradients only; rows without an adapter may hold anything
    d = _inputs(140, 128, 64, 3, 16, 4)
    idx = _idx(140, 3, 8)
    idx[[5, 77]] = [1, -1]
    c = {k: v.cuda() for k, v in d.items()}
    ix = torch.from_numpy(idx.astype(np.int32)).cuda()
    cfg = ops.make_adapter_config(140, 128, 64, 3, 16)

    def go(x, dy):
        plan, u = ops.adapter_plan(cfg, ix), ops.alloc_adapter_saved(cfg)
        y = ops.adapter_fwd(cfg, x, c["A"], c["B"], c["scale"], plan, base=c["base"], u=u)
        return {"y": y, **ops.adapter_bwd(cfg, dy, x, c["A"], c["B"], c["scale"], plan, u, dx_base=c["dx_base"])}

    want = go(c["x"], c["dy"])
    for bad in (float("nan"), float("inf")):
        x, dy = c["x"].clone(), c["dy"].clone()
        x[77], dy[77] = bad, bad      # no adapter
        got = go(x, dy)
        for k in want:
            assert torch.equal(want[k], got[k]), k
        x[5], dy[5] = bad, bad        # adapter 1
        got = go(x, dy)
        keep = torch.arange(140, device="cuda") != 5
        assert torch.equal(want["y"][keep], got["y"][keep]) and torch.equal(want["dx"][keep], got["dx"][keep])
        assert not torch.isfinite(got["y"][5]).any() and not torch.isfinite(got["dx"][5]).any()
        for l in (0, 2):
            assert torch.equal(want["dA"][l], got["dA"][l]) and torch.equal(want["dB"][l], got["dB"][l])
        assert torch.isnan(got["dA"][1]).all() or not torch.isfinite(got["dA"][1]).any()


def test_an_index_out_of_range_counts_as_none_and_is_reported():
    d = _inputs(70, 64, 64, 3, 8, 5)
    c = {k: v.cuda() for k, v in d.items()}
    idx = np.arange(70) % 3
    cfg = ops.make_adapter_config(70, 64, 64, 3, 8)
    bad = idx.copy()
    bad[[4, 69]] = [3, 2 ** 31 - 1]
    ref = idx.copy()
    ref[[4, 69]] = -1
    ys = []
    for i in (bad, ref):
        plan = ops.adapter_plan(cfg, torch.from_numpy(i.astype(np.int32)).cuda())
        ys.append(ops.adapter_fwd(cfg, c["x"], c["A"], c["B"], c["scale"], plan, base=c["base"]))
        assert ops.device_status(plan) == (ops.MOE_ERR_DEVICE_INDEX if i is bad else 0)
    assert torch.equal(*ys)


@pytest.mark.parametrize("T", [100, 3000, 20000])
def test_graph_replay_with_another_batch(T):
    # plan, forward and backward captured once serve any batch of the size
    d = _inputs(T, 128, 192, 5, 32, 6)
    c = {k: v.cuda() for k, v in d.items()}
    cfg = ops.make_adapter_config(T, 128, 192, 5, 32)
    ix = torch.from_numpy(_idx(T, 5, 1).astype(np.int32)).cuda()
    ws, u, plan = ops.adapter_workspace(cfg, True), ops.alloc_adapter_saved(cfg), ops.adapter_plan(cfg, ix)
    grads, y = ops.alloc_adapter_grads(cfg), torch.empty_like(c["base"])

    def step():
        ops.adapter_plan(cfg, ix, plan=plan)
        ops.adapter_fwd(cfg, c["x"], c["A"], c["B"], c["scale"], plan, base=c["base"], y=y, u=u, ws=ws)
        ops.adapter_bwd(cfg, c["dy"], c["x"], c["A"], c["B"], c["scale"], plan, u, dx_base=c["dx_base"], grads=grads,
                        ws=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    eager = [t.clone() for t in (y, *grads.values())]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for t in (y, *grads.values()):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, (y, *grads.values())):
        assert torch.equal(a, b)
    ix.copy_(torch.from_numpy(_idx(T, 5, 2, none=0.5).astype(np.int32)))
    g.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in (y, *grads.values())]
    step()
    torch.cuda.synchronize()
    for a, b in zip(replayed, (y, *grads.values())):
        assert torch.equal(a, b)


def test_one_plan_serves_projections_of_other_sizes():
    idx = _idx(200, 4, 9)
    cfgs = [ops.make_adapter_config(200, 128, 64, 4, 16), ops.make_adapter_config(200, 64, 136, 4, 8, out_fp32=True)]
    plan = ops.adapter_plan(cfgs[0], torch.from_numpy(idx.astype(np.int32)).cuda())
    for cfg in cfgs:
        d = _inputs(cfg.T, cfg.K, cfg.N, cfg.L, cfg.r, cfg.K, bool(cfg.out_fp32))
        c = {k: v.cuda() for k, v in d.items()}
        own = ops.adapter_plan(cfg, torch.from_numpy(idx.astype(np.int32)).cuda())
        a, b = (ops.adapter_fwd(cfg, c["x"], c["A"], c["B"], c["scale"], p, base=c["base"]) for p in (plan, own))
        assert torch.equal(a, b)


def test_a_plan_of_another_batch_is_reported():
    d = _inputs(80, 64, 64, 2, 8, 3)
    c = {k: v.cuda() for k, v in d.items()}
    cfg = ops.make_adapter_config(80, 64, 64, 2, 8)
    other = ops.make_adapter_config(96, 64, 64, 3, 8)
    wrong = ops.adapter_plan(other, torch.zeros(96, dtype=torch.int32, device="cuda"))
    for plan in (wrong, torch.zeros_like(wrong)):
        ws, y = ops.adapter_workspace(cfg), c["base"].clone()
        ops.adapter_fwd(cfg, c["x"], c["A"], c["B"], c["scale"], plan, base=c["base"], y=y, ws=ws)
        assert ops.device_status(ws) == ops.MOE_ERR_DEVICE_INDEX and torch.equal(y, c["base"])


@pytest.mark.parametrize("T,L", [(1, 1), (1024, 3), (2048, 1024), (2049, 7), (70000, 40)])
def test_plan_orders_rows_by_adapter(T, L):
    # the plan's order seen through rank-8 products with one-hot rows: each row gets its own adapter's
    # constant, and the gradient of an adapter counts its rows
    rng = np.random.default_rng(T)
    idx = rng.integers(-1, L, T)
    cfg = ops.make_adapter_config(T, 8, 8, L, 8, out_fp32=True)
    x = torch.zeros((T, 8), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    A = torch.zeros((L, 8, 8), dtype=torch.bfloat16, device="cuda")
    A[:, 0, 0] = 1
    B = torch.zeros((L, 8, 8), dtype=torch.bfloat16, device="cuda")
    B[:, 0, 0] = (torch.arange(L, device="cuda") % 32 + 1).to(torch.bfloat16)
    B[:, 0, 1] = (torch.arange(L, device="cuda") // 32 + 1).to(torch.bfloat16)
    plan = ops.adapter_plan(cfg, torch.from_numpy(idx.astype(np.int32)).cuda())
    u = ops.alloc_adapter_saved(cfg)
    y = ops.adapter_fwd(cfg, x, A, B, torch.ones(L, device="cuda"), plan, u=u).cpu().numpy()
    want = np.where(idx[:, None] >= 0, np.stack([idx % 32 + 1, idx // 32 + 1], 1), 0)
    assert np.array_equal(y[:, :2], want) and not y[:, 2:].any()
    dy = torch.zeros((T, 8), dtype=torch.bfloat16, device="cuda")
    dy[:, 3] = 1
    g = ops.adapter_bwd(cfg, dy, x, A, B, torch.ones(L, device="cuda"), plan, u)
    count = np.bincount(idx[idx >= 0], minlength=L)
    assert np.array_equal(g["dB"][:, 0, 3].cpu().numpy(), count) and int(g["dB"].sum()) == count.sum()


@pytest.mark.parametrize("T", [70, 2100])
@pytest.mark.parametrize("before", ["kernel", "memset", "copy", "join"])
def test_captured_behind_other_work(before, T):
    # the calls' first kernels in a capture behind a torch kernel, a memset, a device copy, or the join of two
    # streams; all of it must have finished before they read
    d = _inputs(T, 128, 192, 3, 16, 6)
    c = {k: v.cuda() for k, v in d.items()}
    cfg = ops.make_adapter_config(T, 128, 192, 3, 16)
    ix = torch.from_numpy(_idx(T, 3, 1).astype(np.int32)).cuda()
    src_x, src_ix = c["x"].clone(), ix.clone()
    big = torch.ones(1 << 26, device="cuda")       # long enough to be still running
    plan, ws, y = ops.adapter_plan(cfg, ix), ops.adapter_workspace(cfg), torch.empty_like(c["base"])
    want = ops.adapter_fwd(cfg, c["x"], c["A"], c["B"], c["scale"], plan, base=c["base"]).clone()
    s, side = torch.cuda.Stream(), torch.cuda.Stream()

    def work():
        big.mul_(1.0)
        if before == "kernel":
            torch.add(src_x, 0, out=c["x"])
            torch.add(src_ix, 0, out=ix)
        elif before == "memset":
            torch.add(src_x, 0, out=c["x"])
            ix.zero_()
        elif before == "copy":
            c["x"].copy_(src_x)
            ix.copy_(src_ix)
        else:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                big.mul_(1.0)
                torch.add(src_x, 0, out=c["x"])
            torch.add(src_ix, 0, out=ix)
            torch.cuda.current_stream().wait_stream(side)
        ops.adapter_plan(cfg, ix, plan=plan)
        if before == "join":
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                big.mul_(1.0)
            torch.cuda.current_stream().wait_stream(side)
        ops.adapter_fwd(cfg, c["x"], c["A"], c["B"], c["scale"], plan, base=c["base"], y=y, ws=ws)

    if before == "memset":
        want = ops.adapter_fwd(cfg, src_x, c["A"], c["B"], c["scale"], ops.adapter_plan(cfg, torch.zeros_like(ix)), base=c["base"])
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        work()
    for _ in range(3):
        y.zero_(), c["x"].zero_(), ix.fill_(2)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("T", [1, 70, 1500, 2100, 5000])
def test_inputs_written_right_before_and_overwritten_right_after(T, captured):
    # the calls' later kernels ask for inputs before the kernel ahead has ended: whatever is enqueued ahead of a
    # call must be seen by all of them, and nothing enqueued behind it by any
    K, N, L, r = 256, 320, 5, 24
    cfg = ops.make_adapter_config(T, K, N, L, r)
    names = ("x", "A", "B", "scale", "base", "dy", "dx_base")
    sets = []
    for seed in (1, 2, 3):
        c = {k: v.cuda() for k, v in _inputs(T, K, N, L, r, seed).items()}
        c["idx"] = torch.from_numpy(_idx(T, L, seed).astype(np.int32)).cuda()
        sets.append(c)
    live = {k: torch.empty_like(v) for k, v in sets[0].items()}
    ws, u, plan = ops.adapter_workspace(cfg, training=True), ops.alloc_adapter_saved(cfg), ops.adapter_plan(cfg, sets[0]["idx"])

    def step(c, grads=None):
        ops.adapter_plan(cfg, c["idx"], plan=plan)
        y = ops.adapter_fwd(cfg, *(c[k] for k in names[:4]), plan, base=c["base"], u=u, ws=ws)
        g = ops.adapter_bwd(cfg, c["dy"], *(c[k] for k in names[:4]), plan, u, dx_base=c["dx_base"], grads=grads, ws=ws)
        return [y, g["dx"], g["dA"], g["dB"]]

    want = []
    for c in sets:
        want.append([t.clone() for t in step(c)])
        torch.cuda.synchronize()

    def run():
        got = []
        for c in sets * 3:
            for k, v in live.items():
                torch.add(c[k], 0, out=v)
            got.append(step(live))
            for v in live.values():
                v.fill_(1)
        return got

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    if captured:
        with torch.cuda.stream(s):
            run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = run()
        g.replay()
    else:
        with torch.cuda.stream(s):
            got = run()
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        for a, b in zip(out, want[i % 3]):
            assert torch.equal(a, b), i
    assert ops.device_status(plan) == 0 and ops.device_status(ws) == 0
