"""What keeps the adapters' fp32 results and weight gradients at fp32 accuracy:
u and du enter their second product in three bf16 parts (24 bits), and sums
leave the tensor cores' accumulators every 512 products.

Parts: every sum below has one term that is not 0 and its factors but the scale
are powers of two, so each result is the scale times a power of two, exactly: a
part that is missing, or lies in the wrong place, changes it by up to 2^-9 (the
second) or 2^-17 (the third) of itself.

Sums: tensor-core accumulation cuts at the last bit. For positive operands a sum of
512 products came out too small by 5e-7 of itself in the mean, one of 8192 in one
go by 8e-6; the fp32 additions that join the runs round to nearest, with no bias.
Bound for the mean: 1e-6."""
import numpy as np
import pytest
import torch

from route_permute_grouped_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("T,L", [(1, 1), (300, 300), (1500, 700), (2047, 3), (2048, 1000), (5000, 7)])
def test_three_parts(T, L, r):
    K, N = 328, 264
    rng = np.random.default_rng(T + r)
    # one row of each adapter (spread over the batch) holds something; the others add zeros
    idx = rng.permutation(T) % L
    row = np.array([np.nonzero(idx == a)[0][rng.integers(0, np.sum(idx == a))] for a in range(L)])
    k, j, n = rng.integers(0, K, L), rng.integers(0, r, L), rng.integers(0, N, L)
    p = lambda: 2.0 ** rng.integers(-6, 7, L)
    px, pa, pb, pd = p(), p(), p(), p()
    s = rng.uniform(0.5, 2.0, L).astype(np.float32)
    at = np.arange(L)
    bf = lambda a: torch.from_numpy(a.astype(np.float32)).cuda().to(torch.bfloat16)
    x, A, B, dy = np.zeros((T, K)), np.zeros((L, K, r)), np.zeros((L, r, N)), np.zeros((T, N))
    x[row, k], A[at, k, j], B[at, j, n], dy[row, n] = px, pa, pb, pd
    cfg = ops.make_adapter_config(T, K, N, L, r, out_fp32=True)
    plan, u = ops.adapter_plan(cfg, torch.from_numpy(idx.astype(np.int32)).cuda()), ops.alloc_adapter_saved(cfg)
    ws, sc = ops.adapter_workspace(cfg, True), torch.from_numpy(s).cuda()
    y = ops.adapter_fwd(cfg, bf(x), bf(A), bf(B), sc, plan, u=u, ws=ws)
    g = ops.adapter_bwd(cfg, bf(dy), bf(x), bf(A), bf(B), sc, plan, u, ws=ws)
    want = {"y": np.zeros((T, N)), "dx": np.zeros((T, K)), "dA": np.zeros((L, K, r)), "dB": np.zeros((L, r, N))}
    want["y"][row, n] = s * px * pa * pb
    want["dx"][row, k] = s * pd * pb * pa
    want["dA"][at, k, j] = s * pd * pb * px
    want["dB"][at, j, n] = s * px * pa * pd
    for name, t in {"y": y, **g}.items():
        assert np.array_equal(t.cpu().numpy(), want[name].astype(np.float32)), name
    assert ops.device_status(ws) == 0


def _bias(got, want):
    return float(((got.double() - want) / want).mean())


@pytest.mark.parametrize("r", [16, 64, 128])
@pytest.mark.parametrize("T", [300, 2100])
@pytest.mark.parametrize("K", [8192, 20000])
def test_long_inner_sums(K, T, r):
    # B and A pick single columns, so y and dx show u and du: sums of K, and N, positive products
    g = torch.Generator(device="cuda").manual_seed(K + T + r)
    pos = lambda *shape: (torch.rand(shape, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    cfg = ops.make_adapter_config(T, K, r, 1, r, out_fp32=True)
    x, A = pos(T, K), pos(1, K, r)
    eye = torch.eye(r, device="cuda", dtype=torch.bfloat16)[None].contiguous()
    one = torch.ones(1, device="cuda")
    plan = ops.adapter_plan(cfg, torch.zeros(T, dtype=torch.int32, device="cuda"))
    y = ops.adapter_fwd(cfg, x, A, eye, one, plan)
    assert abs(_bias(y, x.double() @ A[0].double())) <= 1e-6
    back = ops.make_adapter_config(T, r, K, 1, r, out_fp32=True)
    B, zero = pos(1, r, K), torch.zeros((T, r), dtype=torch.bfloat16, device="cuda")
    u = ops.alloc_adapter_saved(back)
    ops.adapter_fwd(back, zero, eye, B, one, plan, u=u)
    grads = ops.adapter_bwd(back, x, zero, eye, B, one, plan, u)
    assert abs(_bias(grads["dx"], x.double() @ B[0].double().t())) <= 1e-6


@pytest.mark.parametrize("r", [16, 64, 128])
# (10000 columns and more leave a block a run of several thousand rows; narrow ones split them over all blocks)
@pytest.mark.parametrize("T,L,K,N", [(1000, 1, 136, 200), (8192, 1, 136, 200), (30000, 1, 136, 200), (30001, 3, 136, 200),
                                     (12000, 1, 10000, 64), (20001, 2, 64, 16008)])
def test_long_sums_over_rows(T, L, K, N, r):
    # u and du are equal in every row: the weight gradients are their products with column sums of x and of dy
    g = torch.Generator(device="cuda").manual_seed(T + r)
    pos = lambda *shape: (torch.rand(shape, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    cfg = ops.make_adapter_config(T, K, N, L, r, out_fp32=True)
    x, dy = pos(T, K), pos(T, N)
    x[:, 0], dy[:, 0] = 1, 1
    A, B = torch.zeros((L, K, r), dtype=torch.bfloat16, device="cuda"), torch.zeros((L, r, N), dtype=torch.bfloat16, device="cuda")
    A[:, 0], B[:, :, 0] = pos(L, r), pos(L, r)
    scale = torch.rand(L, generator=g, device="cuda") + 0.5
    idx = torch.randint(0, L, (T,), generator=g, device="cuda").to(torch.int32)
    plan, u = ops.adapter_plan(cfg, idx), ops.alloc_adapter_saved(cfg)
    ops.adapter_fwd(cfg, x, A, B, scale, plan, u=u)
    grads = ops.adapter_bwd(cfg, dy, x, A, B, scale, plan, u)
    for a in range(L):
        q = idx == a
        c = scale[a].double()
        assert abs(_bias(grads["dA"][a], x[q].sum(0, dtype=torch.float64)[:, None] * (c * B[a, :, 0].double())[None])) <= 1e-6
        assert abs(_bias(grads["dB"][a], (c * A[a, 0].double())[:, None] * dy[q].sum(0, dtype=torch.float64)[None])) <= 1e-6
