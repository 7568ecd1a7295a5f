"""One scratch buffer lent to one operator after another: each leaves it as the
next one needs it, with no zeroing in between."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as TO
from route_permute_grouped_gb300 import ops

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


# the balance loss counts n_seqs * ceil(E / 32) blocks in the scratch; the norm of `n` values runs on n / 8192 of them
@pytest.mark.parametrize("S,E,n", [(1, 8, 100), (1, 256, 100), (1, 8, 3_000_000), (37, 64, 3_000_000), (61, 256, 9_000_000)])
def test_norm_and_clipping_after_a_balance_loss(S, E, n):
    T = 500
    g = torch.Generator(device="cuda").manual_seed(S + E)
    cfg = ops.make_balance_config(T, E, 2, n_seqs=S, z_coeff=1e-3)
    logits = torch.randn((T, E), generator=g, device="cuda")
    idx = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :2].to(torch.int32).contiguous()
    off = torch.linspace(0, T, S + 1, device="cuda").to(torch.int32)
    nbytes = max(ops.balance_workspace(cfg).numel(), ops.grad_norm_workspace().numel())
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    ws[256:] = 0x5a                     # what an earlier user of the memory left
    t = torch.randn(n, generator=g, device="cuda")
    want = TO.grad_norm([t.cpu().to(torch.float64).numpy()])
    want_losses = ops.balance_loss_fwd(cfg, logits, idx, off)[0]
    for _ in range(2):
        losses = ops.balance_loss_fwd(cfg, logits, idx, off, ws=ws)[0]
        norm = ops.grad_norm([t], ws=ws)
        assert torch.equal(losses, want_losses)
        assert abs(float(norm) - want) <= 18 * HALF * want
        assert ops.device_status(ws) == 0 and not ws[:256].any()
    out = torch.empty_like(t)
    losses = ops.balance_loss_fwd(cfg, logits, idx, off, ws=ws)[0]
    norm = ops.clip_grad_norm(ops.tensor_list([t], out=[out]), 0.5, ws=ws)
    assert abs(float(norm) - want) <= 18 * HALF * want
    ref = t.double() * (0.5 / (want + 1e-6))
    assert bool(((out.double() - ref).abs() <= 25 * HALF * ref.abs()).all())


def test_adapters_leave_the_scratch_to_the_others():
    T, K, L, r = 300, 128, 3, 16
    g = torch.Generator(device="cuda").manual_seed(2)
    bf = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    cfg = ops.make_adapter_config(T, K, K, L, r)
    idx = torch.randint(-1, L, (T,), generator=g, device="cuda").to(torch.int32)
    x, dy, A, B, scale = bf(T, K), bf(T, K), bf(L, K, r), bf(L, r, K), torch.ones(L, device="cuda")
    ws = torch.zeros(max(ops.adapter_workspace(cfg, True).numel(), ops.grad_norm_workspace().numel()), dtype=torch.uint8,
                     device="cuda")
    plan, u = ops.adapter_plan(cfg, idx), ops.alloc_adapter_saved(cfg)
    grads = []
    for _ in range(2):
        ops.adapter_fwd(cfg, x, A, B, scale, plan, u=u, ws=ws)
        grads.append(ops.adapter_bwd(cfg, dy, x, A, B, scale, plan, u, ws=ws))
        norm = ops.grad_norm([grads[-1]["dA"], grads[-1]["dB"]], ws=ws)
        want = TO.grad_norm([grads[-1][n].cpu().to(torch.float64).numpy() for n in ("dA", "dB")])
        assert abs(float(norm) - want) <= 18 * HALF * want and not ws[:256].any()
    assert all(torch.equal(grads[0][n], grads[1][n]) for n in grads[0])
