"""Sums of the router losses over millions of rows: fp32 runs stay short, however
long the batch.

The rows are equal and hold exact values, so what a sum is off by comes from its
additions alone. A run of n equal terms is off by at most half a step of each
partial sum: (n + 1) / 2 half steps of the result. Runs end at 64 rows (33), then
the groups of a warp (at most 4 additions), its 8 warps and the product with the
mean follow: 48 half steps. A run of 431 rows of the values below is off by 100."""
import pytest
import torch

from route_permute_grouped_gb300 import ops

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -24
BOUND = 48 * HALF


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


def _losses(row, T, balance, z, score="softmax", off=None):
    E = row.numel()
    S = 1 if off is None else off.numel() - 1
    cfg = ops.make_balance_config(T, E, 1, n_seqs=S, score=score, balance_coeff=balance, z_coeff=z)
    logits = row.cuda()[None].expand(T, E).contiguous()
    idx = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    losses, counts, _ = ops.balance_loss_fwd(cfg, logits, idx, off)
    assert int(counts.sum()) == T and not counts[:, 1:].any()
    return losses.cpu().double()


@pytest.mark.parametrize("T,E,q", [(1 << 21, 256, 4048), (1 << 21, 256, 3761), (1 << 24, 8, 3208), (1 << 22, 128, 4048)])
def test_z_loss(T, E, q):
    # one expert with logit q, the others switched off: the log-sum-exp is q, its square 24 bits
    row = torch.full((E,), float("-inf"))
    row[0] = float(q)
    assert abs(float(_losses(row, T, 0.0, 1.0)[1]) / (q * q) - 1) <= BOUND


@pytest.mark.parametrize("m", [111, 221, 222, 229, 241, 255])
def test_balance_loss(m):
    # m equal experts, the others switched off: every probability is 1 / m, off by 2 half steps at most
    row = torch.full((256,), float("-inf"))
    row[:m] = 0.0
    assert abs(float(_losses(row, 1 << 21, 1.0, 0.0)[0]) * m / 256 - 1) <= BOUND + 2 * HALF


def test_ragged_sequences_of_a_long_batch():
    T = (1 << 21) + 77
    off = torch.tensor([0, 5, 1 << 20, (1 << 20) + 700, T], dtype=torch.int32, device="cuda")
    row = torch.full((256,), float("-inf"))
    row[0] = 4048.0
    losses = _losses(row, T, 1.0, 1.0, off=off)
    assert abs(float(losses[1]) / 4048.0 ** 2 - 1) <= BOUND and abs(float(losses[0]) / 256 - 1) <= BOUND
