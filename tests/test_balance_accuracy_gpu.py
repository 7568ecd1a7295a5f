"""The accuracy of the router losses' gradient where rows have a common offset:
what a logit is off by must come from the row's own spread, not from where the
row lies.

Tolerance, root mean square over the elements, in half steps of fp32 (2^-24). A
rounding is off by 1 / sqrt(3) of its bound in the mean. A probability is an
exponential (2 ulp: 4 half steps), its row's sum (the same mean error of its
terms, and at most 8 + 5 additions), a reciprocal (2 half steps) and three
products: sqrt((16 + 16 + 13 + 4 + 3) / 3) = 4.2. A gradient against one
expert's weight takes the probability twice: 4.2 sqrt(2) = 5.9, bounded by 6.5;
the z-loss takes it once, and the logarithm of a sum with a product: 4.2 and 1,
bounded by 5. An offset of 35 whose exponent argument is rounded as a whole gives 12
half steps for one probability."""
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


def _gradient(l, score, balance, z):
    """(gradient, the oracle's, losses, the oracle's) with every slot on expert 0."""
    T, E = l.shape
    idx = np.zeros((T, 1), np.int32)
    cfg = ops.make_balance_config(T, E, 1, score=score, balance_coeff=balance, z_coeff=z)
    lg = torch.from_numpy(l).cuda()
    losses, _, stats = ops.balance_loss_fwd(cfg, lg, torch.from_numpy(idx).cuda())
    d = ops.balance_loss_bwd(cfg, lg, stats).cpu().numpy().astype(np.float64)
    f = lambda v: float(np.float32(v))
    want, _, ref, _ = TO.balance(l.astype(np.float64), idx, 1, score, f(balance), f(z))
    return d, ref, losses.cpu().numpy(), want


def _rms(d, ref):
    return float(np.sqrt(np.mean(((d - ref) / ref) ** 2))) / HALF


def _logits(T, E, offset, std=1.0):
    return (np.random.default_rng(E).normal(0, std, (T, E)) + offset).astype(np.float32)


@pytest.mark.parametrize("E", [8, 60, 130, 256])
@pytest.mark.parametrize("offset", [0.0, 10.0, 35.0, -35.0, 60.0, -60.0, 500.0])
def test_softmax_balance_gradient(E, offset):
    d, ref, losses, want = _gradient(_logits(700, E, offset), "softmax", 1.0, 0.0)
    assert _rms(d[:, 1:], ref[:, 1:]) <= 6.5
    assert abs(losses[0] - want[0]) <= 16 * HALF * want[0]


# towards +inf a sigmoid's slope 1 - sigmoid is exp(-l): offsets up to where fp32 holds the products
@pytest.mark.parametrize("E", [8, 60, 130, 256])
@pytest.mark.parametrize("offset", [0.0, 10.0, 35.0, -35.0, -60.0, 60.0])
def test_sigmoid_balance_gradient(E, offset):
    d, ref, losses, want = _gradient(_logits(700, E, offset), "sigmoid", 1.0, 0.0)
    assert _rms(d[:, 1:], ref[:, 1:]) <= 6.5 + 2.0     # the slope: one exponential and its reciprocal more, sqrt((16 + 4) / 3)
    assert abs(losses[0] - want[0]) <= 16 * HALF * want[0]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 60, 130, 256])
@pytest.mark.parametrize("offset", [10.0, 35.0, -35.0, 60.0, -60.0])
def test_z_gradient(E, offset, score):
    d, ref, losses, want = _gradient(_logits(700, E, offset), score, 0.0, 1.0)
    assert _rms(d, ref) <= 5
    assert abs(losses[1] - want[1]) <= 16 * HALF * want[1]


@pytest.mark.parametrize("E", [8, 256])
def test_logarithm_of_sums_near_one(E):
    # rows whose log-sum-exp is near 0: what it is off by is that of the sum, 13 additions and two ulp of its terms
    l = _logits(400, E, 0.0, 0.5)
    l = (l - np.log(np.exp(l.astype(np.float64)).sum(1, keepdims=True)) + 1e-3 * np.arange(400)[:, None] / 400).astype(np.float32)
    d, ref, losses, want = _gradient(l, "softmax", 0.0, 1.0)
    l64 = l.astype(np.float64)
    lse = np.log(np.exp(l64).sum(1, keepdims=True))
    soft = np.exp(l64 - lse)
    err = np.abs(d - ref) / (2 / 400 * soft)           # the error of lse itself, and 26 half steps of the product
    assert float(np.max(err - 26 * HALF * np.abs(lse))) <= 18 * HALF


@pytest.mark.parametrize("E", [6, 40, 256])
def test_infinite_logits_of_valid_rows_under_sigmoid_scores(E):
    # a sigmoid of +inf is 1 with slope 0: without the z-loss (whose log-sum-exp is infinite there) all is finite
    l = _logits(90, E, 0.0)
    l[::7, 2] = np.inf
    l[3, :] = np.inf
    l[::5, 4] = -np.inf
    idx = np.random.default_rng(1).integers(0, E, (90, 3)).astype(np.int32)
    cfg = ops.make_balance_config(90, E, 3, score="sigmoid", balance_coeff=1.0)
    lg = torch.from_numpy(l).cuda()
    losses, counts, stats = ops.balance_loss_fwd(cfg, lg, torch.from_numpy(idx).cuda())
    d = ops.balance_loss_bwd(cfg, lg, stats).cpu().numpy()
    with np.errstate(invalid="ignore"):
        ref_l, ref_c, ref_d, size = TO.balance(l.astype(np.float64), idx, 3, "sigmoid", 1.0)
    assert np.array_equal(counts.cpu().numpy(), ref_c) and float(losses[1]) == 0.0
    assert abs(float(losses[0]) - ref_l[0]) <= 32 * HALF * ref_l[0]
    # terms of at most: three exponentials and three reciprocals (18), two sums (26), six products
    assert np.all(np.abs(d - ref_d) <= 50 * HALF * size + 1e-38)
