"""The router's balance loss and z-loss against the fp64 oracle: values, counts
and the gradient of the logits.

Tolerances (2^-24 is half a step of fp32). A probability is an exp, a sum over
E <= 256 experts in at most 8 + 5 fp32 additions and a few products; the argument
l - max is off by half a step of its own magnitude, at most 2^-24 * 2 * 32 for
the logits drawn here: within 96 half steps together. A loss adds such
probabilities over rows (at most 64 additions in fp32 before fp64 takes over):
relative 160 half steps. Each term of a gradient is a product of at most six
such factors: 128 half steps of the terms' magnitude before they cancel."""
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


def _case(T, E, k, seed, std=1.5):
    rng = np.random.default_rng(seed)
    l = rng.normal(0, std, (T, E)).astype(np.float32)
    idx = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    return l, idx


def _run(l, idx, k, score, off=None, mask=None, coeffs=(0.5, 0.25), dl=(0.75, -1.5), cfg=None, ws=None):
    dev = lambda a, t: None if a is None else torch.from_numpy(np.asarray(a, t)).cuda()
    T, E = l.shape
    S = 1 if off is None else len(off) - 1
    cfg = ops.make_balance_config(T, E, k, n_seqs=S, score=score, balance_coeff=coeffs[0], z_coeff=coeffs[1])
    ws = ops.balance_workspace(cfg) if ws is None else ws
    lg, ix, of, mk = dev(l, np.float32), dev(idx, np.int32), dev(off, np.int32), dev(mask, np.uint8)
    losses, counts, stats = ops.balance_loss_fwd(cfg, lg, ix, of, mk, ws=ws)
    d = ops.balance_loss_bwd(cfg, lg, stats, dev(dl, np.float32), of, mk)
    torch.cuda.synchronize()
    return losses.cpu().numpy(), counts.cpu().numpy(), d.cpu().numpy(), ops.device_status(ws)


def _compare(l, idx, k, score, off=None, mask=None, coeffs=(0.5, 0.25), dl=(0.75, -1.5)):
    losses, counts, d, status = _run(l, idx, k, score, off, mask, coeffs, dl)
    f32 = lambda v: [float(np.float32(x)) for x in v]
    coeffs, dl = f32(coeffs), f32(dl)
    ref_l, ref_c, ref_d, size = TO.balance(l.astype(np.float64), idx, k, score, *coeffs, off, mask, dl)
    assert status == 0
    assert np.array_equal(counts, ref_c)
    assert np.all(np.abs(losses - ref_l) <= 160 * HALF * np.abs(ref_l)), (losses, ref_l)
    assert np.all(np.abs(d - ref_d) <= 128 * HALF * size + 1e-38), np.max(np.abs(d - ref_d) / (size + 1e-30)) / HALF


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (7, 3, 3), (63, 60, 4), (300, 8, 2), (257, 33, 1), (500, 16, 16),
                                   (1000, 100, 6), (129, 128, 8), (777, 130, 8), (2050, 256, 8), (40, 255, 5)])
def test_one_sequence(T, E, k, score):
    _compare(*_case(T, E, k, T + E), k, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("off", [[0, 1, 2, 3, 200], [0, 0, 0, 64, 64, 128, 200], [5, 70, 71, 190], [0, 200, 200], [200, 200, 200],
                                 [17, 17], [0, 33, 66, 99, 132, 165, 198]])
def test_ragged_sequences(off, score):
    l, idx = _case(200, 24, 3, 11)
    rng = np.random.default_rng(1)
    _compare(l, idx, 3, score, off)
    _compare(l, idx, 3, score, off, (rng.random(200) > 0.3).astype(np.uint8))


def test_many_sequences_and_a_long_batch():
    # more sequences than threads of a block; chunks of several hundred rows
    l, idx = _case(5000, 16, 2, 2)
    rng = np.random.default_rng(3)
    off = np.sort(rng.integers(0, 5001, 900))
    _compare(l, idx, 2, "softmax", off.tolist())
    l, idx = _case(40000, 64, 6, 4)
    _compare(l, idx, 6, "sigmoid", [0, 39000, 40000])


def test_everything_masked_gives_zeros():
    l, idx = _case(100, 8, 2, 0)
    losses, counts, d, status = _run(l, idx, 2, "softmax", None, np.zeros(100))
    assert status == 0 and not losses.any() and not counts.any() and not d.any()


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 3.0e38])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_rows_hold_anything(bad, score):
    l, idx = _case(150, 40, 4, 9)
    mask = np.ones(150, np.uint8)
    mask[::3] = 0
    off = [10, 80, 140]
    clean = _run(l, idx, 4, score, off, mask)
    dirty, didx = l.copy(), idx.copy()
    dead = (mask == 0) | (np.arange(150) < 10) | (np.arange(150) >= 140)
    dirty[dead] = bad
    didx[dead] = -7
    got = _run(dirty, didx, 4, score, off, mask)
    for a, b in zip(clean, got):
        assert np.array_equal(a, b)
    assert not got[2][dead].any()


def test_minus_infinity_logits_of_valid_rows():
    # experts switched off by -inf: probability and gradient 0 there
    l, idx = _case(90, 12, 2, 5)
    l[:, 3] = -np.inf
    l[5, :] = -np.inf
    l[5, 7] = 2.0
    idx = np.argsort(-l, axis=1, kind="stable")[:, :2].astype(np.int32)
    for score in ("softmax", "sigmoid"):
        losses, counts, d, _ = _run(l, idx, 2, score)
        with np.errstate(invalid="ignore"):
            lf = np.where(np.isinf(l), -1e4, l)  # exp underflows to 0 in fp64
        ref_l, ref_c, ref_d, size = TO.balance(lf.astype(np.float64), idx, 2, score, 0.5, 0.25, dlosses=(0.75, -1.5))
        assert np.array_equal(counts, ref_c)
        assert np.all(np.abs(losses - ref_l) <= 160 * HALF * np.abs(ref_l))
        assert np.all(np.abs(d - ref_d) <= 128 * HALF * size + 1e-38)


def test_large_logits_do_not_overflow():
    l, idx = _case(64, 20, 2, 6, std=1.0)
    l *= 1e4
    for score in ("softmax", "sigmoid"):
        losses, _, d, _ = _run(l, idx, 2, score)
        assert np.isfinite(losses).all() and np.isfinite(d).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [6, 40, 200])
def test_rows_of_very_small_or_large_scores(score, E):
    # every sigmoid of a row below fp32's range, near its end, or 1
    l, idx = _case(120, E, 3, 13)
    l += np.array([-1000.0, -200.0, -95.0, -60.0, 0.0, 60.0, 500.0], np.float32)[np.arange(120) % 7][:, None]
    _compare(l, idx, 3, score, [0, 50, 120])


def test_default_gradients_and_no_z_loss():
    l, idx = _case(70, 8, 2, 8)
    cfg = ops.make_balance_config(70, 8, 2, balance_coeff=0.5)
    lg = torch.from_numpy(l).cuda()
    losses, counts, stats = ops.balance_loss_fwd(cfg, lg, torch.from_numpy(idx).cuda())
    d = ops.balance_loss_bwd(cfg, lg, stats).cpu().numpy()
    ref_l, _, ref_d, size = TO.balance(l.astype(np.float64), idx, 2, balance_coeff=0.5)
    assert float(losses[1]) == 0.0 and abs(float(losses[0]) - ref_l[0]) <= 160 * HALF * ref_l[0]
    assert np.all(np.abs(d - ref_d) <= 128 * HALF * size)


def test_bad_indices_and_offsets_are_reported():
    l, idx = _case(50, 8, 2, 1)
    idx[3, 1] = 8
    idx[4, 0] = -1
    losses, counts, d, status = _run(l, idx, 2, "softmax")
    assert status == ops.MOE_ERR_DEVICE_INDEX and counts.sum() == 98 and np.isfinite(d).all()
    l, idx = _case(50, 8, 2, 1)
    for off in ([0, 30, 20, 50], [-4, 20, 30, 50], [0, 10, 20, 77]):
        assert _run(l, idx, 2, "softmax", off)[3] == ops.MOE_ERR_DEVICE_INDEX


def test_repeats_and_graph_replays_are_equal_bit_for_bit():
    l, idx = _case(3000, 128, 8, 3)
    off = [0, 700, 700, 1500, 2990]
    cfg = ops.make_balance_config(3000, 128, 8, n_seqs=4, z_coeff=1e-3)
    lg, ix = torch.from_numpy(l).cuda(), torch.from_numpy(idx).cuda()
    of = torch.tensor(off, dtype=torch.int32, device="cuda")
    ws = ops.balance_workspace(cfg)

    def step():
        losses, counts, stats = ops.balance_loss_fwd(cfg, lg, ix, of, ws=ws)
        return losses, counts, ops.balance_loss_bwd(cfg, lg, stats, None, of)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        first = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        outs = step()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, outs):
            assert torch.equal(a, b)
    # other values through the captured buffers
    lg.copy_(torch.from_numpy(l[::-1].copy()))
    g.replay()
    torch.cuda.synchronize()
    again = step()
    for a, b in zip(again, outs):
        assert torch.equal(a, b)


def test_two_streams_with_two_workspaces():
    cases = [_case(4000, 64, 4, s) for s in (1, 2)]
    cfg = ops.make_balance_config(4000, 64, 4, z_coeff=1e-3)
    want, got, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    tens = [(torch.from_numpy(l).cuda(), torch.from_numpy(i).cuda(), ops.balance_workspace(cfg)) for l, i in cases]
    for l, i, ws in tens:
        want.append(ops.balance_loss_fwd(cfg, l, i, ws=ws)[0].clone())
    torch.cuda.synchronize()
    for st, (l, i, ws) in zip(streams, tens):
        with torch.cuda.stream(st):
            for _ in range(20):
                out = ops.balance_loss_fwd(cfg, l, i, ws=ws)[0]
            got.append(out)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
