"""The global gradient norm and clipping against the fp64 oracle.

Tolerances (2^-24 is half a step of fp32): at most 32 squares are added in fp32
before fp64 takes over (33 half steps, halved by the root), and the norm is
rounded once: 18 half steps. A coefficient adds two roundings and a scaled
value one more and its own: 24 half steps and half a step of the type."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as TO
from route_permute_grouped_gb300 import ops

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -24
TYPES = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


def _tensors(sizes, dtypes, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std * 10.0 ** -(i % 3)).to(dtypes[i % len(dtypes)]).cuda()
            for i, n in enumerate(sizes)]


def _f64(ts):
    return [t.detach().cpu().to(torch.float64).numpy() for t in ts]


def _check_clip(before, after, norm, max_norm, kind):
    n, want = TO.clip(before, max_norm, kind)
    assert abs(float(norm) - n) <= 18 * HALF * n
    for t, w in zip(after, want):
        got = t.cpu().to(torch.float64).numpy()
        tiny = 2.0 ** -25 if t.dtype == torch.float16 else 2.0 ** -134  # below the normal range
        assert np.all(np.abs(got - w) <= (24 * HALF + TYPES[t.dtype]) * np.abs(w) + tiny)


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("dtypes", [[torch.float32], [torch.bfloat16], [torch.float16],
                                    [torch.float32, torch.bfloat16, torch.float16]])
@pytest.mark.parametrize("sizes", [[1], [3], [8], [4097], [1, 2, 3, 4, 5, 6, 7, 8, 9], [100000, 1, 33, 8191, 8192, 8193],
                                   [300001, 0, 12]])
def test_norm_and_clip(sizes, dtypes, kind):
    ts = _tensors(sizes, dtypes)
    before = _f64(ts)
    n = ops.grad_norm(ts, kind)
    assert abs(float(n) - TO.grad_norm(before, kind)) <= 18 * HALF * TO.grad_norm(before, kind)
    norm = ops.clip_grad_norm(ts, 0.125, kind)
    assert torch.equal(n, norm)
    _check_clip(before, ts, norm, 0.125, kind)


def test_below_the_threshold_every_bit_stays():
    ts = _tensors([1000, 77], [torch.float32, torch.bfloat16])
    keep = [t.clone() for t in ts]
    ops.clip_grad_norm(ts, 1e6)
    assert all(torch.equal(a, b) for a, b in zip(ts, keep))
    out = [torch.zeros_like(t) for t in ts]
    ops.clip_grad_norm(ops.tensor_list(ts, out=out), 1e6)
    assert all(torch.equal(a, b) for a, b in zip(out, keep))


@pytest.mark.parametrize("apart", [False, True])
def test_more_chunks_than_resident_blocks(apart):
    # 5500 chunks and more: the clipping's later blocks start after the norm is known
    g = torch.Generator("cuda").manual_seed(5)
    ts = [torch.randn(n, generator=g, device="cuda").to(t) for n, t in
          [(45_000_001, torch.float32), (3, torch.float32), (9_000_007, torch.bfloat16)]]
    keep = [t.clone() for t in ts]
    out = [torch.zeros_like(t) for t in ts] if apart else None
    tl = ops.tensor_list(ts, out=out)
    want = float(torch.stack([t.double().square().sum() for t in keep]).sum().sqrt())
    norm = ops.clip_grad_norm(tl, 1e9)
    assert abs(float(norm) - want) <= 18 * HALF * want
    assert all(torch.equal(a, b) for a, b in zip(out if apart else ts, keep))
    norm = ops.clip_grad_norm(tl, 2.5)
    assert abs(float(norm) - want) <= 18 * HALF * want
    for t, k in zip(out if apart else ts, keep):
        w = k.double() * (2.5 / (want + 1e-6))
        assert bool(((t.double() - w).abs() <= (24 * HALF + TYPES[t.dtype]) * w.abs() + 2.0 ** -134).all())
    assert not apart or all(torch.equal(a, b) for a, b in zip(ts, keep))


@pytest.mark.parametrize("shift", [1, 2, 3, 5])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_views_at_odd_offsets(dtype, shift):
    # neighbours inside one buffer stay untouched; outputs aligned otherwise than inputs
    flat = _tensors([5000], [dtype])[0]
    other = torch.full((6000,), 7.0, dtype=dtype, device="cuda")
    ts = [flat[shift:shift + 1001], flat[2000 + shift:2000 + shift + 6], flat[3001:3002], flat[4000 + shift:]]
    outs = [other[i * 1200:i * 1200 + t.numel()] for i, t in enumerate(ts)]
    before, whole = _f64(ts), flat.clone()
    norm = ops.clip_grad_norm(ops.tensor_list(ts, out=outs), 0.5)
    _check_clip(before, outs, norm, 0.5, "l2")
    assert torch.equal(flat, whole)
    for i, t in enumerate(ts):
        assert (other[i * 1200 + t.numel():(i + 1) * 1200] == 7).all()
    norm = ops.clip_grad_norm(ts, 0.5)
    _check_clip(before, ts, norm, 0.5, "l2")
    touched = torch.zeros(5000, dtype=torch.bool, device="cuda")
    for t in ts:
        at = (t.data_ptr() - flat.data_ptr()) // flat.element_size()
        touched[at:at + t.numel()] = True
    assert torch.equal(flat[~touched], whole[~touched])


@pytest.mark.parametrize("count", [16, 17, 128, 129, 768, 769, 2000])
def test_many_tensors(count):
    ts = _tensors([1 + (7 * i) % 97 for i in range(count)], [torch.float32, torch.bfloat16])
    before = _f64(ts)
    norm = ops.clip_grad_norm(ts, 1.0)
    _check_clip(before, ts, norm, 1.0, "l2")


def test_a_tensor_of_many_chunks():
    ts = _tensors([30_000_001, 5], [torch.bfloat16])
    before = _f64(ts)
    norm = ops.clip_grad_norm(ts, 1.0)
    _check_clip(before, ts, norm, 1.0, "l2")


@pytest.mark.parametrize("mag", [1e-38, 1e-30, 1e-22, 1e-19, 1e-18, 1e17, 1e19, 1e25, 1e36])
def test_magnitudes_whose_squares_leave_fp32(mag):
    g = torch.Generator().manual_seed(1)
    ts = [(torch.rand(999, generator=g) + 0.5).mul_(mag).cuda(), torch.zeros(64, device="cuda")]
    before = _f64(ts)
    n = TO.grad_norm(before)
    assert abs(float(ops.grad_norm(ts)) - n) <= 18 * HALF * n + 2.0 ** -149
    if mag > 1:
        norm = ops.clip_grad_norm(ts, 1.0)
        _check_clip(before, ts, norm, 1.0, "l2")


def test_mixed_magnitudes_in_one_group():
    t = torch.full((64,), 1e-25).cuda()
    t[5] = 1e22
    t[40] = 3e-20
    n = TO.grad_norm(_f64([t]))
    assert abs(float(ops.grad_norm([t])) - n) <= 18 * HALF * n


def test_not_finite():
    for kind in ("l2", "max"):
        ts = _tensors([500, 40], [torch.float32])
        ts[0][123] = float("inf")
        assert float(ops.grad_norm(ts, kind)) == float("inf")
        ops.clip_grad_norm(ts, 1.0, kind)      # coefficient 0: inf * 0 is NaN, the rest 0
        assert bool(torch.isnan(ts[0][123])) and not ts[1].any() and int(torch.isnan(ts[0]).sum()) == 1
        ts = _tensors([500, 40], [torch.float32])
        ts[0][123], ts[1][0] = float("nan"), float("inf")
        assert np.isnan(float(ops.grad_norm(ts, kind)))
        ops.clip_grad_norm(ts, 1.0, kind)
        assert bool(torch.isnan(ts[0]).all()) and bool(torch.isnan(ts[1]).all())


def test_empty_list_and_zero_gradients():
    assert float(ops.grad_norm([])) == 0.0 and float(ops.clip_grad_norm([], 1.0)) == 0.0
    z = [torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda")]
    assert float(ops.clip_grad_norm(z, 1.0)) == 0.0 and not z[0].any()
    t = [torch.ones(9, device="cuda")]
    assert float(ops.clip_grad_norm(t, 0.0)) == 3.0 and not t[0].any()


def test_repeats_and_graph_replays_are_equal_bit_for_bit():
    ts = _tensors([3_000_001, 70_000, 3], [torch.float32, torch.bfloat16], seed=4)
    out = [torch.empty_like(t) for t in ts]
    tl, ws = ops.tensor_list(ts, out=out), ops.grad_norm_workspace()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        first = ops.clip_grad_norm(tl, 1.0, ws=ws).clone()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    keep = [t.clone() for t in out]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        norm = ops.clip_grad_norm(tl, 1.0, ws=ws)
    for t in out:
        t.zero_()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, norm) and all(torch.equal(a, b) for a, b in zip(out, keep))
    ts[0].mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert abs(float(norm) - TO.grad_norm(_f64(ts))) <= 18 * HALF * float(norm)
