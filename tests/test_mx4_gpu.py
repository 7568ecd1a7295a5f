"""MXFP4 quantisation of rows and of the layer's weights against the fp64 oracle:
codes, scales and values are equal, bit for bit."""
import numpy as np
import pytest
import torch

from oracle import decode_oracle as DO
from route_permute_grouped_gb300 import ops

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _check_rows(x):
    codes, scales = ops.mx4_quantize(x)
    c, s, v = DO.mx4_quantize(_f64(x))
    packed = c[:, 0::2] | (c[:, 1::2] << 4)
    # a negative zero may keep its sign or not: both stand for 0
    got = codes.cpu().numpy()
    zero = lambda a: np.where(a & 7 == 0, 0, a)
    for shift in (0, 4):
        assert np.array_equal(zero((got >> shift) & 15), zero((packed >> shift) & 15))
    assert np.array_equal(scales.cpu().numpy(), s)
    back = _f64(ops.mx4_dequantize(codes, scales))
    assert np.array_equal(back, v, equal_nan=True)


@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (257, 1504), (64, 4096), (5000, 64)])
def test_rows(M, K):
    g = torch.Generator().manual_seed(M)
    x = torch.randn((M, K), generator=g) * torch.exp(2 * torch.randn((M, 1), generator=g))
    _check_rows(x.to(BF).cuda())


def test_every_bf16_value_in_blocks_of_its_like():
    # every exponent, subnormal numbers among them, with neighbours up to 2^-4 below, and zeros
    g = torch.Generator().manual_seed(7)
    e = torch.arange(-133, 128).repeat_interleave(4)[:, None]
    m = 1 + torch.randint(0, 128, (e.shape[0], 32), generator=g) / 128.0
    x = torch.ldexp(m.double(), e - torch.randint(0, 5, m.shape, generator=g)).to(BF)
    x = torch.where(torch.rand(m.shape, generator=g) < 0.5, -x, x)
    x[::3, 5] = 0.0
    assert torch.isfinite(x.float()).all()
    _check_rows(x.cuda())


def test_infinities_nans_and_zeros():
    x = torch.randn((6, 96)).to(BF)
    x[0, 3], x[1, 40], x[2, 95], x[3, 64:] = float("inf"), float("-inf"), float("nan"), 0.0
    x[4] = 0.0
    x[5, :32] = torch.finfo(BF).max
    _check_rows(x.cuda())


def _weights(E, H, F, Fs=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: (torch.randn(s, generator=g) / s[-2] ** 0.5).to(BF).cuda()
    return r(E, H, F), r(E, H, F), r(E, F, H), (r(H, Fs), r(H, Fs), r(Fs, H)) if Fs else None


@pytest.mark.parametrize("E,H,F,Fs", [(1, 128, 128, 0), (3, 256, 384, 0), (2, 384, 128, 256), (1, 640, 256, 128)])
def test_layer_weights(E, H, F, Fs):
    W1, W3, W2, Ws = _weights(E, H, F, Fs)
    W1[0, 5, 7] = float("nan")
    cfg = ops.make_config(1, H, E, 1, F, F_shared=Fs)
    q = ops.mx4_quantize_weights(cfg, W1, W3, W2, Ws=Ws)
    assert set(q) == {"w13", "w2"} | ({"w13s", "w2s"} if Fs else set())
    back = ops.mx4_dequantize_weights(cfg, q)
    assert (back[3] is None) == (Fs == 0)
    pairs = list(zip(back[:3], (W1, W3, W2))) + (list(zip(back[3], Ws)) if Fs else [])
    for got, w in pairs:
        assert np.array_equal(_f64(got), DO.mx4_weights(_f64(w)), equal_nan=True)
    # what stands for the weights is quantised to itself (but for the block of NaN, whose codes are 0 either way)
    again = ops.mx4_quantize_weights(cfg, *back[:3], Ws=back[3])
    assert all(torch.equal(q[n], again[n]) for n in q)


def test_captured_and_replayed():
    x = torch.randn((100, 256), device="cuda").to(BF)
    want = [ops.mx4_quantize(x * s) for s in (1.0, 3.0)]
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        y = x.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            c, s = ops.mx4_quantize(y)
            v = ops.mx4_dequantize(c, s)
        for i, f in enumerate((1.0, 3.0)):
            y.copy_(x * f)
            graph.replay()
            st.synchronize()
            assert torch.equal(c, want[i][0]) and torch.equal(s, want[i][1])
            assert torch.equal(v, ops.mx4_dequantize(*want[i]))


def test_offsets_beyond_32_bits():
    # 2^32 + elements: the last rows against the same rows alone
    M, K = (1 << 32) // 4096 + 3, 4096
    x = torch.zeros((M, K), dtype=BF, device="cuda")
    x[-5:] = torch.randn((5, K), device="cuda").to(BF)
    c, s = ops.mx4_quantize(x)
    c5, s5 = ops.mx4_quantize(x[-5:].contiguous())
    assert torch.equal(c[-5:], c5) and torch.equal(s[-5:], s5) and not c[:-5].any()
    v = ops.mx4_dequantize(c, s)
    assert torch.equal(v[-5:], ops.mx4_dequantize(c5, s5))


def test_refusals():
    x = torch.zeros((4, 64), dtype=BF, device="cuda")
    for bad in (x.float(), x[:, :48].contiguous(), x[:, ::2], x[0], x[:0], None, x.cpu()):
        with pytest.raises(ops.MoeError):
            ops.mx4_quantize(bad)
    c, s = ops.mx4_quantize(x)
    for a, b in ((c, s[:, :1].contiguous()), (c[:, :8].contiguous(), s), (c.float(), s), (c, s.cpu())):
        with pytest.raises(ops.MoeError):
            ops.mx4_dequantize(a, b)
    W1, W3, W2, Ws = _weights(2, 128, 128, 128)
    cfg = ops.make_config(1, 128, 2, 1, 128, F_shared=128)
    with pytest.raises(ops.MoeError):
        ops.mx4_quantize_weights(cfg, W1, W3, W2)  # the shared expert's weights are missing
    with pytest.raises(ops.MoeError):
        ops.mx4_quantize_weights(cfg, W1, W3.float(), W2, Ws=Ws)
    q = ops.mx4_quantize_weights(cfg, W1, W3, W2, Ws=Ws)
    with pytest.raises(ops.MoeError):
        ops.mx4_dequantize_weights(cfg, {n: q[n] for n in ("w13", "w2")})
    with pytest.raises(ops.MoeError):
        ops.mx4_quantize_weights(ops.make_config(1, 192, 2, 1, 128), W1, W3, W2)
