"""Host checks of the few-token layer, MXFP4 and the block norms: bad arguments are
refused before any CUDA work. CPU only (no call here launches)."""
import ctypes

import pytest
import torch

from route_permute_grouped_gb300 import build as B
from route_permute_grouped_gb300 import ops

BAD, SHAPE, SMALL = ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_UNSUPPORTED_SHAPE, ops.MOE_ERR_WORKSPACE_TOO_SMALL
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    B.build()
    return ops.lib()


def _weights(*ptrs):
    return ctypes.byref(ops.MoeMx4Weights(*[p if p else None for p in ptrs]))


@pytest.mark.parametrize("over,code", [(dict(T=0), BAD), (dict(T=65), SHAPE), (dict(H=96), SHAPE), (dict(F=100), SHAPE), (dict(E=257), SHAPE),
                                       (dict(k=9), BAD), (dict(F_shared=32), SHAPE), (dict(H=(1 << 17) + 64), SHAPE),
                                       (dict(F=(1 << 17) + 64), SHAPE), (dict(gate_scale=0.0), BAD), (dict(score=3), BAD)])
def test_few_configs(lib, over, code):
    cfg = ops.make_config(**(dict(T=4, H=128, E=8, k=2, F=128) | over))
    for mx in (0, 1):
        assert lib.moe_few_workspace_bytes(ctypes.byref(cfg), mx) == 0
    assert lib.moe_layer_few_fwd(ctypes.byref(cfg), *[P(4096)] * 14, 1 << 40, None) == code
    assert lib.moe_layer_few_fwd_mxfp4(ctypes.byref(cfg), *[P(4096)] * 4, _weights(4096, 4096, 4096, 4096), *[P(4096)] * 4, 1 << 40, None) == code
    with pytest.raises(ops.MoeError):
        ops.few_workspace(cfg, device="cpu")


def test_few_of_multiples_of_64_has_no_mxfp4_form(lib):
    for over in (dict(H=192), dict(F=192), dict(F_shared=64)):
        cfg = ops.make_config(**(dict(T=4, H=128, E=8, k=2, F=128) | over))
        assert lib.moe_few_workspace_bytes(ctypes.byref(cfg), 0) > 0 and lib.moe_few_workspace_bytes(ctypes.byref(cfg), 1) == 0
        assert all(lib.moe_mx4_weight_bytes(ctypes.byref(cfg), i) == 0 for i in range(4))
        assert lib.moe_mx4_quantize_weights(ctypes.byref(cfg), *[P(4096)] * 6, _weights(4096, 4096, 4096, 4096), None) == SHAPE


def _apart(n):
    return [P((i + 1) << 24) for i in range(n)]


def _off(p):
    return P(p.value + 8)


def test_few_pointers(lib):
    # order: x router_w expert_bias logit_bias W1 W3 W2 Ws1 Ws3 Ws2 idx gate y ws
    cfg = ops.make_config(4, 128, 8, 2, 128, F_shared=128)
    call = lambda p: lib.moe_layer_few_fwd(ctypes.byref(cfg), *p, 16, None)
    assert call(_apart(14)) == SMALL
    for i in range(14):
        for v in (None, "off"):
            p = _apart(14)
            p[i] = P(None) if v is None else _off(p[i])
            assert call(p) == (SMALL if v is None and i in (2, 3) else BAD), (i, v)
    plain = ops.make_config(4, 128, 8, 2, 128)
    p = _apart(14)
    p[7] = p[8] = p[9] = P(None)
    assert lib.moe_layer_few_fwd(ctypes.byref(plain), *p, 16, None) == SMALL
    mx = lambda c, w, p: lib.moe_layer_few_fwd_mxfp4(ctypes.byref(c), *p[:4], w, *p[4:], 16, None)
    q, w = _apart(8), [(i + 20) << 24 for i in range(4)]
    assert mx(cfg, _weights(*w), q) == SMALL and mx(plain, _weights(*w[:2], None, None), q) == SMALL
    assert mx(cfg, _weights(*w[:2], None, w[3]), q) == BAD and mx(plain, _weights(w[0], None, None, None), q) == BAD
    assert mx(cfg, _weights(w[0], w[1] + 8, *w[2:]), q) == BAD and mx(cfg, None, q) == BAD
    assert lib.moe_layer_few_fwd(None, *_apart(14), 1 << 40, None) == BAD


def test_few_refuses_overlapping_outputs(lib):
    cfg = ops.make_config(4, 128, 8, 2, 128, F_shared=128)
    call = lambda c, p: lib.moe_layer_few_fwd(ctypes.byref(c), *p, 16, None)
    for out in (10, 11, 12, 13):
        for other in range(14):
            if other != out:
                p = _apart(14)
                p[out] = P(p[other].value + 16)
                assert call(cfg, p) == BAD, (out, other)
    p = _apart(14)
    p[12] = p[0]  # y over x
    assert call(cfg, p) == SMALL
    assert call(ops.make_config(4, 128, 8, 2, 128, F_shared=128, out_fp32=True), p) == BAD
    q, w = _apart(8), [(i + 20) << 24 for i in range(4)]
    for i in range(4):
        p = list(q)
        p[6] = P(w[i] + 16)
        assert lib.moe_layer_few_fwd_mxfp4(ctypes.byref(cfg), *p[:4], _weights(*w), *p[4:], 16, None) == BAD


def test_mx4_sizes(lib):
    cfg = ops.make_config(1, 384, 3, 1, 256, F_shared=128)
    size = lambda i: lib.moe_mx4_weight_bytes(ctypes.byref(cfg), i)
    tile = 16384 + 1024  # 128 columns x 256 of k
    assert [size(i) for i in range(-1, 5)] == [0, 3 * 2 * 2 * 2 * tile, 3 * 3 * 1 * tile, 2 * 1 * 2 * tile, 3 * 1 * tile, 0]
    none = ops.make_config(1, 384, 3, 1, 256)
    assert lib.moe_mx4_weight_bytes(ctypes.byref(none), 2) == 0 and lib.moe_mx4_weight_bytes(ctypes.byref(none), 3) == 0


def test_mx4_pointers(lib):
    for fn, ptrs in ((lambda a, M, K: lib.moe_mx4_quantize(a[0], M, K, a[1], a[2], None), 3),
                     (lambda a, M, K: lib.moe_mx4_dequantize(a[0], a[1], M, K, a[2], None), 3)):
        good = [P(4096)] * ptrs
        assert fn(good, 0, 32) == BAD and fn(good, 4, 0) == BAD and fn(good, 4, 48) == SHAPE and fn(good, 1 << 60, 32) == SHAPE
        for i in range(ptrs):
            for v in (P(None), P(4104)):
                a = list(good)
                a[i] = v
                assert fn(a, 4, 32) == BAD
    cfg = ops.make_config(1, 128, 2, 1, 128, F_shared=128)
    for i in range(6):
        for v in (P(None), P(4104)):
            p = [P(4096)] * 6
            p[i] = v
            assert lib.moe_mx4_quantize_weights(ctypes.byref(cfg), *p, _weights(4096, 4096, 4096, 4096), None) == BAD
            assert lib.moe_mx4_dequantize_weights(ctypes.byref(cfg), _weights(4096, 4096, 4096, 4096), *p, None) == BAD
    assert lib.moe_mx4_quantize_weights(ctypes.byref(cfg), *[P(4096)] * 6, _weights(4096, 4096, 4096, None), None) == BAD
    assert lib.moe_mx4_quantize_weights(None, *[P(4096)] * 6, _weights(4096, 4096, 4096, 4096), None) == BAD


@pytest.mark.parametrize("over,code", [(dict(T=0), BAD), (dict(H=0), BAD), (dict(eps=-1e-6), BAD), (dict(eps=float("nan")), BAD),
                                       (dict(gate=3), BAD), (dict(gate=-1), BAD), (dict(residual_scale=float("nan")), BAD),
                                       (dict(H=12), SHAPE), (dict(H=16392), SHAPE)])
def test_norm_configs(lib, over, code):
    cfg = ops.make_norm_config(**(dict(T=4, H=64) | over))
    assert lib.moe_norm_workspace_bytes(ctypes.byref(cfg)) == 0
    assert lib.moe_block_norm_fwd(ctypes.byref(cfg), *[P(4096)] * 8, None) == code
    assert lib.moe_block_norm_bwd(ctypes.byref(cfg), *[P(4096)] * 14, 1 << 40, None) == code


def test_norm_pointers(lib):
    cfg = ops.make_norm_config(4, 64, gate="channel", post=True)
    bwd = lambda p: lib.moe_block_norm_bwd(ctypes.byref(cfg), *p, 16, None)
    assert bwd(_apart(14)) == SMALL
    for i in range(14):
        for v in (P(None), P(((i + 1) << 24) + 8)):
            p = _apart(14)
            p[i] = v
            assert bwd(p) == (SMALL if v.value is None and i == 0 else BAD), (i, v)
    fwd = lambda p: lib.moe_block_norm_fwd(ctypes.byref(cfg), *p, None)
    for i in (0, 1, 2, 3, 4, 6, 7):
        p = _apart(8)
        p[i] = P(None)
        assert fwd(p) == BAD, i
    for i in range(8):
        p = _apart(8)
        p[i] = P(((i + 1) << 24) + 8)
        assert fwd(p) == BAD, i
    # neither h nor n
    bare = ops.make_norm_config(4, 64, pre=False)
    p = _apart(8)
    p[5] = p[6] = P(None)
    assert lib.moe_block_norm_fwd(ctypes.byref(bare), *p, None) == BAD
    assert lib.moe_block_norm_bwd(ctypes.byref(bare), None, *_apart(13), 1 << 40, None) == BAD  # no gradient at all


def test_norm_refuses_overlapping_outputs(lib):
    # order forward: y residual post gate pre h n stats; backward: dh dn y residual post gate pre stats dy dresidual dpost dgate dpre ws
    cfg = ops.make_norm_config(4, 64, gate="channel", post=True)
    nbytes = 4 * 64 * 2
    for a, b in ((5, 0), (5, 1), (6, 0), (6, 1), (6, 5), (7, 0), (7, 5), (5, 2), (6, 4), (7, 3)):
        p = _apart(8)
        p[a] = P(p[b].value + 16)
        assert lib.moe_block_norm_fwd(ctypes.byref(cfg), *p, None) == BAD, (a, b)
    for out in range(8, 14):
        for other in range(14):
            if other == out:
                continue
            p = _apart(14)
            p[out] = P(p[other].value + 16)
            assert lib.moe_block_norm_bwd(ctypes.byref(cfg), *p, 16, None) == BAD, (out, other)
    for out, over in ((9, 0), (8, 1)):  # dresidual over dh, dy over dn
        p = _apart(14)
        p[out] = p[over]
        assert lib.moe_block_norm_bwd(ctypes.byref(cfg), *p, 16, None) == SMALL
    p = _apart(14)
    p[8] = P(p[1].value + nbytes)  # behind it
    assert lib.moe_block_norm_bwd(ctypes.byref(cfg), *p, 16, None) == SMALL


def test_mx4_refuses_overlaps(lib):
    x, q, s = 1 << 24, 2 << 24, 3 << 24
    call = lambda x, q, s: {lib.moe_mx4_quantize(P(x), 4, 64, P(q), P(s), None), lib.moe_mx4_dequantize(P(q), P(s), 4, 64, P(x), None)}
    for a in ((x, x + 496, s), (x, x - 112, s), (x, q, x + 16), (x, q, q + 112), (x, x, s)):
        assert call(*a) == {BAD}, a
    cfg = ops.make_config(1, 128, 2, 1, 128, F_shared=128)
    for i in range(4):
        for over in list(range(1, 7)) + [10 + j for j in range(4) if j != i]:
            w = [(10 + j) << 24 for j in range(4)]
            w[i] = (over << 24) + 16
            p = _apart(6)
            assert lib.moe_mx4_quantize_weights(ctypes.byref(cfg), *p, _weights(*w), None) == BAD, (i, over)
            assert lib.moe_mx4_dequantize_weights(ctypes.byref(cfg), _weights(*w), *p, None) == BAD, (i, over)


def test_norm_rows_beyond_32_bit_indices_are_refused(lib):
    # a thread's next row, row + blocks, would pass 2^31
    for T in ((1 << 30) + 1, (1 << 31) - 1):
        cfg = ops.make_norm_config(T, 8)
        assert lib.moe_norm_workspace_bytes(ctypes.byref(cfg)) == 0
        far = [P((i + 1) << 44) for i in range(14)]
        assert lib.moe_block_norm_fwd(ctypes.byref(cfg), *far[:8], None) == SHAPE
        assert lib.moe_block_norm_bwd(ctypes.byref(cfg), *far, 1 << 40, None) == SHAPE
