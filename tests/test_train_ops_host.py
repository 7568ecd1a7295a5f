"""Host checks of the router losses, the adapters and the gradient norm: bad
arguments are refused before any CUDA work. CPU only (no call here launches)."""
import ctypes

import pytest
import torch

from route_permute_grouped_gb300 import build as B
from route_permute_grouped_gb300 import ops

OK, BAD, SHAPE, SMALL = ops.MOE_OK, ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_UNSUPPORTED_SHAPE, ops.MOE_ERR_WORKSPACE_TOO_SMALL
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    B.build()
    return ops.lib()


def _moved(call, n, optional=()):
    """call(ptrs) with every pointer aligned, then each one off by 8 bytes, then each one null."""
    assert call([P(4096)] * n) == SMALL
    for i in range(n):
        for v in (P(4104), P(None)):
            p = [P(4096)] * n
            p[i] = v
            want = SMALL if v.value is None and i in optional else BAD
            assert call(p) == want, (i, v)


@pytest.mark.parametrize("over,code", [(dict(T=0), BAD), (dict(E=0), BAD), (dict(k=0), BAD), (dict(k=9), BAD), (dict(n_seqs=0), BAD),
                                       (dict(score=2), BAD), (dict(balance_coeff=float("nan")), BAD),
                                       (dict(z_coeff=float("inf")), BAD), (dict(E=257), SHAPE), (dict(E=64, k=17), SHAPE),
                                       (dict(T=2 ** 30), SHAPE), (dict(n_seqs=65537), SHAPE)])
def test_balance_configs(lib, over, code):
    d = dict(T=64, E=8, k=2) | over
    cfg = ops.make_balance_config(**d)
    assert lib.moe_balance_workspace_bytes(ctypes.byref(cfg)) == 0 and lib.moe_balance_stats_floats(ctypes.byref(cfg)) == 0
    assert lib.moe_balance_loss_fwd(ctypes.byref(cfg), *[P(4096)] * 8, 1 << 40, None) == code
    assert lib.moe_balance_loss_bwd(ctypes.byref(cfg), *[P(4096)] * 6, None) == code
    with pytest.raises(ops.MoeError):
        ops.balance_workspace(cfg, "cpu")


def test_balance_pointers(lib):
    cfg = ops.make_balance_config(64, 8, 2)
    _moved(lambda p: lib.moe_balance_loss_fwd(ctypes.byref(cfg), *p, 16, None), 8, optional=(2, 3))
    many = ops.make_balance_config(64, 8, 2, n_seqs=3)
    assert lib.moe_balance_loss_fwd(ctypes.byref(many), P(4096), P(4096), None, *[P(4096)] * 5, 16, None) == BAD
    assert lib.moe_balance_loss_bwd(ctypes.byref(many), P(4096), P(4096), None, None, None, P(4096), None) == BAD
    assert lib.moe_balance_loss_fwd(None, *[P(4096)] * 8, 16, None) == BAD
    for i in (0, 1, 5):
        p = [P(4096)] * 6
        p[i] = P(None)
        assert lib.moe_balance_loss_bwd(ctypes.byref(cfg), *p, None) == BAD
    for i in range(6):
        p = [P(4096)] * 6
        p[i] = P(4104)
        assert lib.moe_balance_loss_bwd(ctypes.byref(cfg), *p, None) == BAD


@pytest.mark.parametrize("over,code", [(dict(T=0), BAD), (dict(K=0), BAD), (dict(N=-8), BAD), (dict(L=0), BAD), (dict(r=0), BAD),
                                       (dict(out_fp32=2), BAD), (dict(K=12), SHAPE), (dict(N=20), SHAPE), (dict(r=12), SHAPE),
                                       (dict(r=136), SHAPE), (dict(L=1025), SHAPE), (dict(T=2 ** 21 + 1), SHAPE)])
def test_adapter_configs(lib, over, code):
    cfg = ops.make_adapter_config(**(dict(T=64, K=64, N=64, L=4, r=16) | over))
    for n in (lib.moe_adapter_plan_bytes(ctypes.byref(cfg)), lib.moe_adapter_saved_bytes(ctypes.byref(cfg)),
              lib.moe_adapter_workspace_bytes(ctypes.byref(cfg), 1)):
        assert n == 0
    assert lib.moe_adapter_plan(ctypes.byref(cfg), P(4096), P(4096), 1 << 40, None) == code
    assert lib.moe_adapter_fwd(ctypes.byref(cfg), *[P(4096)] * 9, 1 << 40, None) == code
    assert lib.moe_adapter_bwd(ctypes.byref(cfg), *[P(4096)] * 12, 1 << 40, None) == code


def test_adapter_pointers(lib):
    cfg = ops.make_adapter_config(64, 64, 64, 4, 16)
    _moved(lambda p: lib.moe_adapter_plan(ctypes.byref(cfg), *p, 16, None), 2)
    _moved(lambda p: lib.moe_adapter_fwd(ctypes.byref(cfg), *p, 16, None), 9, optional=(5, 7))
    apart = lambda p: [P(None if q.value is None else q.value + (i << 24)) for i, q in enumerate(p)]
    _moved(lambda p: lib.moe_adapter_bwd(ctypes.byref(cfg), *apart(p), 16, None), 12, optional=(7,))
    assert lib.moe_adapter_plan(None, P(4096), P(4096), 1 << 40, None) == BAD


def test_adapter_refuses_overlapping_outputs(lib):
    # y over a shifted base, dx over x, dy or a shifted dx_base; the small workspace stops what is allowed
    cfg = ops.make_adapter_config(64, 64, 64, 4, 16)
    nbytes = 64 * 64 * 2
    def fwd(base, y):
        p = [P(1 << 20)] * 9
        p[5], p[6] = P(base), P(y)
        return lib.moe_adapter_fwd(ctypes.byref(cfg), *p, 16, None)
    assert fwd(1 << 16, 1 << 16) == SMALL and fwd(1 << 16, (1 << 16) + nbytes) == SMALL and fwd(None, 1 << 16) == SMALL
    assert fwd(1 << 16, (1 << 16) + 16) == BAD and fwd((1 << 16) + nbytes - 16, 1 << 16) == BAD
    def bwd(dy, x, dx_base, dx):
        p = [P((i + 1) << 24) for i in range(12)]
        p[0], p[1], p[7], p[8] = P(dy), P(x), P(dx_base), P(dx)
        return lib.moe_adapter_bwd(ctypes.byref(cfg), *p, 16, None)
    a, b, c, d = (i << 16 for i in (1, 2, 3, 4))
    assert bwd(a, b, c, d) == SMALL and bwd(a, b, c, c) == SMALL and bwd(a, b, None, d) == SMALL
    assert bwd(a, b, c, a) == BAD and bwd(a, b, c, b) == BAD and bwd(a, b, c, c + 32) == BAD and bwd(a, b, c, b + nbytes - 16) == BAD


def _build(lib, items, n=None):
    n = len(items) if n is None else n
    arr = (ops.MoeTensor * max(1, len(items)))(*[ops.MoeTensor(*i, 0) for i in items])
    size = lib.moe_tensor_list_bytes(n)
    buf = (ctypes.c_uint64 * (size // 8 + 1))()
    return lib.moe_tensor_list_build(arr, n, buf, size), buf


@pytest.mark.parametrize("items,code", [
    ([(4096, None, 100, 0)], OK), ([(4096, None, 0, 0), (None, None, 0, 1)], OK), ([], OK),
    ([(4096, None, 100, 3)], BAD), ([(4096, None, -1, 0)], BAD), ([(None, None, 5, 0)], BAD),
    ([(4098, None, 10, 0)], BAD), ([(4097, None, 10, 1)], BAD), ([(4098, None, 10, 1)], OK), ([(4096, 8194, 10, 0)], BAD),
    ([(4096, None, 100, 0), (4096, None, 100, 0)], BAD),          # the same tensor twice
    ([(4096, None, 100, 0), (4492, None, 100, 0)], BAD),          # the last element shared
    ([(4096, None, 100, 0), (4496, None, 100, 0)], OK),           # neighbours
    ([(4496, None, 100, 0), (4096, None, 101, 0)], BAD),
    ([(4096, 8192, 100, 0), (4096, 16384, 100, 0)], OK),          # read twice, written apart
    ([(4096, 8192, 100, 0), (20480, 8192, 100, 0)], BAD),         # two written to one place
    ([(4096, 4100, 100, 0)], BAD),                                # written over itself, shifted
    ([(4096, 4096, 100, 0)], OK),
    ([(4096, 8192, 100, 0), (8192, 20480, 100, 0)], BAD),         # written where another is read
    ([(4096, None, 1 << 42, 1)], SHAPE),
])
def test_tensor_lists(lib, items, code):
    assert _build(lib, items)[0] == code


def test_tensor_list_sizes(lib):
    assert lib.moe_tensor_list_bytes(-1) == 0 and lib.moe_tensor_list_bytes(49153) == 0
    assert 0 < lib.moe_tensor_list_bytes(0) < lib.moe_tensor_list_bytes(769) < lib.moe_tensor_list_bytes(49152)
    arr = (ops.MoeTensor * 1)(ops.MoeTensor(4096, None, 4, 0, 0))
    buf = (ctypes.c_uint64 * 10000)()
    assert lib.moe_tensor_list_build(arr, 1, buf, 64) == SMALL
    assert lib.moe_tensor_list_build(None, 1, buf, 80000) == BAD
    assert lib.moe_tensor_list_build(arr, 1, None, 80000) == BAD
    assert lib.moe_tensor_list_build(arr, 1, P(ctypes.addressof(buf) + 4), 79000) == BAD


def test_norm_calls(lib):
    st, buf = _build(lib, [(4096, None, 100, 0)])
    n = lib.moe_grad_norm_workspace_bytes()
    norm = lambda l, kind, out, ws, nb: lib.moe_grad_norm(l, kind, out, ws, nb, None)
    clip = lambda l, kind, out, ws, nb, m=1.0: lib.moe_clip_grad_norm(l, kind, m, out, ws, nb, None)
    for call in (norm, clip):
        assert call(None, 0, P(4096), P(4096), n) == BAD
        assert call(buf, 2, P(4096), P(4096), n) == BAD
        assert call(buf, 0, None, P(4096), n) == BAD and call(buf, 0, P(4096), None, n) == BAD
        assert call(buf, 0, P(4104), P(4096), n) == BAD and call(buf, 0, P(4096), P(4104), n) == BAD
        assert call(buf, 0, P(4096), P(4096), n - 1) == SMALL
        bad, broken = _build(lib, [(4096, None, 100, 0)] * 2)      # refused: not a list
        assert bad == BAD and call(broken, 0, P(4096), P(4096), n) == BAD
    for m in (-1.0, float("nan")):
        assert clip(buf, 0, P(4096), P(4096), n, m) == BAD


def test_binding_refuses_what_the_library_cannot_see(lib):
    cfg = ops.make_balance_config(4, 8, 2)
    logits, idx = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ops.MoeError, match="CUDA device"):
        ops.balance_loss_fwd(cfg, logits, idx)
    with pytest.raises(ops.MoeError, match="logits must be"):
        ops.balance_loss_fwd(cfg, logits.double(), idx)
    with pytest.raises(ops.MoeError, match="logits must be"):
        ops.balance_loss_fwd(cfg, torch.zeros(5, 8), idx)
    acfg = ops.make_adapter_config(4, 64, 64, 2, 8)
    with pytest.raises(ops.MoeError, match="adapter_idx"):
        ops.adapter_plan(acfg, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ops.MoeError, match="x must be"):
        ops.adapter_fwd(acfg, torch.zeros(4, 64), None, None, None, None)
    with pytest.raises(ops.MoeError, match="CUDA device"):
        ops.tensor_list([torch.zeros(4)])
    with pytest.raises(ops.MoeError, match="fp32, bf16 or fp16"):
        ops.tensor_list([torch.zeros(4, dtype=torch.float64)])
    with pytest.raises(ops.MoeError, match="contiguous"):
        ops.tensor_list([torch.zeros(4, 4).t()])
    with pytest.raises(ops.MoeError, match="one tensor for each"):
        ops.tensor_list([], out=[torch.zeros(4)])
