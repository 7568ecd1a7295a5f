"""The fp64 oracle of the training-step operators, pinned: gradients against
central differences of its own values, the losses against the layer's aux loss
and hand-made cases. CPU only."""
import numpy as np
import pytest

from oracle import train_oracle as TO


def _logits(T, E, seed, std=1.5):
    return np.random.default_rng(seed).normal(0, std, (T, E))


def _topk(l, k):
    return np.argsort(-l, axis=1, kind="stable")[:, :k]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("off,mask", [(None, None), ([0, 3, 3, 9], None), ([1, 4, 8], [1, 0, 1, 1, 0, 0, 1, 1, 1, 1])])
def test_balance_gradient_against_differences(score, off, mask):
    T, E, k = 10, 6, 2
    if off is not None and mask is None:
        T = 9
    l = _logits(T, E, 3)
    idx = _topk(l, k)
    kw = dict(k=k, score=score, balance_coeff=0.3, z_coeff=0.07, seq_offsets=off, token_mask=mask)
    g = np.array([0.7, -1.3])
    _, _, d, _ = TO.balance(l, idx, dlosses=g, **kw)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            lp, lm = l.copy(), l.copy()
            lp[t, e] += h
            lm[t, e] -= h
            num = ((TO.balance(lp, idx, **kw)[0] - TO.balance(lm, idx, **kw)[0]) / (2 * h)) @ g
            # central difference: third derivatives are O(1) here, so h^2, plus 2^-53 / h
            assert abs(num - d[t, e]) < 1e-8


def test_balance_is_the_layers_aux_loss():
    l = _logits(40, 8, 5)
    idx = _topk(l, 2)
    p, _ = TO.router_probs(l, "softmax")
    c = np.bincount(idx.reshape(-1), minlength=8)
    losses, counts, _, _ = TO.balance(l, idx, 2, balance_coeff=0.01)
    assert np.array_equal(counts[0], c)
    assert abs(losses[0] - 0.01 * 8 * ((c / 80) * p.mean(0)).sum()) < 1e-15
    assert losses[1] == 0.0


def test_balance_uniform_router_has_loss_one():
    # equal scores and equal counts: f = 1, P = 1 / E, so the loss is alpha
    E, k, T = 4, 1, 8
    idx = (np.arange(T) % E)[:, None]
    for score in ("softmax", "sigmoid"):
        losses, _, d, _ = TO.balance(np.zeros((T, E)), idx, k, score=score, balance_coeff=2.0, z_coeff=1.0)
        assert abs(losses[0] - 2.0) < 1e-15 and abs(losses[1] - np.log(4) ** 2) < 1e-14


def test_adapter_gradients_against_differences():
    rng = np.random.default_rng(0)
    T, K, N, L, r = 7, 5, 4, 3, 2
    x, A, B = rng.normal(size=(T, K)), rng.normal(size=(L, K, r)), rng.normal(size=(L, r, N))
    scale, base, dy, dxb = rng.normal(size=L), rng.normal(size=(T, N)), rng.normal(size=(T, N)), rng.normal(size=(T, K))
    idx = np.array([0, 2, -1, 0, 2, 2, -1])
    out, _ = TO.adapter(x, A, B, scale, idx, base, dy, dxb)
    loss = lambda x, A, B: (TO.adapter(x, A, B, scale, idx, base)[0]["y"] * dy).sum()
    h = 1e-6
    for name, v, g in (("x", x, out["dx"] - dxb), ("A", A, out["dA"]), ("B", B, out["dB"])):
        for i in np.ndindex(v.shape):
            keep = v[i]
            v[i] = keep + h
            up = loss(x, A, B)
            v[i] = keep - h
            down = loss(x, A, B)
            v[i] = keep
            assert abs((up - down) / (2 * h) - g[i]) < 1e-7, name
    assert np.array_equal(out["y"][2], base[2]) and not out["dA"][1].any() and not out["dB"][1].any()


def test_grad_norm_and_clip():
    a, b = np.array([3.0]), np.array([[4.0, 0.0]])
    assert TO.grad_norm([a, b]) == 5.0 and TO.grad_norm([a, b], "max") == 4.0 and TO.grad_norm([]) == 0.0
    n, c = TO.clip([a, b], 1.0)
    assert n == 5.0 and abs(c[0][0] - 0.6) < 1e-6
    assert np.array_equal(TO.clip([a, b], 10.0)[1][1], b)
    assert np.isclose(TO.grad_norm([np.array([3e200, 4e200])]), 5e200, rtol=1e-15)
