"""Pins of the fp64 oracle of the few-token layer, MXFP4 and the block norms. CPU only."""
import numpy as np
import pytest

import oracle as O
from oracle import decode_oracle as DO


def test_mx4_values_are_the_nearest_and_ties_go_to_the_even_code():
    m = np.array([0.0, 0.2, 0.25, 0.26, 0.74, 0.75, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 6.0, 7.9])
    want = np.array([0.0, 0.0, 0.0, 0.5, 0.5, 1.0, 1.0, 1.5, 2.0, 2.0, 3.0, 4.0, 4.0, 6.0, 6.0, 6.0])
    assert np.array_equal(DO.E2M1[DO.mx4_codes(m)], want)


def test_mx4_blocks():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((7, 96)) * np.exp2(rng.integers(-30, 30, (7, 1)))
    x[0, :32] = 0.0
    x[1, 40] = np.inf
    x[2, 70] = np.nan
    codes, scales, v = DO.mx4_quantize(x)
    assert scales[0, 0] == 0 and not v[0, :32].any()
    assert scales[1, 1] == 255 and np.isnan(v[1, 32:64]).all() and np.isfinite(v[1, :32]).all()
    assert scales[2, 2] == 255 and np.isnan(v[2, 64:]).all()
    b = np.abs(x.reshape(7, 3, 32)).max(2)
    ok = np.isfinite(x.reshape(7, 3, 32)).all(2) & (b > 0)
    unit = np.exp2(scales[ok] - 127.0)
    assert ((b[ok] / unit >= 4) & (b[ok] / unit < 8)).all()
    # off by at most half the largest step, or by what saturates beyond 6
    err = np.abs(v - x).reshape(7, 3, 32)[ok].max(1)
    assert (err <= np.maximum(1.0, b[ok] / unit - 6) * unit).all()
    again = DO.mx4_quantize(np.nan_to_num(v))
    assert np.array_equal(again[2], np.nan_to_num(v))


def test_few_layer_is_the_layer():
    rng = np.random.default_rng(2)
    T, H, E, k, F, Fs = 5, 64, 8, 3, 32, 32
    x, wr = rng.standard_normal((T, H)), rng.standard_normal((E, H)) / 8
    W1, W3, W2 = (rng.standard_normal(s) / 8 for s in ((E, H, F), (E, H, F), (E, F, H)))
    Ws = [rng.standard_normal(s) / 8 for s in ((H, Fs), (H, Fs), (Fs, H))]
    opts = dict(score="sigmoid", expert_bias=rng.uniform(-.1, .1, E), n_groups=4, topk_groups=2, gate_scale=2.5)
    a = DO.few_layer(x, wr, W1, W3, W2, k, Ws=Ws, **opts)
    b = O.layer_fwd(x, wr, W1, W3, W2, k, Ws=Ws, prec=O.EXACT, **opts)
    assert np.array_equal(a["topk_idx"], b["topk_idx"])
    assert np.allclose(a["y"], b["y"], rtol=0, atol=1e-12 * np.abs(b["y"]).max())
    assert (a["dy"] > 0).all() and (a["dy"] < 1e-3 * np.abs(a["y"]).max()).all()


@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("pre", [False, True])
def test_norm_gradients_by_differences(gate, post, residual, pre):
    rng = np.random.default_rng(3)
    T, H = 3, 8
    p = {"y": rng.standard_normal((T, H))}
    if residual:
        p["residual"] = rng.standard_normal((T, H))
    if post:
        p["post"] = rng.standard_normal(H)
    if gate:
        p["gate"] = rng.standard_normal(H if gate == "channel" else T)
    if pre:
        p["pre"] = rng.standard_normal(H)
    dh, dn = rng.standard_normal((T, H)), rng.standard_normal((T, H)) if pre else None
    kw = dict(residual_scale=0.7, eps=1e-3)

    def loss(q):
        o, _ = DO.block_norm(**q, **kw)
        return (o["h"] * dh).sum() + ((o["n"] * dn).sum() if pre else 0.0)

    g, mag = DO.block_norm(**p, **kw, dh=dh, dn=dn)
    names = {"y": "dy", "residual": "dresidual", "post": "dpost", "gate": "dgate", "pre": "dpre"}
    for n, v in p.items():
        num = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            s = 1e-6
            a, b = v.copy(), v.copy()
            a[i] += s
            b[i] -= s
            num[i] = (loss({**p, n: a}) - loss({**p, n: b})) / (2 * s)
        assert np.abs(num - g[names[n]]).max() < 1e-7, n
        assert (np.abs(g[names[n]]) <= mag[names[n]] + 1e-12).all(), n
