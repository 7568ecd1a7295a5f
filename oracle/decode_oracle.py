"""fp64 restatement of the layer for a few tokens, of MXFP4 and of the norms
around a block, with bounds on what fp32 sums and the operands' parts may add:
plain numpy, one expert, block or tensor at a time."""
import numpy as np

from .moe_oracle import route, silu

F32, BF16 = 2.0 ** -24, 2.0 ** -8  # half a step, relative

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ----------------------------------------------------------------------------
# MXFP4
# ----------------------------------------------------------------------------
def mx4_scale_exponent(amax):
    """floor(log2 amax) - 2, clamped to [-127, 127]; -127 for 0."""
    amax = np.asarray(amax, np.float64)
    e = np.where(amax > 0, np.frexp(np.where(amax > 0, amax, 1.0))[1] - 1 - 2, -127)
    return np.clip(e, -127, 127)


def mx4_codes(m):
    """Codes 0..7 of magnitudes: nearest value, a tie to the even code, 6 beyond."""
    m = np.minimum(np.asarray(m, np.float64), 6.0)
    hi = np.clip(np.searchsorted(E2M1, m, side="left"), 1, 7)
    lo = hi - 1
    up, down = E2M1[hi] - m, m - E2M1[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def mx4_quantize(x):
    """(codes [M, K] 0..15, scale bytes [M, K/32], values [M, K]) of rows."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(b).all(2)
    safe = np.where(bad[:, :, None], 0.0, b)
    s = mx4_scale_exponent(np.abs(safe).max(2))
    unit = np.exp2(s.astype(np.float64))[:, :, None]
    c = mx4_codes(np.abs(safe) / unit)
    values = np.copysign(E2M1[c] * unit, safe)
    values[bad] = np.nan
    codes = np.where(np.signbit(safe), c + 8, c)
    codes[bad] = 0
    return codes.reshape(x.shape), np.where(bad, 255, s + 127), values.reshape(x.shape)


def mx4_weights(w):
    """Values of a weight [.., K, N] quantised in blocks along K."""
    w = np.asarray(w, np.float64)
    t = np.swapaxes(w, -1, -2)
    v = mx4_quantize(t.reshape(-1, w.shape[-2]))[2]
    return np.swapaxes(v.reshape(t.shape), -1, -2)


# ----------------------------------------------------------------------------
# the layer for a few tokens
# ----------------------------------------------------------------------------
def _chain(K, per):
    """Bound, relative to the sum of magnitudes, of a product summed over K by the tensor
    cores (`per` products a step, each step cut off at one step of fp32) and of the fp32
    additions that join its parts."""
    return (K / per + 16) * 2.0 ** -23


def _block_max(v):
    """The largest magnitude of the 32 elements that each element shares a scale with."""
    b = np.abs(v).reshape(v.shape[0], -1, 32)
    return np.broadcast_to(b.max(2, keepdims=True), b.shape).reshape(v.shape)


def few_layer(x, w_r, W1, W3, W2, k, Ws=None, out_fp32=False, mxfp4=False, **router):
    """topk_idx, topk_gate, y and the bounds of the kernel's gates and y (before the
    rounding of y). mxfp4: the weights are quantised here."""
    x, w_r = np.asarray(x, np.float64), np.asarray(w_r, np.float64)
    r = route(x, w_r, k, **router)
    idx, gate = r["topk_idx"], r["topk_gate"]
    T, H = x.shape
    # a logit: chains of H / 2048 * 8 products and some twenty additions; a gate: a ratio of
    # exponentials of them
    dl = (H / 256 + 32) * F32 * (np.abs(x) @ np.abs(w_r).T)
    dgate = gate * (4 * dl.max(1, keepdims=True) + 64 * F32)
    per = 64 if mxfp4 else 16
    q = mx4_weights if mxfp4 else (lambda w: np.asarray(w, np.float64))
    # parts: an element of x or a within `part` of itself, or of the largest of its 32
    part = (2.0 ** -22 if out_fp32 else 2.0 ** -13) if mxfp4 else (2.0 ** -25 if out_fp32 else 2.0 ** -17)

    def expert(rows, g, dg, W1, W3, W2):
        W1, W3, W2 = q(W1), q(W3), q(W2)
        F = W1.shape[1]
        dx = part * _block_max(rows) if mxfp4 else np.zeros_like(rows)
        h1, h3 = rows @ W1, rows @ W3
        d1 = _chain(H, per) * (np.abs(rows) @ np.abs(W1)) + dx @ np.abs(W1)
        d3 = _chain(H, per) * (np.abs(rows) @ np.abs(W3)) + dx @ np.abs(W3)
        a = silu(h1) * h3
        # |silu'| < 1.1
        da = 1.1 * d1 * np.abs(h3) + np.abs(silu(h1)) * d3 + 1.1 * d1 * d3 + 16 * F32 * np.abs(a)
        ga = g * a
        dga = g * da + dg * (np.abs(a) + da) + part * (_block_max(ga) if mxfp4 else np.abs(ga))
        return ga @ W2, dga @ np.abs(W2) + _chain(F, per) * (np.abs(ga) @ np.abs(W2))

    y, dy = np.zeros((T, H)), np.zeros((T, H))
    for e in np.unique(idx):
        t, i = np.nonzero(idx == e)
        v, d = expert(x[t], gate[t, i][:, None], dgate[t, i][:, None], W1[e], W3[e], W2[e])
        y[t] += v
        dy[t] += d + 2 * F32 * np.abs(v)
    if Ws is not None:
        v, d = expert(x, np.ones((T, 1)), np.zeros((T, 1)), *Ws)
        y += v
        dy += d + 2 * F32 * np.abs(v)
    return {"topk_idx": idx, "topk_gate": gate, "dgate": dgate, "y": y, "dy": dy, "z": r["z"]}


# ----------------------------------------------------------------------------
# norms around a block
# ----------------------------------------------------------------------------
def _rms(v, eps):
    return 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def block_norm(y, residual=None, residual_scale=1.0, post=None, gate=None, pre=None, eps=1e-6, dh=None, dn=None):
    """h, n and, given the gradients dh (None: zeros) and dn, those of every input; `mag`
    bounds the magnitudes whose fp32 roundings add up in each."""
    f = lambda v: None if v is None else np.asarray(v, np.float64)
    y, residual, post, gate, pre, dh, dn = map(f, (y, residual, post, gate, pre, dh, dn))
    T, H = y.shape
    g = np.ones((1, 1)) if gate is None else gate[None, :] if gate.shape == (H,) else gate[:, None]
    if gate is not None and T == H:
        raise ValueError("ambiguous gate")
    ry = _rms(y, eps) if post is not None else np.ones((T, 1))
    w = np.ones(H) if post is None else post
    u = y * ry * w
    h = g * u
    big = np.abs(h)
    if residual is not None:
        h = h + residual_scale * residual
        big = big + np.abs(residual_scale * residual)
    out, mag = {"h": h}, {"h": big}
    rh = _rms(h, eps)
    if pre is not None:
        out["n"] = h * rh * pre
        # rh is off by what h is in the mean
        mag["n"] = rh * np.abs(pre) * (big + np.abs(h) * rh * np.sqrt((big * big).mean(1, keepdims=True)))
    if dh is None and dn is None:
        return out, mag
    dH = np.zeros_like(h) if dh is None else dh
    mH = np.abs(dH)
    if pre is not None:
        dw, hh, bh = dn * pre, h * rh, big * rh
        dH = dH + rh * (dw - hh * (dw * hh).mean(1, keepdims=True))
        mH = mH + rh * (np.abs(dw) + bh * (np.abs(dw) * bh).mean(1, keepdims=True) * (1 + 2 * (bh * bh).mean(1, keepdims=True)))
        out["dpre"], mag["dpre"] = (dn * hh).sum(0), (np.abs(dn) * bh).sum(0)
    if residual is not None:
        out["dresidual"], mag["dresidual"] = residual_scale * dH, np.abs(residual_scale) * mH
    if gate is not None:
        axis = 0 if gate.shape == (H,) else 1
        out["dgate"], mag["dgate"] = (dH * u).sum(axis), (mH * np.abs(u)).sum(axis)
    du, mu = g * dH, np.abs(g) * mH
    if post is not None:
        yy = y * ry
        out["dpost"], mag["dpost"] = (du * yy).sum(0), (mu * np.abs(yy)).sum(0)
        dyy, my = du * w, mu * np.abs(w)
        du = ry * (dyy - yy * (dyy * yy).mean(1, keepdims=True))
        mu = ry * (my + np.abs(yy) * (my * np.abs(yy)).mean(1, keepdims=True))
    out["dy"], mag["dy"] = du, mu
    return out, mag
