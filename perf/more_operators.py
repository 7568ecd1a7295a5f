"""Timed cases of the layer's decoding form, its 4-bit weights and the norms around it.

Three operators, each beside what the layer already computes:

* the norms before and after the MoE block with its gate and the scaled residual: forward, and
  forward with backward (``norm``);
* the whole layer for a few tokens, router to combine, with bf16 weights or with MXFP4 ones
  (``few``);
* MXFP4 quantisation of rows and of the layer's weights, and the way back (``mx4``).

``run`` computes a case either in plain torch operations (``own`` false: fp32, the router's
selection in fp64, rounded once at the end) or through this package's entry points (``own`` true).
"""
import math

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of four requests: residual sum and the block's norm, launch latency alone
        _norm("norm_decode", T=4, H=4096, gate="none", post=False, residual=True, pre=True),
        # the Qwen3-shaped training step: residual sum and norm of 16384 tokens, forward and backward
        _norm("norm_train", T=16384, H=4096, gate="none", post=False, residual=True, pre=True, backward=True),
        # norms before and after the block, its output gated per channel, fp32 residual stream, odd row count
        _norm("norm_sandwich_train", T=5003, H=7168, gate="channel", post=True, residual=True, pre=True,
              residual_fp32=True, residual_scale=0.8, backward=True),
        # one token of one request through a Qwen3-shaped layer: eight experts' weights are read
        _few("few_one_token", T=1, H=4096, E=128, k=8, F=1536),
        # a few requests through a DeepSeek-V3-shaped layer: group-limited sigmoid router, shared expert
        _few("few_shared_grouped", T=7, H=7168, E=256, k=8, F=2048, F_shared=2048, score="sigmoid", groups=8,
             topk_groups=4, gate_scale=2.5),
        # a decoding batch of an odd size: nearly every expert is read for a few rows each
        _few("few_batch", T=61, H=4096, E=128, k=8, F=1536),
        # few wide experts (Mixtral-shaped), several rows each, fp32 result
        _few("few_wide", T=16, H=4096, E=8, k=2, F=14336, out_fp32=True),
        # the one-token and the batch step with 4-bit weights: a quarter of the bytes
        _few("few_mxfp4_one_token", T=1, H=4096, E=128, k=8, F=1536, mxfp4=True),
        _few("few_mxfp4_batch", T=33, H=4096, E=128, k=8, F=1536, mxfp4=True),
        # rows to MXFP4 and back: a small odd matrix, and activations of a large batch
        _mx4("mx4_rows_small", M=257, K=1504),
        _mx4("mx4_rows", M=16384, K=4096),
        # the weights of a layer with 32 experts, once after loading or after an update
        _mx4("mx4_weights", E=32, H=4096, F=1536),
    ]


def _norm(name, T, H, gate, post, residual, pre, residual_fp32=False, residual_scale=1.0, backward=False):
    return {"name": name, "op": "norm", "T": T, "H": H, "gate": gate, "post": post, "residual": residual, "pre": pre,
            "residual_fp32": residual_fp32, "residual_scale": residual_scale, "backward": backward}


def _few(name, T, H, E, k, F, F_shared=0, score="softmax", groups=1, topk_groups=1, gate_scale=1.0, out_fp32=False,
         mxfp4=False):
    return {"name": name, "op": "few", "T": T, "H": H, "E": E, "k": k, "F": F, "F_shared": F_shared, "score": score,
            "groups": groups, "topk_groups": topk_groups, "gate_scale": gate_scale, "out_fp32": out_fp32,
            "mxfp4": mxfp4}


def _mx4(name, M=0, K=0, E=0, H=0, F=0):
    return {"name": name, "op": "mx4", "M": M, "K": K, "E": E, "H": H, "F": F}


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "few", "few", "mx4"])
    if op == "norm":
        backward = rng.random() < 0.5
        case = _norm("", T=_spread(rng, 1, 10000), H=8 * _spread(rng, 16, 896),
                     gate=rng.choice(["none", "channel", "token"]), post=rng.random() < 0.5,
                     residual=rng.random() < 0.8, pre=True, residual_fp32=rng.random() < 0.4,
                     residual_scale=rng.choice([1.0, 0.5, 0.8]), backward=backward)
    elif op == "few":
        mxfp4 = rng.random() < 0.5
        unit = 128 if mxfp4 else 64
        E = rng.choice([4, 8, 16, 32, 60, 64, 100, 128])
        k = rng.randint(1, min(E, 8))
        grouped = E % 4 == 0 and E >= 16 and rng.random() < 0.3 and k <= E // 2
        H = unit * _spread(rng, 4, 5120 // unit)
        # at most 2^32 weights in all
        F = unit * _spread(rng, 2, max(2, min(8192, (1 << 32) // (3 * E * H)) // unit))
        case = _few("", T=_spread(rng, 1, 64), H=H, E=E, k=k, F=F,
                    F_shared=rng.choice([0, 0, unit * rng.randint(1, 2048 // unit)]),
                    score=rng.choice(["softmax", "sigmoid"]), groups=4 if grouped else 1,
                    topk_groups=2 if grouped else 1, gate_scale=rng.choice([1.0, 2.5]), out_fp32=rng.random() < 0.3,
                    mxfp4=mxfp4)
    elif rng.random() < 0.7:
        case = _mx4("", M=_spread(rng, 1, 16384), K=32 * _spread(rng, 1, 128))
    else:
        case = _mx4("", E=_spread(rng, 1, 32), H=128 * _spread(rng, 1, 32), F=128 * _spread(rng, 1, 12))
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _weights(g, E, K, N):
    """[E, K, N] bf16 weights scaled by their fan-in, drawn an expert at a time."""
    w = torch.empty((E, K, N), dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        w[e] = torch.randn((K, N), generator=g, device="cuda") * K ** -0.5
    return w


def _on_grid(w):
    """The values that MXFP4 with blocks along a matrix's rows (axis -2) makes of bf16 weights, in place."""
    for e in range(w.shape[0]):
        w[e] = _round_mx4(w[e].float().t().contiguous()).t()
    return w


def prepare(case, seed):
    g = _gen(seed)
    state = dict(case)
    bf = torch.bfloat16
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        stream = torch.float32 if case["residual_fp32"] else bf
        # tokens of a residual stream differ in size, a few channels are large
        size = torch.exp(0.5 * _normal(g, (T, 1)))
        channel = torch.exp(0.7 * _normal(g, (1, H)))
        state["y"] = (_normal(g, (T, H)) * size).to(bf)
        state["residual_in"] = (_normal(g, (T, H)) * size * channel).to(stream) if case["residual"] else None
        state["post_w"] = 1.0 + 0.2 * _normal(g, (H,)) if case["post"] else None
        state["pre_w"] = 1.0 + 0.2 * _normal(g, (H,)) if case["pre"] else None
        state["gate_v"] = {"none": None, "channel": 0.5 + 0.2 * _normal(g, (H,)),
                           "token": torch.sigmoid(_normal(g, (T,)))}[case["gate"]]
        if case["backward"]:
            state["dh"] = _normal(g, (T, H), 0.1, stream)
            state["dn"] = _normal(g, (T, H), 0.1, bf)
        if own:
            from route_permute_grouped_gb300 import ops
            cfg = ops.make_norm_config(T, H, eps=EPS, residual=case["residual"],
                                       residual_scale=case["residual_scale"], gate=case["gate"], post=case["post"],
                                       pre=case["pre"], residual_fp32=case["residual_fp32"])
            state["cfg"], state["ws"] = cfg, ops.norm_workspace(cfg)
    elif case["op"] == "few":
        T, H, E, F, Fs = (case[n] for n in ("T", "H", "E", "F", "F_shared"))
        state["x"] = _normal(g, (T, H), 1.0, bf)
        # logits of a trained router spread over a few units
        state["router_w"] = _normal(g, (E, H), 1.5 * H ** -0.5, bf)
        state["expert_bias"] = 0.2 * torch.rand(E, generator=g, device="cuda") - 0.1 if case["score"] == "sigmoid" else None
        W = {"W1": _weights(g, E, H, F), "W3": _weights(g, E, H, F), "W2": _weights(g, E, F, H)}
        if Fs:
            W |= {"Ws1": _weights(g, 1, H, Fs), "Ws3": _weights(g, 1, H, Fs), "Ws2": _weights(g, 1, Fs, H)}
        shared = lambda: [W[n][0] for n in ("Ws1", "Ws3", "Ws2")] if Fs else None
        if own:
            from route_permute_grouped_gb300 import ops
            cfg = ops.make_config(T, H, E, case["k"], F, F_shared=Fs, score=case["score"], n_groups=case["groups"],
                                  topk_groups=case["topk_groups"], gate_scale=case["gate_scale"],
                                  out_fp32=case["out_fp32"])
            state["cfg"], state["ws"] = cfg, ops.few_workspace(cfg, mxfp4=case["mxfp4"])
            if case["mxfp4"]:
                # a program that serves 4-bit weights holds nothing else of them
                state["q"] = ops.mx4_quantize_weights(cfg, W["W1"], W["W3"], W["W2"], Ws=shared())
                return state
        elif case["mxfp4"]:
            for n in W:
                _on_grid(W[n])
        state |= {n: W[n] for n in ("W1", "W3", "W2")}
        state["Ws"] = shared()
    elif case["M"]:
        # rows of activations: sizes differ from row to row and by channel
        M, K = case["M"], case["K"]
        state["x"] = (_normal(g, (M, K)) * torch.exp(_normal(g, (M, 1))) * torch.exp(0.7 * _normal(g, (1, K)))).to(bf)
    else:
        E, H, F = case["E"], case["H"], case["F"]
        state |= {"W1": _weights(g, E, H, F), "W3": _weights(g, E, H, F), "W2": _weights(g, E, F, H)}
        if own:
            from route_permute_grouped_gb300 import ops
            state["cfg"] = ops.make_config(1, H, E, 1, F)
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return {"norm": _run_norm, "few": _run_few, "mx4": _run_mx4}[state["op"]](state)


def _run_norm(s):
    y_in, res, post_w, pre_w, gate = (s[n] for n in ("y", "residual_in", "post_w", "pre_w", "gate_v"))
    if own:
        from route_permute_grouped_gb300 import ops
        h, n, stats = ops.block_norm_fwd(s["cfg"], y_in, residual=res, post_weight=post_w, gate=gate, pre_weight=pre_w)
        out = {"h": h, "n": n}
        if s["backward"]:
            out |= ops.block_norm_bwd(s["cfg"], s["dn"], y_in, stats, dh=s["dh"], residual=res, post_weight=post_w,
                                      gate=gate, pre_weight=pre_w, ws=s["ws"])
        return out
    stream = torch.float32 if s["residual_fp32"] else torch.bfloat16
    a = s["residual_scale"]
    y = y_in.float()
    g = None if gate is None else (gate[None, :] if s["gate"] == "channel" else gate[:, None])
    ry = torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) if s["post"] else None
    u = y * ry * post_w if s["post"] else y
    h = u if g is None else u * g
    if res is not None:
        h = h + a * res.float()
    out = {"h": h.to(stream)}
    rh = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    out["n"] = (h * rh * pre_w).to(torch.bfloat16)
    if not s["backward"]:
        return out
    dn = s["dn"].float()
    hh = h * rh
    dhh = dn * pre_w
    dh = s["dh"].float() + rh * (dhh - hh * (dhh * hh).mean(1, keepdim=True))
    out["dpre"] = (dn * hh).sum(0)
    if res is not None:
        out["dresidual"] = (a * dh).to(stream)
    if s["gate"] == "channel":
        out["dgate"] = (dh * u).sum(0)
    elif s["gate"] == "token":
        out["dgate"] = (dh * u).sum(1)
    du = dh if g is None else dh * g
    if s["post"]:
        yy = y * ry
        out["dpost"] = (du * yy).sum(0)
        dyy = du * post_w
        du = ry * (dyy - yy * (dyy * yy).mean(1, keepdim=True))
    out["dy"] = du.to(torch.bfloat16)
    return out


def _route(s):
    """Selected experts and gates of every token, the scores in fp64."""
    E, k = s["E"], s["k"]
    logits = s["x"].double() @ s["router_w"].double().t()
    score = torch.softmax(logits, 1) if s["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-logits))
    z = score if s["expert_bias"] is None else score + s["expert_bias"].double()
    if s["groups"] > 1:
        per = z.view(-1, s["groups"], E // s["groups"])
        two = torch.sort(per, dim=2, descending=True)[0][:, :, :2].sum(2)
        kept = torch.sort(two, dim=1, descending=True, stable=True)[1][:, :s["topk_groups"]]
        keep = (kept[:, :, None] == torch.arange(s["groups"], device="cuda")).any(1)
        z = torch.where(keep[:, :, None], per, -math.inf).view(-1, E)
    idx = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :k]
    w = torch.gather(score, 1, idx)
    return idx, s["gate_scale"] * w / w.sum(1, keepdim=True)


def _run_few(s):
    if own:
        from route_permute_grouped_gb300 import ops
        if s["mxfp4"]:
            y, idx, gate = ops.layer_few_fwd_mxfp4(s["cfg"], s["x"], s["router_w"], s["q"],
                                                   expert_bias=s["expert_bias"], ws=s["ws"])
        else:
            y, idx, gate = ops.layer_few_fwd(s["cfg"], s["x"], s["router_w"], s["W1"], s["W3"], s["W2"],
                                             expert_bias=s["expert_bias"], Ws=s["Ws"], ws=s["ws"])
        return {"y": y, "topk_idx": idx, "topk_gate": gate}
    idx, gate = _route(s)
    gate = gate.float()
    x = s["x"].float()
    T, E, k = s["T"], s["E"], s["k"]

    def expert(rows, W1, W3, W2, weight=None):
        h = rows @ W1.float()
        a = h / (1.0 + torch.exp(-h)) * (rows @ W3.float())
        return (a if weight is None else a * weight) @ W2.float()

    if T * k < E:
        # a product for each selected slot, with its expert's weights
        of = idx.reshape(-1)
        rows = x[:, None, :].expand(T, k, -1).reshape(T * k, 1, -1)
        y = expert(rows, s["W1"][of], s["W3"][of], s["W2"][of], gate.reshape(-1, 1, 1)).view(T, k, -1).sum(1)
    else:
        # every expert on every token, those that are not selected weighted 0
        weight = torch.zeros((T, E), device="cuda").scatter_(1, idx, gate).t().unsqueeze(2)
        y = expert(x, s["W1"], s["W3"], s["W2"], weight).sum(0)
    if s["Ws"] is not None:
        y = y + expert(x, *s["Ws"])
    return {"y": y if s["out_fp32"] else y.to(torch.bfloat16), "topk_idx": idx.to(torch.int32), "topk_gate": gate}


def _round_mx4(x):
    """Rows of fp32 values to the nearest values of MXFP4 (blocks of 32 along the rows)."""
    v = x.view(x.shape[0], -1, 32)
    top = v.abs().amax(2, keepdim=True)
    # 2^(floor(log2 top) - 2): E2M1's largest power of two is 4
    scale = torch.ldexp(torch.ones_like(top), torch.where(top > 0, torch.frexp(top)[1] - 3, 0).clamp(min=-126))
    m = (v / scale).abs()
    # halfway values go to the even code
    q = (0.5 * ((m > 0.25).float() + (m >= 0.75).float() + (m > 1.25).float() + (m >= 1.75).float())
         + (m > 2.5).float() + (m >= 3.5).float() + 2.0 * (m > 5.0).float())
    return (torch.sign(v) * q * scale).view_as(x)


def _run_mx4(s):
    if own:
        from route_permute_grouped_gb300 import ops
        if s["M"]:
            codes, scales = ops.mx4_quantize(s["x"])
            return {"values": ops.mx4_dequantize(codes, scales)}
        q = ops.mx4_quantize_weights(s["cfg"], s["W1"], s["W3"], s["W2"])
        W1, W3, W2, _ = ops.mx4_dequantize_weights(s["cfg"], q)
        return {"W1": W1, "W3": W3, "W2": W2}
    if s["M"]:
        return {"values": _round_mx4(s["x"].float()).to(torch.bfloat16)}
    # blocks lie along the axis that the product sums over
    along = lambda w: _round_mx4(w.float().transpose(1, 2).reshape(-1, w.shape[1])).view(
        w.shape[0], w.shape[2], w.shape[1]).transpose(1, 2).to(torch.bfloat16).contiguous()
    return {n: along(s[n]) for n in ("W1", "W3", "W2")}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        stream = 4 if case["residual_fp32"] else 2
        res = stream if case["residual"] else 0
        gate = {"none": 0, "channel": 4 * H, "token": 4 * T}[case["gate"]]
        small = gate + 4 * H * (case["post"] + case["pre"])
        # forward: y and the residual in, h and n out
        b = T * H * (2 + res + stream + 2) + small
        f = T * H * (5 + 4 * case["post"])
        if case["backward"]:
            # y, the residual, dh and dn in, dy and the residual's gradient out
            b += T * H * (2 + res + stream + 2 + 2 + res) + 2 * small
            f += T * H * (14 + 12 * case["post"])
        return {"bytes": b, "flops": f}
    if case["op"] == "few":
        T, H, E, k, F, Fs = (case[n] for n in ("T", "H", "E", "k", "F", "F_shared"))
        used = E * (1.0 - (1.0 - k / E) ** T)  # experts that an even router selects at least once
        weight = 0.53125 if case["mxfp4"] else 2
        b = 3 * H * weight * (used * F + Fs) + 2 * E * H + 2 * T * H + (4 if case["out_fp32"] else 2) * T * H + 8 * T * k
        return {"bytes": int(b), "flops": 6 * T * H * (k * F + Fs) + 2 * T * E * H}
    n = case["M"] * case["K"] if case["M"] else 3 * case["E"] * case["H"] * case["F"]
    # bf16 in, codes and scales out and in again, bf16 out
    return {"bytes": int(n * (2 + 2 * 0.53125 + 2)), "flops": 4 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed) if not own else _prepare_plain(case, seed)
    return {"norm": _exact_norm, "few": _exact_few, "mx4": _exact_mx4}[case["op"]](s)


def _prepare_plain(case, seed):
    global own
    own = False
    try:
        return prepare(case, seed)
    finally:
        own = True


def _exact_norm(s):
    d = lambda n: None if s.get(n) is None else s[n].double()
    y, res, post, pre, gate = d("y"), d("residual_in"), d("post_w"), d("pre_w"), d("gate_v")
    H, a = s["H"], s["residual_scale"]
    if gate is None:
        gate = torch.ones((), dtype=torch.float64, device="cuda")
    elif s["gate"] == "token":
        gate = gate.unsqueeze(1)
    norm = lambda v: torch.linalg.vector_norm(v, dim=1, keepdim=True).square().div(H).add(EPS).sqrt()
    sy = norm(y) if post is not None else None
    u = y if post is None else y / sy * post
    h = gate * u
    if res is not None:
        h += a * res
    sh = norm(h)
    out = {"h": h, "n": h / sh * pre}
    if not s["backward"]:
        return out
    # d(v / s)/dv with s^2 = |v|^2 / H + eps: (g - v <g, v> / (H s^2)) / s
    back = lambda g, v, sv: (g - v * (g * v).sum(1, keepdim=True) / (H * sv * sv)) / sv
    dn = d("dn")
    dh = d("dh") + back(dn * pre, h, sh)
    out["dpre"] = torch.einsum("th,th->h", dn, h / sh)
    if res is not None:
        out["dresidual"] = a * dh
    if s["gate"] != "none":
        out["dgate"] = torch.einsum("th,th->h" if s["gate"] == "channel" else "th,th->t", dh, u)
    du = gate * dh
    if post is not None:
        out["dpost"] = torch.einsum("th,th->h", du, y / sy)
        du = back(du * post, y, sy)
    out["dy"] = du
    return out


def _exact_few(s):
    x, wr = s["x"].double(), s["router_w"].double()
    T, E, k = s["T"], s["E"], s["k"]
    logits = x @ wr.t()
    p = torch.sigmoid(logits) if s["score"] == "sigmoid" else torch.softmax(logits, 1)
    idx = torch.zeros((T, k), dtype=torch.int32)
    gates = torch.zeros((T, k), dtype=torch.float64)
    scores = p.tolist()
    bias = [0.0] * E if s["expert_bias"] is None else s["expert_bias"].double().tolist()
    size = E // s["groups"]
    for t in range(T):
        sel = [scores[t][e] + bias[e] for e in range(E)]
        group = [sum(sorted(sel[i * size:(i + 1) * size])[-2:]) for i in range(s["groups"])]
        best = sorted(range(s["groups"]), key=lambda i: (-group[i], i))[:s["topk_groups"]]
        of = sorted((e for i in best for e in range(i * size, (i + 1) * size)), key=lambda e: (-sel[e], e))[:k]
        total = sum(scores[t][e] for e in of)
        for i, e in enumerate(of):
            idx[t, i], gates[t, i] = e, s["gate_scale"] * scores[t][e] / total
    weight = torch.zeros((T, E), dtype=torch.float64).scatter_(1, idx.long(), gates).cuda()
    y = torch.zeros_like(x)
    for e in sorted(set(idx.flatten().tolist())):
        t = torch.nonzero(weight[:, e])[:, 0]
        h1, h3 = x[t] @ s["W1"][e].double(), x[t] @ s["W3"][e].double()
        y[t] += weight[t, e, None] * ((h1 * torch.sigmoid(h1) * h3) @ s["W2"][e].double())
    if s["Ws"] is not None:
        W1, W3, W2 = (w.double() for w in s["Ws"])
        y += (torch.nn.functional.silu(x @ W1) * (x @ W3)) @ W2
    return {"y": y, "topk_idx": idx.cuda(), "topk_gate": gates.cuda()}


def _exact_mx4(s):
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")

    def nearest(w, axis):
        """Values of blocks of 32 along an axis: the closest grid value times the block's power of two."""
        v = w.double().movedim(axis, -1)
        b = v.reshape(-1, 32)
        # fp32 holds bf16 magnitudes: its exponent field gives floor(log2)
        top = b.abs().amax(1, keepdim=True).float()
        unit = torch.exp2(((top.view(torch.int32) >> 23) - 127 - 2).clamp(min=-127).double())
        m = b.abs() / unit
        hi = torch.searchsorted(grid, m.contiguous()).clamp(max=7)
        lo = (hi - 1).clamp(min=0)
        up, down = grid[hi] - m, m - grid[lo]
        code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        return (torch.sign(b) * grid[code] * unit).view(v.shape).movedim(-1, axis)

    if s["M"]:
        return {"values": nearest(s["x"], 1)}
    return {n: torch.stack([nearest(w, 0) for w in s[n]]) for n in ("W1", "W3", "W2")}
