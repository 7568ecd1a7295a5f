"""Timed cases of the operators around the MoE layer's training step and its fine-tuned serving.

Three operators, each beside what the layer already computes:

* the router's balance loss and z-loss from the logits and the selected experts, with the expert
  counts of every sequence and the gradient of the logits (``balance``);
* low-rank adapters of many requests added to a shared projection's output, each row with the
  adapter of its request, forward and backward (``adapter``);
* the global norm of a list of gradients and its clipping (``clip``).

``run`` computes a case either in plain torch operations (``own`` false: fp32, fp64 for long sums,
rounded once at the end) or through this package's entry points (``own`` true).
"""
import math

import torch

own = False

INT = torch.int32


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one micro-batch of a Mixtral-shaped router (8 experts, top 2): the whole step is launch latency
        _balance("balance_e8_small", T=512, E=8, k=2, S=1, score="softmax", masked=False),
        # the Qwen3-shaped training step's router: 16384 tokens packed into a few sequences, some padding
        _balance("balance_e128_train", T=16384, E=128, k=8, S=5, score="softmax", masked=True),
        # DeepSeek-V3-shaped router (256 experts, sigmoid scores): sequence-wise loss of a large ragged batch
        _balance("balance_e256_ragged", T=131021, E=256, k=8, S=61, score="sigmoid", masked=True),
        # the same number of experts with the loss over the whole batch, nothing masked
        _balance("balance_e256_batch", T=65536, E=256, k=8, S=1, score="softmax", masked=False),
        # one decoded token of one request
        _adapter("adapter_one_token", T=1, K=4096, N=4096, L=8, r=16, order="random"),
        # a decode batch: 64 requests over 48 adapters, some rows without one
        _adapter("adapter_decode", T=64, K=7168, N=4096, L=48, r=16, order="random"),
        # prompts of several requests in one batch, ragged, into an fp32 output
        _adapter("adapter_prefill", T=4133, K=7168, N=2048, L=11, r=32, order="runs", out_fp32=True),
        # a fine-tuning step over sequences of a few adapters: forward, backward, adapter gradients
        _adapter("adapter_train", T=16384, K=4096, N=4096, L=8, r=64, order="runs", backward=True),
        # the same with rows of 40 adapters interleaved and an odd row count
        _adapter("adapter_train_mixed", T=5003, K=4096, N=1536, L=40, r=24, order="random", backward=True),
        # the adapters' own gradients: many small tensors of odd sizes
        _clip("clip_adapters", groups=96, sizes=[4096 * 16, 16 * 1531, 257, 1], dtypes=["float32"], max_norm=1.0),
        # bf16 gradients with fp32 ones among them, below the threshold: nothing is scaled
        _clip("clip_mixed_below", groups=6, sizes=[4096 * 1536, 128 * 4096 + 3, 4099], dtypes=["bfloat16", "float32"],
              max_norm=1e9, inplace=True),
        # every weight gradient of a layer with the Qwen3 expert shape and 32 experts
        _clip("clip_layer", groups=1, sizes=[32 * 4096 * 1536, 32 * 4096 * 1536, 32 * 4096 * 1536, 32 * 4096],
              dtypes=["float32"], max_norm=1.0),
    ]


def _balance(name, T, E, k, S, score, masked):
    return {"name": name, "op": "balance", "T": T, "E": E, "k": k, "S": S, "score": score, "masked": masked}


def _adapter(name, T, K, N, L, r, order, out_fp32=False, backward=False):
    return {"name": name, "op": "adapter", "T": T, "K": K, "N": N, "L": L, "r": r, "order": order,
            "out_fp32": out_fp32, "backward": backward}


def _clip(name, groups, sizes, dtypes, max_norm, inplace=False):
    # plain values only: the lists travel as text
    return {"name": name, "op": "clip", "groups": groups, "sizes": " ".join(map(str, sizes)),
            "dtypes": " ".join(dtypes), "max_norm": max_norm, "inplace": inplace}


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "adapter", "adapter", "clip"])
    if op == "balance":
        T = _spread(rng, 1, 131021)
        E = rng.choice([8, 16, 33, 60, 64, 100, 128, 160, 256])
        case = _balance("", T=T, E=E, k=rng.randint(1, min(E, 8)), S=_spread(rng, 1, 64),
                        score=rng.choice(["softmax", "sigmoid"]), masked=rng.random() < 0.5)
    elif op == "adapter":
        backward = rng.random() < 0.5
        case = _adapter("", T=_spread(rng, 1, 12000 if backward else 16384), K=8 * _spread(rng, 32, 640),
                        N=8 * _spread(rng, 32, 640), L=_spread(rng, 1, 64), r=8 * rng.randint(1, 8),
                        order=rng.choice(["random", "runs"]), out_fp32=rng.random() < 0.25, backward=backward)
    else:
        n = rng.randint(1, 5)
        groups = _spread(rng, 1, 64)
        most = max(64, 200_000_000 // (groups * n))
        case = _clip("", groups=groups, sizes=[_spread(rng, 1, most) for _ in range(n)],
                     dtypes=[rng.choice(["float32", "bfloat16", "float16"]) for _ in range(rng.randint(1, 2))],
                     max_norm=rng.choice([0.1, 1.0, 1e9]))
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


def _cuts(g, T, S):
    """Offsets [S+1] of S ragged sequences over T rows (some may be empty; the last rows of a
    batch of more than a thousand belong to none)."""
    end = T - T // 1024
    inner = (torch.rand(S - 1, generator=g, device="cuda") * (end + 1)).to(torch.int64).clamp_(max=end)
    ends = torch.tensor([0, end], device="cuda")
    return torch.sort(torch.cat([ends, inner]))[0].to(INT)


def prepare(case, seed):
    g = _gen(seed)
    state = dict(case)
    if case["op"] == "balance":
        T, E, k, S = (case[n] for n in "TEkS")
        # logits of a router in training: expert popularity differs, tokens agree in part
        popular = _normal(g, (1, E), 0.7)
        logits = _normal(g, (T, E), 1.5) + popular
        state["logits"] = logits
        state["topk_idx"] = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k].to(INT).contiguous()
        state["seq_offsets"] = _cuts(g, T, S)
        state["token_mask"] = (torch.rand(T, generator=g, device="cuda") > 0.06).to(torch.uint8) if case["masked"] else None
        state["dlosses"] = torch.tensor([1.0, 0.5], device="cuda")
        state["balance_coeff"], state["z_coeff"] = 1e-2, 1e-3
        if own:
            from route_permute_grouped_gb300 import ops
            cfg = ops.make_balance_config(T, E, k, n_seqs=S, score=case["score"], balance_coeff=1e-2, z_coeff=1e-3)
            state["cfg"], state["ws"] = cfg, ops.balance_workspace(cfg)
    elif case["op"] == "adapter":
        T, K, N, L, r = (case[n] for n in ("T", "K", "N", "L", "r"))
        state["x"] = _normal(g, (T, K), 1.0, torch.bfloat16)
        state["A"] = _normal(g, (L, K, r), K ** -0.5, torch.bfloat16)
        state["B"] = _normal(g, (L, r, N), 0.5 * r ** -0.5, torch.bfloat16)
        state["scale"] = 0.5 + 1.5 * torch.rand(L, generator=g, device="cuda")
        state["base"] = _normal(g, (T, N), 1.0, torch.float32 if case["out_fp32"] else torch.bfloat16)
        # -1: a request without an adapter (about one in sixteen)
        if case["order"] == "random":
            idx = torch.randint(0, L, (T,), generator=g, device="cuda")
            idx = torch.where(torch.rand(T, generator=g, device="cuda") < 1 / 16, -1, idx)
            if T == 1:
                idx = torch.randint(0, L, (T,), generator=g, device="cuda")
        else:
            runs = 2 * L + 1
            of_run = torch.randint(0, L, (runs,), generator=g, device="cuda")
            of_run = torch.where(torch.rand(runs, generator=g, device="cuda") < 1 / 16, -1, of_run)
            cuts = torch.sort((torch.rand(runs - 1, generator=g, device="cuda") * T).to(torch.int64))[0]
            idx = of_run[torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)]
        state["adapter_idx"] = idx.to(INT)
        if case["backward"]:
            state["dy"] = _normal(g, (T, N), 1.0, torch.bfloat16)
            state["dx_base"] = _normal(g, (T, K), 1.0, state["base"].dtype)
        if own:
            from route_permute_grouped_gb300 import ops
            cfg = ops.make_adapter_config(T, K, N, L, r, out_fp32=case["out_fp32"])
            state["cfg"], state["ws"] = cfg, ops.adapter_workspace(cfg, training=case["backward"])
    else:
        sizes = [int(n) for n in case["sizes"].split()]
        dtypes = [getattr(torch, d) for d in case["dtypes"].split()]
        # gradients are pieces of one flat buffer for each type, as optimizers keep them, so odd
        # sizes put the next tensor at an odd offset
        per_type = {d: [] for d in dtypes}
        state["grads"] = []
        for i in range(case["groups"] * len(sizes)):
            per_type[dtypes[i % len(dtypes)]].append(i)
        place = {}
        state["flat"], state["flat_out"] = [], []
        for d, mine in per_type.items():
            lengths = [sizes[i % len(sizes)] for i in mine]
            # gradients of different layers differ by orders of magnitude
            flat = _normal(g, (sum(lengths),), 1.0, d)
            out = flat if case["inplace"] else torch.empty_like(flat)
            state["flat"].append(flat)
            state["flat_out"].append(out)
            for i, a, b in zip(mine, flat.split(lengths), out.split(lengths)):
                a.mul_(10.0 ** -((i // len(sizes) + i % len(sizes)) % 4))
                place[i] = (a, b)
        state["grads"] = [place[i][0] for i in range(len(place))]
        state["out"] = [place[i][1] for i in range(len(place))]
        if own:
            from route_permute_grouped_gb300 import ops
            state["list"] = ops.tensor_list(state["grads"], out=None if case["inplace"] else state["out"])
            state["ws"] = ops.grad_norm_workspace()
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return {"balance": _run_balance, "adapter": _run_adapter, "clip": _run_clip}[state["op"]](state)


def _run_balance(s):
    if own:
        from route_permute_grouped_gb300 import ops
        losses, counts, stats = ops.balance_loss_fwd(s["cfg"], s["logits"], s["topk_idx"], s["seq_offsets"],
                                                     s["token_mask"], ws=s["ws"])
        dlogits = ops.balance_loss_bwd(s["cfg"], s["logits"], stats, s["dlosses"], s["seq_offsets"], s["token_mask"])
        return {"losses": losses, "counts": counts, "dlogits": dlogits}
    logits, T, E, k, S = s["logits"], s["T"], s["E"], s["k"], s["S"]
    row = torch.arange(T, device="cuda", dtype=INT)
    seq = torch.searchsorted(s["seq_offsets"][1:].contiguous(), row, right=True)
    valid = (row >= s["seq_offsets"][0]) & (seq < S)
    if s["token_mask"] is not None:
        valid = valid & (s["token_mask"] != 0)
    logits = torch.where(valid[:, None], logits, 0.0)
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    soft = e / total
    if s["score"] == "softmax":
        p = soft
    else:
        sg = 1.0 / (1.0 + torch.exp(-logits))
        sg_sum = sg.sum(1, keepdim=True)
        p = sg / sg_sum
    one_hot = ((seq[None, :] == torch.arange(S, device="cuda")[:, None]) & valid[None, :]).float()
    slot = torch.where(valid, seq, S)[:, None] * E + s["topk_idx"]
    counts = torch.zeros((S + 1) * E, dtype=INT, device="cuda").index_add_(
        0, slot.reshape(-1), torch.ones(T * k, dtype=INT, device="cuda"))[:S * E].view(S, E)
    n_seq = one_hot.double().sum(1)
    per = torch.where(n_seq > 0, 1.0 / n_seq.clamp(min=1), 0.0)
    share = 1.0 / (n_seq > 0).sum().clamp(min=1)
    n = n_seq.sum().clamp(min=1)
    mean_p = (one_hot @ p).double() * per[:, None]
    f = counts.double() * (E / k) * per[:, None]
    balance = s["balance_coeff"] * share * (f * mean_p).sum()
    z = s["z_coeff"] / n * torch.where(valid, lse, 0.0).double().square().sum()
    weight = s["dlosses"][0] * s["balance_coeff"] * share * per[:, None] * f
    dp = weight.float()[seq.clamp(max=S - 1)]
    inner = (p * dp).sum(1, keepdim=True)
    if s["score"] == "softmax":
        d = p * (dp - inner)
    else:
        d = sg * (1.0 - sg) / sg_sum * (dp - inner)
    dz = (2.0 * s["dlosses"][1] * s["z_coeff"] / n).float() * lse
    return {"losses": torch.stack([balance, z]).float(), "counts": counts,
            "dlogits": torch.where(valid[:, None], d + dz[:, None] * soft, 0.0)}


def _run_adapter(s):
    if own:
        from route_permute_grouped_gb300 import ops
        cfg, ws = s["cfg"], s["ws"]
        plan = ops.adapter_plan(cfg, s["adapter_idx"])
        if not s["backward"]:
            return {"y": ops.adapter_fwd(cfg, s["x"], s["A"], s["B"], s["scale"], plan, base=s["base"], ws=ws)}
        u = ops.alloc_adapter_saved(cfg)
        y = ops.adapter_fwd(cfg, s["x"], s["A"], s["B"], s["scale"], plan, base=s["base"], u=u, ws=ws)
        g = ops.adapter_bwd(cfg, s["dy"], s["x"], s["A"], s["B"], s["scale"], plan, u, dx_base=s["dx_base"], ws=ws)
        return {"y": y, "dx": g["dx"], "dA": g["dA"], "dB": g["dB"]}
    L, r, K, N, T = s["L"], s["r"], s["K"], s["N"], s["T"]
    # every row against every adapter side by side, the products of other adapters set to zero
    of_row = s["adapter_idx"][:, None] == torch.arange(L, device="cuda", dtype=INT)[None, :]
    pick = (of_row * s["scale"][None, :])[:, :, None]
    A = s["A"].float().permute(1, 0, 2).reshape(K, L * r)
    B = s["B"].float().reshape(L * r, N)
    x = s["x"].float()
    u = ((x @ A).view(T, L, r) * pick).view(T, L * r)
    out = {"y": (s["base"].float() + u @ B).to(s["base"].dtype)}
    if s["backward"]:
        dy = s["dy"].float()
        du = ((dy @ B.t()).view(T, L, r) * pick).view(T, L * r)
        out["dx"] = (s["dx_base"].float() + du @ A.t()).to(s["dx_base"].dtype)
        out["dA"] = (x.t() @ du).view(K, L, r).permute(1, 0, 2).contiguous()
        out["dB"] = (u.t() @ dy).view(L, r, N)
    return out


def _run_clip(s):
    if own:
        from route_permute_grouped_gb300 import ops
        norm = ops.clip_grad_norm(s["list"], s["max_norm"], ws=s["ws"])
        return {"norm": norm, "grads": s["flat_out"]}
    total = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]]).sum()
    norm = torch.sqrt(total).float()
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    [out.copy_(t.float() * coef) for t, out in zip(s["grads"], s["out"])]
    return {"norm": norm.view(1), "grads": s["flat_out"]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "balance":
        T, E, k, S = (case[n] for n in "TEkS")
        # the logits read once, their gradient written once
        b = 8 * T * E + 4 * T * k + 4 * (S + 1) + (T if case["masked"] else 0) + 4 * S * E + 8
        return {"bytes": b, "flops": 16 * T * E}
    if case["op"] == "adapter":
        T, K, N, L, r = (case[n] for n in ("T", "K", "N", "L", "r"))
        out = 4 if case["out_fp32"] else 2
        used = min(T, L)  # at most so many adapters are read
        b = 2 * T * K + 2 * out * T * N + 2 * used * r * (K + N) + 8 * T
        f = 2 * T * r * (K + N)
        if case["backward"]:
            b += 2 * T * N + 2 * out * T * K + 4 * L * r * (K + N)
            f += 4 * T * r * (K + N)
        return {"bytes": b, "flops": f}
    sizes = [int(n) for n in case["sizes"].split()]
    width = [2 if d != "float32" else 4 for d in case["dtypes"].split()]
    total = sum(n * width[(i * len(sizes) + j) % len(width)] for i in range(case["groups"]) for j, n in enumerate(sizes))
    count = case["groups"] * sum(sizes)
    scaled = case["max_norm"] < 1e6  # the other thresholds lie above any norm that is met here
    return {"bytes": total * (2 if scaled or not case["inplace"] else 1), "flops": count * (3 if scaled else 2)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"balance": _exact_balance, "adapter": _exact_adapter, "clip": _exact_clip}[case["op"]](s)


def _exact_balance(s):
    E, k, S = s["E"], s["k"], s["S"]
    off = s["seq_offsets"].tolist()
    keep = torch.ones(s["T"], dtype=torch.bool, device="cuda") if s["token_mask"] is None else s["token_mask"].bool()
    logits = s["logits"].double()
    rows = [torch.nonzero(keep[off[i]:off[i + 1]])[:, 0] + off[i] for i in range(S)]
    filled = sum(1 for q in rows if len(q))
    n = sum(len(q) for q in rows)
    counts = torch.zeros((S, E), dtype=torch.int64, device="cuda")
    d = torch.zeros_like(logits)
    balance = torch.zeros((), dtype=torch.float64, device="cuda")
    z = torch.zeros_like(balance)
    for i, q in enumerate(rows):
        if not len(q):
            continue
        l = logits[q]
        counts[i] = torch.bincount(s["topk_idx"][q].reshape(-1).long(), minlength=E)
        f = counts[i].double() * E / (k * len(q))
        raw = torch.sigmoid(l) if s["score"] == "sigmoid" else torch.softmax(l, 1)
        p = raw / raw.sum(1, keepdim=True)
        lse = torch.logsumexp(l, 1)
        balance += s["balance_coeff"] / filled * (f * p.mean(0)).sum()
        z += s["z_coeff"] / n * (lse ** 2).sum()
        dp = s["dlosses"][0].double() * s["balance_coeff"] / filled * f / len(q)
        # d p_e / d l_j = slope_j p_j ([e = j] - p_e)
        slope = (1 - raw) if s["score"] == "sigmoid" else torch.ones_like(raw)
        d[q] = p * slope * (dp - (p * dp).sum(1, keepdim=True)) + (
            2 * s["dlosses"][1].double() * s["z_coeff"] / n * lse)[:, None] * torch.softmax(l, 1)
    return {"losses": torch.stack([balance, z]), "counts": counts.to(INT), "dlogits": d}


def _exact_adapter(s):
    idx = s["adapter_idx"]
    y = s["base"].double()
    if s["backward"]:
        dx = s["dx_base"].double()
        dA = torch.zeros(s["A"].shape, dtype=torch.float64, device="cuda")
        dB = torch.zeros(s["B"].shape, dtype=torch.float64, device="cuda")
    for a in range(s["L"]):
        q = torch.nonzero(idx == a)[:, 0]
        if not len(q):
            continue
        A, B, c = s["A"][a].double(), s["B"][a].double(), s["scale"][a].double()
        x = s["x"][q].double()
        u = x @ A
        y[q] += c * (u @ B)
        if s["backward"]:
            dy = s["dy"][q].double() * c
            du = dy @ B.t()
            dx[q] += du @ A.t()
            dA[a] = x.t() @ du
            dB[a] = u.t() @ dy
    return {"y": y, "dx": dx, "dA": dA, "dB": dB} if s["backward"] else {"y": y}


def _exact_clip(s):
    norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(t.double()) for t in s["grads"]]))
    coef = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    return {"norm": norm.view(1), "grads": [t.double() * coef for t in s["flat"]]}
