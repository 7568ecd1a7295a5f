"""Inputs written right before the calls and overwritten right after, eager and
captured, and captures behind kernels, memsets, copies and joins of streams: the
router losses' and the norm's and clipping's kernels start before the one ahead
has ended and must see all of it, and nothing enqueued behind."""
import pytest
import torch

from route_permute_grouped_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from route_permute_grouped_gb300 import build
    build.build()
    ops.lib()


class Balance:
    """Forward and backward of the router losses on buffers that are rewritten."""

    def __init__(self, T, E, S, seed):
        self.cfg = ops.make_balance_config(T, E, 2, n_seqs=S, score="sigmoid" if E % 3 else "softmax", z_coeff=1e-3)
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.rand(s, generator=g, device="cuda")
        self.inputs = {"logits": rand(T, E) * 4 - 2, "idx": (rand(T, 2) * E).to(torch.int32).clamp_(max=E - 1),
                       "off": torch.sort((rand(S + 1) * (T + 1)).to(torch.int32).clamp_(max=T))[0].contiguous(),
                       "mask": (rand(T) > 0.2).to(torch.uint8), "dl": rand(2) + 0.5}
        self.ws = ops.balance_workspace(self.cfg)

    def step(self, c):
        losses, counts, stats = ops.balance_loss_fwd(self.cfg, c["logits"], c["idx"], c["off"], c["mask"], ws=self.ws)
        return [losses, counts, ops.balance_loss_bwd(self.cfg, c["logits"], stats, c["dl"], c["off"], c["mask"])]


class Clip:
    """Norm and clipping; the lists hold the rewritten buffers' addresses."""

    def __init__(self, sizes, apart, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        types = [torch.float32, torch.bfloat16, torch.float16]
        self.inputs = {str(i): torch.randn(n, generator=g, device="cuda").to(types[i % 3]) for i, n in enumerate(sizes)}
        self.apart, self.ws = apart, ops.grad_norm_workspace()
        self.lists = {}

    def step(self, c):
        key = c["0"].data_ptr()
        if key not in self.lists:
            ts = list(c.values())
            out = [torch.empty_like(t) for t in ts] if self.apart else None
            self.lists[key] = (ops.tensor_list(ts, out=out), out or ts)
        tl, out = self.lists[key]
        norm = ops.clip_grad_norm(tl, 0.5, ws=self.ws)
        return [norm] + [torch.add(t, 0) for t in out]      # read by the next kernel in the stream


KINDS = {"balance_small": lambda seed: Balance(60, 8, 1, seed), "balance_ragged": lambda seed: Balance(9001, 64, 37, seed),
         "balance_256": lambda seed: Balance(40000, 256, 3, seed), "clip_small": lambda seed: Clip([5, 1001, 33], False, seed),
         "clip_many": lambda seed: Clip([7 + 13 * i for i in range(900)], True, seed),
         "clip_large": lambda seed: Clip([9_000_001, 3, 5_000_000], False, seed),
         "clip_large_apart": lambda seed: Clip([9_000_001, 3, 5_000_000], True, seed)}


def _sets(kind):
    made = [KINDS[kind](seed) for seed in (1, 2, 3)]
    op = made[0]
    sets = [m.inputs for m in made]
    want = []
    for c in sets:
        want.append([t.clone() for t in op.step({k: v.clone() for k, v in c.items()})])
        torch.cuda.synchronize()
    live = {k: torch.empty_like(v) for k, v in sets[0].items()}
    return op, sets, want, live


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("kind", list(KINDS))
def test_inputs_written_right_before_and_overwritten_right_after(kind, captured):
    op, sets, want, live = _sets(kind)

    def run():
        got = []
        for c in sets * 3:
            for k, v in live.items():
                torch.add(c[k], 0, out=v)
            got.append(op.step(live))
            for v in live.values():
                v.fill_(1)
        return got

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run()
    if captured:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = run()
        g.replay()
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        for a, b in zip(out, want[i % 3]):
            assert torch.equal(a, b), (kind, i)
    assert ops.device_status(op.ws) == 0


@pytest.mark.parametrize("before", ["kernel", "copy", "memset", "join"])
@pytest.mark.parametrize("kind", list(KINDS))
def test_captured_behind_other_work(kind, before):
    op, sets, want, live = _sets(kind)
    src, want = sets[0], want[0]
    big = torch.ones(1 << 26, device="cuda")            # long enough to be still running
    s, side = torch.cuda.Stream(), torch.cuda.Stream()
    first = next(iter(live))
    if before == "memset":                              # the last thing ahead of the call is a memset of an input
        zeroed = {k: v.clone() for k, v in src.items()}
        zeroed[first].zero_()
        want = [t.clone() for t in op.step({k: v.clone() for k, v in zeroed.items()})]

    def work():
        big.mul_(1.0)
        if before == "copy":
            for k, v in live.items():
                v.copy_(src[k])
        elif before == "join":
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                big.mul_(1.0)
                for k, v in live.items():
                    torch.add(src[k], 0, out=v)
            torch.cuda.current_stream().wait_stream(side)
        else:
            for k, v in live.items():
                torch.add(src[k], 0, out=v)
            if before == "memset":
                live[first].zero_()
        return op.step(live)

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = work()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = work()
    for _ in range(3):
        for v in live.values():
            v.fill_(1)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
