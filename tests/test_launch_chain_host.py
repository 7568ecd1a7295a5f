"""What the overlapping launches rely on, read from the sources. CPU only."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "route_permute_grouped_gb300", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _body(src, at):
    """The braces' contents that begin behind position at."""
    first = src.index("{", at)
    depth = 0
    for i in range(first, len(src)):
        depth += {"{": 1, "}": -1}.get(src[i], 0)
        if depth == 0:
            return src[first:i + 1]
    raise AssertionError("no end")


def test_tensor_memory_is_allocated_before_the_next_kernel_may_start():
    # a kernel that waits for the one ahead with tensor memory in hand must find that one's blocks with theirs:
    # tcgen05.alloc of a block beside it would wait without a limit
    src = _source("adapter_tc.cuh")
    init = _body(src, src.index("void tc_init("))
    alloc, sync, release = init.index("tmem_alloc("), init.rindex("__syncthreads()"), init.index("chain_release()")
    assert alloc < sync < release
    kernels = [m for m in re.finditer(r"\n\s+(adapter_\w+_tc)\(const", src)]
    assert [m.group(1) for m in kernels] == ["adapter_shrink_tc", "adapter_expand_tc", "adapter_wgrad_tc"]
    for m in kernels:
        body = _body(src, src.index(")", m.end()))
        assert body.count("tc_init<R>(") == 1
        assert "chain_release()" not in body, m.group(1)
        # what is released ahead of it are blocks that leave
        before = body[:body.index("tc_init<R>(")]
        for leave in re.finditer(r"chain_leave\(\)", before):
            assert before[:leave.start()].rstrip().endswith("return"), m.group(1)
