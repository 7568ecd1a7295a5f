"""What the overlapping launches rely on, read from the sources or asked of the
compiler. CPU only."""
import concurrent.futures as cf
import os
import re
import subprocess

from route_permute_grouped_gb300 import build as B

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


LAUNCHES = """
#include "host_util.h"
namespace moe {
__global__ void k(const float* p, size_t n, uint64_t lim) {}
cudaError_t go(float* p, const int* q, int i, size_t n, uint64_t lim) { return launch_chained(k, 1, 32, 0, nullptr, %s); }
}
"""


def test_launches_take_arguments_of_the_parameters_types_only(tmp_path):
    # a launch hands the kernel the addresses of its arguments: one too few or of another width would be read past its end
    forms = {"p, n, lim": True, "p, n": False, "p, i, lim": False, "p, n, i": False, "q, n, lim": False, "p, n, lim, i": False}

    def compiles(item):
        i, args = item
        src = tmp_path / f"t{i}.cu"
        src.write_text(LAUNCHES % args)
        cmd = [B._nvcc(), *B.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-O0", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
               "-c", str(src), "-o", str(tmp_path / f"t{i}.o")]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return args, r.returncode == 0, r.stderr

    with cf.ThreadPoolExecutor(len(forms)) as ex:
        for args, ok, err in ex.map(compiles, enumerate(forms)):
            assert ok == forms[args], (args, err)
            assert ok or "argument" in err, (args, err)
