"""What the few-token kernel does with copies and products under way when a wait runs out,
read from its source: a copy that lands after its block has left would write into the
shared memory of the next. CPU only."""
import re

from tests.test_launch_chain_host import _body, _source


def test_a_block_that_gives_up_waits_for_what_it_began():
    src = _source("few.cu")
    kernel = _body(src, src.index("few_kernel(const __grid_constant__"))
    # no role lets time pass in place of a wait
    assert "nanosleep" not in kernel and "globaltimer" not in kernel
    # every role has ended, then the copies' and the products' barriers, then the tensor memory
    sync = kernel.rindex("__syncthreads()", 0, kernel.index("few_drain<MX>("))
    drain, free = kernel.index("few_drain<MX>("), kernel.index("tmem_dealloc(")
    assert kernel.index("few_route<MX>(") < sync < drain < free
    assert re.search(r"if \(\*abort_flag\)\s*few_drain<MX>\(", kernel)


def test_the_copies_own_barriers_are_waited_for():
    src = _source("few.cu")
    drain = _body(src, src.index("void few_drain("))
    # the stages that any of the copying threads began are announced by all of them, before the wait
    most, arrive, wait = drain.index("atomicMax(&c->stages"), drain.index("mbar_arrive(c->full"), drain.index("mbar_wait_bounded(c->full")
    assert drain.index("__syncthreads()", most) < arrive < wait
    assert "umma_commit(&c->drain)" in drain and "mbar_wait_bounded(&c->drain" in drain
    # with limits of their own: the block's flag is set already
    assert "&c->abort" not in drain and "abort_flag" not in drain
