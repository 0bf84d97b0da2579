"""The order of waits in the operators' kernels, held in the source (host): what it forbids could
only be seen on a GPU as a hang."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fully_sharded_gb300", "csrc")


def kernel(name):
    """The text of a kernel's body, without comments."""
    source = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "newton_schulz.cu")).read())
    at = source.index("{", source.index(" %s(const __grid_constant__" % name))
    depth, end = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(source[end], 0)
        if depth == 0:
            return source[at:end]
        end += 1


def places(body, what):
    return [m.start() for m in re.finditer(re.escape(what), body)]


def test_one_block_kernel_holds_tensor_memory_only_between_the_waits():
    """It queues for its columns after the previous grid has ended, and the next grid starts when all
    blocks have theirs: a block barrier lies between the allocation and the release."""
    body = kernel("ns_small")
    (wait,), (alloc,), (release,) = (places(body, w) for w in ("griddepcontrol.wait", "tmem_alloc", "griddepcontrol.launch_dependents"))
    assert wait < alloc < release
    assert any(alloc < b < release for b in places(body, "__syncthreads()"))


def test_products_release_the_next_launch_with_their_tensor_memory_in_hand():
    body = kernel("ns_product")
    (alloc,), (release,) = places(body, "tmem_alloc"), places(body, "griddepcontrol.launch_dependents")
    assert any(alloc < b < release for b in places(body, "__syncthreads()"))


def test_no_bounded_wait_of_the_products_begins_before_the_previous_grids_end():
    """Each role waits for the previous grid before its first wait that depends on it: the 2 s limit
    would otherwise run while earlier kernels of the stream do, and the launch be given up in a correct run."""
    body = kernel("ns_product")
    starts = [body.index(role) for role in ("if (warp == 0)", "else if (warp == 1 && rank == 0)", "else if (warp == 2", "else if (warp >= 4)")]
    for begin, end in zip(starts, starts[1:] + [len(body)]):
        role = body[begin:end]
        awaited = places(role, "await_inputs()")
        assert len(awaited) == 1
        # barriers that only the block's own progress arms are free at first and may be passed before
        depends = [p for bar in ("full_bar", "in_bar", "done_bar") for w in ("bar_wait(", "bar_wait_warp(")
                   for p in places(role, w + "smem_addr(&" + bar)]
        assert all(awaited[0] < p for p in depends)
