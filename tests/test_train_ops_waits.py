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
