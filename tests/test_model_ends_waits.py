"""The order of waits in the cross entropy's products, held in the source (host): what it forbids could only be
seen on a GPU as a hang."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fully_sharded_gb300", "csrc")


def text(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def body(source, name):
    at = source.index("{", source.index(" %s(const __grid_constant__" % name))
    depth, end = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(source[end], 0)
        if depth == 0:
            return source[at:end]
        end += 1


def places(where, what):
    return [m.start() for m in re.finditer(re.escape(what), where)]


def test_products_release_the_next_launch_with_their_tensor_memory_in_hand():
    kernel = body(text("cross_entropy.cu"), "ce_product")
    (alloc,), (release,) = places(kernel, "tmem_alloc"), places(kernel, "griddepcontrol.launch_dependents")
    assert any(alloc < b < release for b in places(kernel, "__syncthreads()"))


def test_no_bounded_wait_begins_before_the_previous_grids_end():
    """Only barriers that the block's own progress arms (free at first) are passed before the wait for earlier kernels."""
    kernel = body(text("cross_entropy.cu"), "ce_product")
    roles = [kernel.index(r) for r in ("if (warp == 0) {", "else if (warp == 1 && rank == 0)", "epilogue" if "epilogue" in kernel else "setmaxnreg.inc")]
    for begin, end in zip(roles, roles[1:] + [len(kernel)]):
        role = kernel[begin:end]
        awaited = places(role, "await_inputs()")
        assert len(awaited) == 1
        depends = [p for bar in ("full_bar", "done_bar") for w in ("bar_wait(", "bar_wait_warp(") for p in places(role, w + "smem_addr(&" + bar)]
        assert all(awaited[0] < p for p in depends)


def test_every_kernel_waits_for_the_previous_grid():
    for name in ("cross_entropy.cu", "embedding.cu", "dropout.cu"):
        source = text(name)
        kernels = re.findall(r"__global__[^{;]*?\s(\w+)\(const __grid_constant__", source)
        assert kernels
        for k in kernels:
            assert re.search(r"griddepcontrol\.wait|begin_after_previous\(\)", body(source, k)), k


def test_registers_after_the_split_are_those_of_the_launch():
    source = text("cross_entropy.cu")
    lean, epilogue = map(int, re.search(r"kLeanRegisters = (\d+), kEpilogueRegisters = (\d+)", source).groups())
    assert lean % 8 == epilogue % 8 == 0 and 128 * lean + 256 * epilogue <= 384 * 168


def test_no_collective_of_a_warp_depends_on_a_threads_own_index():
    """A reduction or ballot over all lanes inside `if (has_digit)` (or the like) would wait for lanes that never come."""
    source = text("embedding.cu")
    for match in re.finditer(r"if \((has_digit|digit_of < bins|static_cast<int>\(threadIdx\.x\) < bins)\)\s*({)?", source):
        begin = match.end()
        if match.group(2):
            depth, end = 1, begin
            while depth:
                depth += {"{": 1, "}": -1}.get(source[end], 0)
                end += 1
        else:
            end = source.index(";", begin)
        assert "_sync(" not in source[begin:end]
