"""Dropout against a host generator of the same draws (the published Philox4x32-10, with its known answers).

Tolerance: the product and the residual's sum round in fp32 (2^-24 each) and once to the output's type.
"""
import numpy as np
import pytest

fs = pytest.importorskip("fully_sharded_gb300")
torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32
ROUND = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
gpu = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda(request):
    if request.node.get_closest_marker("gpu") and not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def philox(counter, key):
    """Philox4x32-10 of one 128-bit counter (four words) and key (two), in Python integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def test_the_generators_published_answers():
    """The known answers of the generator's authors, for zeros and for ones."""
    assert philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert philox([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def draws(first, count, seed, offset):
    """The 16-bit draws of elements first .. first + count - 1."""
    out = []
    for g in range(first // 8, (first + count + 7) // 8):
        words = philox([g & 0xFFFFFFFF, g >> 32, offset & 0xFFFFFFFF, offset >> 32], [seed & 0xFFFFFFFF, seed >> 32])
        out += [h for w in words for h in (w & 0xFFFF, w >> 16)]
    return np.array(out[first % 8:first % 8 + count])


def want(x, residual, p, seed, offset):
    rows, cols = x.shape
    t = int(np.floor(65536 * p + 0.5))
    keep = torch.from_numpy((draws(0, rows * cols, seed, offset) >= t).reshape(rows, cols)).cuda()
    v = torch.where(keep, x.double() * 65536 / (65536 - t), 0.0)
    return (v if residual is None else v + residual.double()), keep


def check(out, x, residual, p, seed, offset):
    v, keep = want(x, residual, p, seed, offset)
    size = torch.where(keep, x.double().abs() * 65536 / (65536 - int(np.floor(65536 * p + 0.5))), 0.0)
    if residual is not None:
        size = size + residual.double().abs()
    assert bool(((out.double() - v).abs() <= 4 * 2.0 ** -24 * size + ROUND[out.dtype] * v.abs()).all())
    if residual is None:
        assert bool((out[~keep] == 0).all())


def matrix(gen, rows, cols, dtype, stride=None, offset=0):
    whole = torch.full((offset + max(1, rows) * (stride or cols) + 20,), 7.0, dtype=dtype, device="cuda")
    view = torch.as_strided(whole, (rows, cols), (stride or cols, 1), offset)
    view.copy_(torch.randn(rows, cols, generator=gen, device="cuda"))
    return view


@gpu
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (1, 8), (3, 5), (2, 1000), (33, 769), (50, 64), (5, 4096)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (0, 1), (3, 2), (8, 8)])
def test_elements(rows, cols, dtype, pad, offset):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    x, r = (matrix(gen, rows, cols, dtype, cols + pad, offset) for _ in range(2))
    for p, seed, at in ((0.0, 1, 2), (0.1, 3, 0), (0.5, 2 ** 64 - 1, 2 ** 64 - 1), (0.999, 2 ** 40 + 5, 2 ** 33 + 1)):
        for residual in (None, r):
            out = matrix(gen, rows, cols, dtype, cols + pad, offset)
            whole = torch.as_strided(out, (out.untyped_storage().nbytes() // out.element_size(),), (1,), 0)
            fs.fsdp_dropout(x, out, p, seed, at, residual=residual)
            check(out, x, residual, p, seed, at)
            out.fill_(7.0)
            assert bool((whole == 7.0).all())


@gpu
def test_in_place_and_gradient():
    """The gradient is the same call: every element is kept or dropped as in the forward, times the same factor."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, r, dy = (matrix(gen, 40, 96, F32) for _ in range(3))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    fs.fsdp_dropout(x, y, 0.3, 5, 6, residual=r)
    fs.fsdp_dropout(dy, dx, 0.3, 5, 6)
    check(dx, dy, None, 0.3, 5, 6)
    moved = torch.empty_like(x)
    fs.fsdp_dropout(x + dy, moved, 0.3, 5, 6, residual=r)  # linear in x: y(x + d) - y(x) = gradient's map of d
    assert bool(((moved - y) - dx).abs().max() <= 2.0 ** -20 * 8)
    for target in ("x", "r"):
        a, b = x.clone(), r.clone()
        out = a if target == "x" else b
        fs.fsdp_dropout(a, out, 0.3, 5, 6, residual=b)
        assert torch.equal(out, y)


@gpu
def test_the_rate_and_the_mean():
    """Of n = 2^22 elements a share p_16 is dropped, within 6 sqrt(p (1 - p) / n)."""
    x = torch.ones(1024, 4096, dtype=F32, device="cuda")
    for p in (0.1, 0.37):
        out = torch.empty_like(x)
        fs.fsdp_dropout(x, out, p, 11, 12)
        share = float((out == 0).double().mean())
        exact = np.floor(65536 * p + 0.5) / 65536
        assert abs(share - exact) <= 6 * (exact * (1 - exact) / x.numel()) ** 0.5
        other = torch.empty_like(x)
        fs.fsdp_dropout(x, other, p, 11, 13)
        both = float(((out == 0) & (other == 0)).double().mean())
        assert abs(both - exact ** 2) <= 6 * (exact ** 2 * (1 - exact ** 2) / x.numel()) ** 0.5


@gpu
def test_dropped_nan_has_no_effect():
    x = torch.full((64, 64), float("nan"), device="cuda")
    r, out = torch.ones_like(x), torch.empty_like(x)
    fs.fsdp_dropout(x, out, 0.5, 1, 1, residual=r)
    keep = want(torch.ones_like(x), None, 0.5, 1, 1)[1]
    assert bool(torch.isnan(out[keep]).all()) and bool((out[~keep] == 1).all())


@gpu
def test_a_place_beyond_32_bits():
    """Elements whose counters need more than 32 bits: 8 * 2^32 elements are beyond a test, a wide stride's are not, so
    the check is of the last rows of a long matrix against the draws of their places."""
    x = torch.ones(70000, 1024, dtype=BF16, device="cuda")
    out = torch.empty_like(x)
    fs.fsdp_dropout(x, out, 0.25, 2, 3)
    first = 69999 * 1024
    keep = torch.from_numpy(draws(first, 1024, 2, 3) >= 16384).cuda()
    assert torch.equal(out[69999] != 0, keep)


@gpu
def test_counter_in_a_graph():
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = matrix(gen, 30, 64, BF16)
    counter, out = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fs.fsdp_dropout(x, out, 0.5, 9, 100, counter=counter)
        counter.add_(1)
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        check(out, x, None, 0.5, 9, 100 + step)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fs.fsdp_dropout(x, out, 0.5, 9, 101, stream=side)
    side.synchronize()
    check(out, x, None, 0.5, 9, 101)


@gpu
def test_no_rows():
    x = torch.empty(0, 8, device="cuda")
    fs.fsdp_dropout(x, x, 0.5, 1)
