"""RMS norm with the residual's addition, forward and backward, against the formulas in 64 bits.

Tolerances, from the operations' roundings (u = 2^-24 for fp32, 2^-8 for bf16):
  - a sum of n terms in fp32 is off by at most (n / 32 + 16) u of the sum of the
    terms' absolute values (every variant adds at most n / 32 terms in sequence,
    then a tree); products and the reciprocal square root add a few u;
  - each output is rounded once to its type;
  - an 8-bit output is off by half a step of e4m3, 2^-4 of its value or 2^-10
    scales where it is subnormal, and by one more rounding boundary's width, 1e-5.
"""
import pytest

import gpu_util as gu

pytestmark = pytest.mark.gpu

fs = pytest.importorskip("fully_sharded_gb300")
torch = pytest.importorskip("torch")

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
UNIT = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def rand(gen, *shape, dtype=F32, scale=1.0):
    return (scale * torch.randn(*shape, generator=gen, device="cuda")).to(dtype)


def guarded(rows, cols, dtype, stride=None, offset=0, guard=64):
    """A matrix inside a buffer of canary bytes; returns (whole, view)."""
    stride = stride or cols
    size = torch.empty(0, dtype=dtype).element_size()
    n = offset + max(1, rows) * stride + 2 * guard
    whole = torch.full((n * size,), 0x5A, dtype=torch.uint8, device="cuda").view(dtype)
    return whole, torch.as_strided(whole, (rows, cols), (stride, 1), guard + offset)


def untouched(whole, view):
    """Every byte of `whole` outside `view` still holds the canary."""
    bytes_ = whole.view(torch.uint8).clone()
    size = whole.element_size()
    if view.numel():
        torch.as_strided(bytes_, (view.shape[0], view.shape[1] * size), (view.stride(0) * size, 1),
                         view.storage_offset() * size).fill_(0x5A)
    return bool((bytes_ == 0x5A).all())


def want_forward(x, residual, gain, eps):
    h = x.double() + (residual.double() if residual is not None else 0)
    rstd = 1 / torch.sqrt(h.square().mean(1) + eps)
    return h, rstd, h * rstd[:, None] * gain.double()


def check_y(y, want, cols):
    rel = (cols / 32 + 16) * 2.0 ** -24 + (UNIT[y.dtype] if y.dtype is BF16 else 0)
    assert bool(((y.double() - want).abs() <= rel * want.abs() + 1e-30).all())


def check_8bit(y, scales, want, group):
    rows, cols = want.shape
    group = group or cols
    padded = torch.nn.functional.pad(want, (0, -cols % group)).view(rows, -1, group)
    s = (padded.abs().amax(2) / 448).clamp(min=2.0 ** -126)
    assert bool(((scales.double() - s).abs() <= ((cols / 32 + 16) * 2.0 ** -24) * s).all())
    each = scales.double().repeat_interleave(group, 1)[:, :cols]
    err = (y.double() * each - want).abs()
    assert bool((err <= (2.0 ** -4 + 1e-5) * want.abs() + (2.0 ** -10 + 1e-5) * each).all())


SHAPES = [(1, 1), (3, 1), (2, 7), (5, 8), (1, 4096), (7, 768), (33, 769), (4, 1000), (3, 4095), (2, 11008), (130, 256),
          (2, 16384), (3, 16385), (2, 50001), (1, 100000), (700, 24)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("with_residual", [False, True], ids=["plain", "residual"])
def test_forward(rows, cols, dtype, with_residual):
    gen = torch.Generator(device="cuda").manual_seed(rows * 100003 + cols)
    x, gain = rand(gen, rows, cols, dtype=dtype), rand(gen, cols, dtype=dtype) + 1
    residual = rand(gen, rows, cols, dtype=dtype, scale=3.0) if with_residual else None
    whole_y, y = guarded(rows, cols, dtype)
    whole_h, h = guarded(rows, cols, dtype)
    rstd = torch.empty(rows, device="cuda")
    fs.fsdp_rmsnorm(x, gain, y, residual=residual, h_out=h if with_residual else None, rstd=rstd, eps=1e-5)
    want_h, want_rstd, want_y = want_forward(x, residual, gain, 1e-5)
    check_y(y, want_y, cols)
    assert bool(((rstd.double() - want_rstd).abs() <= (cols / 32 + 16) * 2.0 ** -24 * want_rstd).all())
    if with_residual:
        assert torch.equal(h, (x.float() + residual.float()).to(dtype))
    assert untouched(whole_y, y) and untouched(whole_h, h if with_residual else h[:0])


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 31), (1, 4096), (9, 769), (3, 11008), (4, 1000), (2, 16385), (65, 4096)])
@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_forward_8bit(rows, cols, group, dtype):
    gen = torch.Generator(device="cuda").manual_seed(cols + group)
    x, residual = rand(gen, rows, cols, dtype=dtype), rand(gen, rows, cols, dtype=dtype)
    x[0, ::3] = 0
    gain = rand(gen, cols, dtype=F32)
    whole, y = guarded(rows, cols, E4M3)
    scales = torch.empty(rows, -(-cols // group) if group else 1, device="cuda")
    h = torch.empty_like(x)
    fs.fsdp_rmsnorm(x, gain, y, residual=residual, h_out=h, scales=scales, group=group)
    check_8bit(y, scales, want_forward(x, residual, gain, 1e-6)[2], group)
    assert torch.equal(h, (x.float() + residual.float()).to(dtype))
    assert untouched(whole, y)


@pytest.mark.parametrize("rows,cols", [(600, 8), (600, 40), (521, 64), (513, 65), (1100, 100), (600, 128), (515, 129), (530, 769), (600, 1024),
                                       (1100, 2000), (700, 4104)])
@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_forward_8bit_of_many_rows(rows, cols, group, dtype):
    """Rows that share a warp or a block keep their own scales: each is of another size than its neighbours."""
    gen = torch.Generator(device="cuda").manual_seed(rows + cols + group)
    x = rand(gen, rows, cols, dtype=dtype)
    x[:, 0] = 0.5
    x[1::3] = 0  # rows of zeros, whose scale is the smallest
    x[2::3, 1:] = 0  # and rows of a single value, whose scale is the largest
    gain = rand(gen, cols, dtype=F32) + 2
    whole, y = guarded(rows, cols, E4M3)
    scales = torch.empty(rows, -(-cols // group) if group else 1, device="cuda")
    fs.fsdp_rmsnorm(x, gain, y, scales=scales, group=group)
    check_8bit(y, scales, want_forward(x, None, gain, 1e-6)[2], group)
    assert untouched(whole, y)


@pytest.mark.parametrize("rows,cols", [(513, 65), (600, 100), (1000, 128), (700, 129)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_forward_and_backward_of_many_short_rows(rows, cols, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x, residual, gain = rand(gen, rows, cols, dtype=dtype), rand(gen, rows, cols, dtype=dtype), rand(gen, cols, dtype=F32)
    whole, y = guarded(rows, cols, dtype)
    h = torch.empty_like(x)
    fs.fsdp_rmsnorm(x, gain, y, residual=residual, h_out=h)
    check_y(y, want_forward(x, residual, gain, 1e-6)[2], cols)
    assert torch.equal(h, (x.float() + residual.float()).to(dtype)) and untouched(whole, y)
    check_backward(rand(gen, rows, cols, dtype=dtype), h, gain, residual)


@pytest.mark.parametrize("cols,stride,offset", [(768, 1024, 0), (768, 769, 1), (100, 104, 3), (4096, 4104, 4), (1000, 1001, 0)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_forward_strides_and_offsets(cols, stride, offset, dtype):
    gen = torch.Generator(device="cuda").manual_seed(stride)
    rows = 19
    _, x = guarded(rows, cols, dtype, stride, offset)
    _, residual = guarded(rows, cols, dtype, stride + 8, 0)
    x.copy_(rand(gen, rows, cols))
    residual.copy_(rand(gen, rows, cols))
    gain = rand(gen, cols + 1, dtype=BF16)[1:]  # a gain at an odd place of a flat parameter
    whole_h, h = guarded(rows, cols, dtype, stride, offset + 1)
    whole_y, y = guarded(rows, cols, dtype, stride + 1, 0)
    fs.fsdp_rmsnorm(x, gain, y, residual=residual, h_out=h)
    check_y(y, want_forward(x, residual, gain, 1e-6)[2], cols)
    assert torch.equal(h, (x.float() + residual.float()).to(dtype))
    assert untouched(whole_h, h) and untouched(whole_y, y)


@pytest.mark.parametrize("cols", [64, 769, 4096, 20000])
@pytest.mark.parametrize("eight", [False, True])
def test_forward_in_place(cols, eight):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x, residual, gain = rand(gen, 6, cols, dtype=BF16), rand(gen, 6, cols, dtype=BF16), rand(gen, cols, dtype=BF16)
    want_h, _, want_y = want_forward(x, residual, gain, 1e-6)
    rounded = (x.float() + residual.float()).to(BF16)
    if eight:
        y, scales = torch.empty(6, cols, dtype=E4M3, device="cuda"), torch.empty(6, 1, device="cuda")
        fs.fsdp_rmsnorm(x, gain, y, residual=residual, h_out=x, scales=scales)
        check_8bit(y, scales, want_y, 0)
        assert torch.equal(x, rounded)
    else:
        fs.fsdp_rmsnorm(x, gain, x, residual=residual, h_out=residual)
        check_y(x, want_y, cols)
        assert torch.equal(residual, rounded)


def test_forward_of_column_slices():
    gen = torch.Generator(device="cuda").manual_seed(5)
    buffer = rand(gen, 11, 384, dtype=BF16)
    before = buffer.clone()
    fs.fsdp_rmsnorm(buffer[:, :128], torch.ones(128, device="cuda"), buffer[:, 256:])
    check_y(buffer[:, 256:].contiguous(), want_forward(before[:, :128], None, torch.ones(128, device="cuda"), 1e-6)[2], 128)
    assert torch.equal(buffer[:, :256], before[:, :256])


def test_special_rows_stay_in_their_rows():
    gen = torch.Generator(device="cuda").manual_seed(6)
    x, gain = rand(gen, 6, 1000, dtype=BF16), rand(gen, 1000, dtype=BF16)
    x[1] = 0
    x[2, 17] = float("inf")
    x[3, 5] = float("nan")
    y, rstd = torch.empty_like(x), torch.empty(6, device="cuda")
    fs.fsdp_rmsnorm(x, gain, y, rstd=rstd)
    ok = [0, 4, 5]
    check_y(y[ok], want_forward(x[ok], None, gain, 1e-6)[2], 1000)
    assert bool((y[1] == 0).all()) and float(rstd[1]) == pytest.approx(1e3, rel=1e-6)
    assert float(rstd[2]) == 0 and bool(y[2, 17].isnan()) and bool((y[2, :17] == 0).all())
    assert bool(y[3].isnan().all())
    q, scales = torch.empty(6, 1000, dtype=E4M3, device="cuda"), torch.empty(6, 1, device="cuda")
    fs.fsdp_rmsnorm(x, gain, q, scales=scales)
    check_8bit(q[ok], scales[ok], want_forward(x[ok], None, gain, 1e-6)[2], 0)
    assert bool((q[1].float() == 0).all()) and float(scales[1]) == 2.0 ** -126


def test_offsets_past_32_bits():
    """Rows 2^30 elements apart (2^31 bytes): the last row starts past 2^32 bytes."""
    stride, cols = 1 << 30, 513
    buffer = torch.empty(3 * stride, dtype=BF16, device="cuda")
    x, y = torch.as_strided(buffer, (3, cols), (stride, 1)), torch.as_strided(buffer, (3, cols), (stride, 1), 4096)
    gen = torch.Generator(device="cuda").manual_seed(7)
    x.copy_(rand(gen, 3, cols))
    gain = rand(gen, cols, dtype=BF16)
    fs.fsdp_rmsnorm(x, gain, y)
    check_y(y.contiguous(), want_forward(x, None, gain, 1e-6)[2], cols)
    dx = torch.as_strided(buffer, (3, cols), (stride, 1), 8192)
    check_backward(rand(gen, 3, cols, dtype=BF16), x, gain, None, dx=dx)


def want_backward(dy, h, gain, rstd, dh):
    n = h * rstd[:, None]
    u = dy * gain
    dx = rstd[:, None] * (u - n * (u * n).mean(1, keepdim=True))
    return (dx + dh if dh is not None else dx), (dy * n).sum(0)


def check_backward(dy, h, gain, dh, dx=None, dgain=None):
    rows, cols = h.shape
    rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    dx = torch.empty_like(h) if dx is None else dx
    dgain = torch.empty_like(gain) if dgain is None else dgain
    d = dy.double(), h.double(), gain.double(), rstd.double(), dh.double() if dh is not None else None
    want_dx, want_dgain = want_backward(*d)
    workspace = torch.empty(fs.fsdp_rmsnorm_backward_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    fs.fsdp_rmsnorm_backward(dy, h, gain, rstd, dx, dgain, workspace, dh=dh)
    u, n = (d[0] * d[2]).abs(), (d[1] * d[3][:, None]).abs()
    room = (cols / 32 + 16) * 2.0 ** -24 * (d[3][:, None] * (u + n * (u * n).mean(1, keepdim=True))
                                            + (d[4].abs() if dh is not None else 0))
    own = UNIT[BF16] if h.dtype is BF16 else 0
    assert bool(((dx.double() - want_dx).abs() <= room + own * (want_dx.abs() + room) + 1e-30).all())
    room = (rows + 16) * 2.0 ** -24 * (d[0].abs() * n).sum(0)
    own = UNIT[BF16] if gain.dtype is BF16 else 0
    assert bool(((dgain.double() - want_dgain).abs() <= room + own * (want_dgain.abs() + room) + 1e-30).all())


@pytest.mark.parametrize("rows,cols", SHAPES + [(333, 769), (1200, 40), (2000, 512)])
@pytest.mark.parametrize("dtype,gain_dtype", [(BF16, BF16), (F32, F32), (BF16, F32)], ids=["bf16", "f32", "mixed"])
@pytest.mark.parametrize("with_dh", [False, True], ids=["plain", "dh"])
def test_backward(rows, cols, dtype, gain_dtype, with_dh):
    gen = torch.Generator(device="cuda").manual_seed(rows * 7 + cols)
    dh = rand(gen, rows, cols, dtype=dtype) if with_dh else None
    gain = rand(gen, cols, dtype=gain_dtype) + 1
    whole, dx = guarded(rows, cols, dtype)
    check_backward(rand(gen, rows, cols, dtype=dtype), rand(gen, rows, cols, dtype=dtype), gain, dh, dx=dx)
    assert untouched(whole, dx)


@pytest.mark.parametrize("cols,stride,offset", [(768, 1024, 0), (768, 769, 1), (100, 104, 3), (4096, 4104, 4)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_backward_strides_and_offsets(cols, stride, offset, dtype):
    gen = torch.Generator(device="cuda").manual_seed(stride)
    rows = 23
    made = [guarded(rows, cols, dtype, stride + 8 * k, offset * (k % 2)) for k in range(4)]
    dy, h, dh, dx = (view for _, view in made)
    for t in (dy, h, dh):
        t.copy_(rand(gen, rows, cols))
    flat = torch.full((cols + 9,), 3.0, dtype=BF16, device="cuda")  # a rank's gradient row
    check_backward(dy, h, rand(gen, cols + 1, dtype=BF16)[1:], dh, dx=dx, dgain=flat[5:5 + cols])
    assert bool((flat[:5] == 3).all()) and bool((flat[5 + cols:] == 3).all())
    assert untouched(made[3][0], dx)


@pytest.mark.parametrize("which", ["dy", "dh"])
@pytest.mark.parametrize("cols", [100, 4096, 20000])
def test_backward_in_place(which, cols):
    gen = torch.Generator(device="cuda").manual_seed(8)
    dy, h, dh = (rand(gen, 5, cols) for _ in range(3))
    gain = rand(gen, cols)
    check_backward(dy, h, gain, dh, dx={"dy": dy, "dh": dh}[which])


def test_backward_of_no_rows_clears_dgain():
    dgain = torch.full((77,), 5.0, dtype=BF16, device="cuda")
    none = torch.empty(0, 77, dtype=BF16, device="cuda")
    fs.fsdp_rmsnorm(none, torch.ones(77, dtype=BF16, device="cuda"), none.clone())
    fs.fsdp_rmsnorm_backward(none, none, dgain.clone(), torch.empty(0, device="cuda"), none.clone(), dgain,
                             torch.empty(8192, dtype=torch.uint8, device="cuda"))
    assert bool((dgain == 0).all())


def test_gradients_match_differences():
    """dx and dgain against central differences of the 64-bit forward, along random directions.

    With step t the difference's own error is O(t^2) of third derivatives (values of order 1):
    t = 1e-4 leaves 1e-7; the fp32 kernel's is about 1e-6 of the terms' size."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    rows, cols, t = 6, 37, 1e-4
    x, residual, gain, dy, dh = (rand(gen, *s) for s in ((rows, cols), (rows, cols), (cols,), (rows, cols), (rows, cols)))
    y, h, rstd, dx, dgain = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty_like(x), torch.empty_like(gain)
    fs.fsdp_rmsnorm(x, gain, y, residual=residual, h_out=h, rstd=rstd)
    workspace = torch.empty(fs.fsdp_rmsnorm_backward_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    fs.fsdp_rmsnorm_backward(dy, h, gain, rstd, dx, dgain, workspace, dh=dh)

    def loss(x, residual, gain):
        h, _, y = want_forward(x, residual, gain, 1e-6)
        return float((y * dy.double()).sum() + (h * dh.double()).sum())

    for _ in range(4):
        a, b, c = (torch.randn(*s, generator=gen, device="cuda", dtype=torch.float64) for s in ((rows, cols), (rows, cols), (cols,)))
        plus = loss(x.double() + t * a, residual.double() + t * b, gain.double() + t * c)
        minus = loss(x.double() - t * a, residual.double() - t * b, gain.double() - t * c)
        got = float((dx.double() * (a + b)).sum() + (dgain.double() * c).sum())
        assert got == pytest.approx((plus - minus) / (2 * t), abs=2e-4)


def test_on_another_stream_and_repeatable():
    gen = torch.Generator(device="cuda").manual_seed(10)
    x, gain, dy = rand(gen, 500, 1024, dtype=BF16), rand(gen, 1024, dtype=BF16), rand(gen, 500, 1024, dtype=BF16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    results = []
    for stream in (torch.cuda.current_stream(), side, side):
        y, dx, dgain, rstd = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(gain), torch.zeros(500, device="cuda")
        workspace = torch.empty(fs.fsdp_rmsnorm_backward_workspace(500, 1024) + 1, dtype=torch.uint8, device="cuda")[1:]
        torch.cuda.synchronize()
        fs.fsdp_rmsnorm(x, gain, y, rstd=rstd, stream=stream)
        fs.fsdp_rmsnorm_backward(dy, x, gain, rstd, dx, dgain, workspace, stream=stream)
        torch.cuda.synchronize()
        results.append((y, rstd, dx, dgain))
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))


def test_in_a_graph():
    gen = torch.Generator(device="cuda").manual_seed(11)
    x, gain = rand(gen, 64, 768, dtype=BF16), rand(gen, 768, dtype=BF16)
    y, rstd, dx, dgain = torch.empty_like(x), torch.empty(64, device="cuda"), torch.empty_like(x), torch.empty_like(gain)
    workspace = torch.empty(fs.fsdp_rmsnorm_backward_workspace(64, 768), dtype=torch.uint8, device="cuda")

    def both():
        fs.fsdp_rmsnorm(x, gain, y, rstd=rstd)
        fs.fsdp_rmsnorm_backward(y, x, gain, rstd, dx, dgain, workspace)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    x.copy_(rand(gen, 64, 768))
    graph.replay()
    got = [t.clone() for t in (y, rstd, dx, dgain)]
    both()
    assert all(torch.equal(a, b) for a, b in zip(got, (y, rstd, dx, dgain)))
