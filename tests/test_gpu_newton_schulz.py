"""Newton-Schulz orthogonalisation against the iteration in 64 bits.

Tolerances: with operands of 11 bits (terms = 1, short sides from 256 on) the
result is off by at most 0.3 % of its norm, with three products (terms = 3) by
1e-4, beyond the rounding to bf16, which is at most half a step of each value. One
element may be off by eight times its even share: 0.024 and 0.0008 of its size or
of the root mean square, whichever is more.
"""
import pytest

pytestmark = pytest.mark.gpu

fs = pytest.importorskip("fully_sharded_gb300")
torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def reference(g, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7):
    x = g.double()
    if x.shape[0] > x.shape[1]:
        return reference(g.t(), steps, coefficients, eps).t()
    per_step = [coefficients] * steps if not hasattr(coefficients[0], "__len__") else coefficients
    x = x / (x.norm() + eps)
    for a, b, c in per_step:
        gram = x @ x.t()
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x


def run(sources, outs=None, hyper=None, stream=None, spare=0):
    outs = outs or [torch.empty(s.shape, dtype=BF16, device="cuda") for s in sources]
    batch = fs.NewtonSchulzBatch(sources, outs)
    workspace = torch.empty(fs.fsdp_newton_schulz_workspace(batch, hyper) + spare, dtype=torch.uint8, device="cuda")
    fs.fsdp_newton_schulz(batch, workspace[spare:], hyper, stream=stream)
    torch.cuda.synchronize()
    return outs


def check(out, want, terms):
    rel = 0.003 if terms == 1 else 1e-4
    half_step = torch.exp2(torch.frexp(out.double())[1] - 9.0)
    err = ((out.double() - want).abs() - half_step).clamp(min=0)
    assert bool(err.isfinite().all())
    norm = float(want.norm())
    assert float(err.norm()) <= rel * norm
    rms = norm / max(1, want.numel()) ** 0.5
    assert float((err / want.abs().clamp(min=rms)).max()) <= 8 * rel


def terms_of(shape, terms=0):
    return terms or (3 if min(shape) < 256 else 1)


def gauss(seed, rows, cols, dtype=F32, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(rows, cols, generator=gen, device="cuda")).to(dtype)


SHAPES = [(1, 1), (1, 5), (7, 1), (3, 3), (16, 32), (64, 32), (33, 65), (127, 129), (128, 128), (130, 70), (255, 256),
          (256, 255), (256, 256), (300, 1100), (1100, 300), (257, 513), (512, 512), (768, 2304), (1000, 999), (1537, 769),
          (31, 5000), (5000, 31), (2048, 1280)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_one_matrix(rows, cols, dtype):
    g = gauss(rows * 10007 + cols, rows, cols, dtype)
    check(run([g])[0], reference(g), terms_of((rows, cols)))


LONG = [(1, 5440), (1, 5441), (140, 6000), (6000, 140), (255, 20000), (33, 100003), (300, 16385), (16400, 300), (1100, 17000),
        (1 << 20, 8), (7, 262147)]


@pytest.mark.parametrize("rows,cols", LONG)
def test_long_inner_dimension(rows, cols):
    """Products cut into segments: the same precision whatever the length."""
    g = gauss(rows + cols, rows, cols)
    check(run([g])[0], reference(g), terms_of((rows, cols)))


def test_long_inner_dimension_of_one_sign():
    g = 1 + 0.1 * gauss(8, 1, 1 << 22)
    check(run([g])[0], reference(g), 3)


def test_long_and_short_together():
    sources = [gauss(i, r, c) for i, (r, c) in enumerate(LONG[:9] + [(300, 400), (140, 600), (16, 20)])]
    for hyper in (None, fs.NewtonSchulz(terms=3)):
        outs = run(sources, hyper=hyper)
        for g, out in zip(sources, outs):
            check(out, reference(g), 3 if hyper else terms_of(g.shape))
            assert torch.equal(out, run([g], hyper=hyper)[0])


@pytest.mark.parametrize("rows,cols", [(40, 56), (200, 600), (512, 700), (900, 300)])
@pytest.mark.parametrize("terms", [1, 3])
def test_terms(rows, cols, terms):
    g = gauss(3, rows, cols)
    out = run([g], hyper=fs.NewtonSchulz(terms=terms))[0]
    check(out, reference(g), 3 if terms == 3 else 1)


def test_matrices_of_many_shapes_together():
    sources = [gauss(i, r, c, BF16 if i % 2 else F32, 10.0 ** (i % 5 - 2)) for i, (r, c) in enumerate(SHAPES[:21] + [(0, 5), (5, 0)])]
    outs = run(sources)
    for g, out in zip(sources, outs):
        if g.numel():
            check(out, reference(g), terms_of(g.shape))
            assert torch.equal(out, run([g])[0])  # the company changes nothing


def test_more_matrices_than_one_launch_takes():
    sources = [gauss(100 + i, 24 + i % 7, 40) for i in range(150)] + [gauss(300 + i, 260 + i, 270) for i in range(40)]
    for g, out in zip(sources, run(sources)):
        check(out, reference(g), terms_of(g.shape))


@pytest.mark.parametrize("rows,cols", [(300, 400), (400, 300), (20, 30)])
def test_special_spectra(rows, cols):
    """Rank one, a few strong directions over noise, a decaying spectrum, and equal singular values."""
    k = min(rows, cols)
    u, v = gauss(1, rows, k), gauss(2, k, cols)
    decay = torch.arange(1, k + 1, device="cuda", dtype=F32) ** -1.0
    q, _ = torch.linalg.qr(gauss(4, max(rows, cols), k).double())
    q = (q if rows >= cols else q.t()).float().contiguous()
    for g in (u[:, :1] @ v[:1], u[:, :3] @ v[:3] + 0.01 * gauss(3, rows, cols), (u * decay) @ v, q):
        check(run([g])[0], reference(g), terms_of((rows, cols)))


@pytest.mark.parametrize("scale", [1e-9, 1e-4, 1e6, 1e15])
def test_scales(scale):
    for shape in ((50, 80), (300, 280)):
        g = gauss(5, *shape, scale=scale)
        check(run([g])[0], reference(g), terms_of(shape))


def test_zero_and_nan_matrices_stay_apart():
    zero, good, bad = torch.zeros(300, 310, device="cuda"), gauss(6, 300, 310), gauss(7, 300, 310)
    bad[4, 5] = float("nan")
    small = torch.zeros(9, 4, device="cuda")
    outs = run([zero, good, bad, small])
    assert bool((outs[0] == 0).all()) and bool((outs[3] == 0).all())
    check(outs[1], reference(good), 1)
    assert bool(outs[2].isnan().any())


@pytest.mark.parametrize("rows,cols", [(300, 513), (60, 41)])
def test_strides_offsets_and_canaries(rows, cols):
    buffer = torch.full((rows + 2, cols + 9), 7.0, dtype=BF16, device="cuda")
    source = buffer[1:1 + rows, 3:3 + cols]
    source.copy_(gauss(8, rows, cols))
    outs = torch.full((rows + 2, cols + 5), 9.0, dtype=BF16, device="cuda")
    out = outs[1:1 + rows, 5:]
    out.fill_(0)
    before = buffer.clone()
    run([source], [out], spare=1)
    check(out, reference(source), terms_of((rows, cols)))
    assert torch.equal(buffer, before)
    assert bool((outs[:, :5] == 9).all()) and bool((outs[0] == 9).all()) and bool((outs[-1] == 9).all())
    run([source], [source])  # in place
    assert torch.equal(source, out)


@pytest.mark.parametrize("shape", [(48, 100), (320, 260)])
def test_coefficients_and_steps(shape):
    g = gauss(9, *shape)
    cubic = (1.5, -0.5, 0.0)
    mixed = [(3.4445, -4.7750, 2.0315), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)]
    for steps, co in ((1, None), (8, None), (12, cubic), (3, mixed)):
        out = run([g], hyper=fs.NewtonSchulz(steps=steps, coefficients=co))[0]
        want = reference(g, steps, co or (3.4445, -4.7750, 2.0315))
        check(out, want, terms_of(shape))


def test_result_is_nearly_orthogonal():
    out = run([gauss(10, 300, 500)], hyper=fs.NewtonSchulz(steps=12, coefficients=(1.875, -1.25, 0.375)))[0].double()
    values = torch.linalg.svdvals(out)
    assert float(values.max()) < 1.01 and float(values.min()) > 0.9


def test_on_another_stream_repeatable_and_in_a_graph():
    sources = [gauss(11, 300, 700), gauss(12, 70, 90)]
    first = run(sources)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(first, run(sources, stream=side)))
    outs = [torch.empty_like(t) for t in first]
    batch = fs.NewtonSchulzBatch(sources, outs)
    workspace = torch.empty(fs.fsdp_newton_schulz_workspace(batch), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fs.fsdp_newton_schulz(batch, workspace)
    workspace.fill_(0xFF)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
