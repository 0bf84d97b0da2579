"""8-bit outputs of rows with an infinity or a NaN: what the formulas give, in each of the kernel's forms."""
import pytest

pytestmark = pytest.mark.gpu

fs = pytest.importorskip("fully_sharded_gb300")
torch = pytest.importorskip("torch")

from test_gpu_rmsnorm import BF16, E4M3, F32, check_8bit, rand, want_forward  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


# whole vectors, rows off alignment, rows that a warp shares, rows beyond the registers
@pytest.mark.parametrize("rows,cols", [(7, 1024), (600, 4096), (7, 1001), (700, 1001), (7, 100), (600, 40), (600, 129), (7, 20001)])
@pytest.mark.parametrize("group", [0, 32, 256])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_special_values_reach_their_scales(rows, cols, group, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols + group)
    x = rand(gen, rows, cols, dtype=dtype)
    x[1, cols // 2] = float("nan")
    x[3, cols // 3] = float("inf")
    x[rows - 1, cols - 1] = -float("inf")
    gain = rand(gen, cols, dtype=F32) + 2
    for special_gain in (None, float("nan"), float("inf")):
        if special_gain is not None:
            gain[cols - 1] = special_gain
        y = torch.empty(rows, cols, dtype=E4M3, device="cuda")
        scales = torch.empty(rows, -(-cols // group) if group else 1, device="cuda")
        fs.fsdp_rmsnorm(x, gain, y, scales=scales, group=group)
        want = want_forward(x, None, gain, 1e-6)[2]
        width = group or cols
        padded = torch.nn.functional.pad(want, (0, -cols % width)).view(rows, -1, width)
        s = (padded.abs().amax(2) / 448).clamp(min=2.0 ** -126)  # amax and clamp pass a NaN on
        assert torch.equal(scales.isnan(), s.isnan()) and torch.equal(scales.isinf(), s.isinf())
        q = (padded * (1 / s)[:, :, None]).view(rows, -1)[:, :cols]
        assert torch.equal(y.float().isnan(), q.isnan())
        # groups without special values keep theirs, also in the rows that have some
        fine = s.isfinite()
        assert bool(((scales.double() - s).abs()[fine] <= ((cols / 32 + 16) * 2.0 ** -24 * s)[fine]).all())
        if special_gain is None:
            rest = [r for r in range(rows) if r not in (1, 3, rows - 1)]
            check_8bit(y[rest], scales[rest], want[rest], group)
