"""Norm rows beyond the registers: the sums' error does not grow with the row.

Tolerance, u = 2^-24: a thread's group of 8 is off by 8 u of itself, its compensated sum by 2 u, the
tree over the block's threads by 13 u, mean and reciprocal square root by 4 u: 32 u holds all of it, and
half of it reaches rstd. Equal values make the roundings systematic, so that a running sum
over the 2^24 columns (65536 elements a thread) would be off by 2000 u and more."""
import pytest

pytestmark = pytest.mark.gpu

fs = pytest.importorskip("fully_sharded_gb300")
torch = pytest.importorskip("torch")

ROOM = 32 * 2.0 ** -24
COLS = 1 << 24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("value", [0.7, 1.1, 0.33])
def test_a_long_row_of_equal_values(value):
    x = torch.full((1, COLS), value, device="cuda")
    gain, y, rstd = torch.full((COLS,), 1.5, device="cuda"), torch.empty_like(x), torch.empty(1, device="cuda")
    fs.fsdp_rmsnorm(x, gain, y, rstd=rstd)
    v = float(x[0, 0])
    want = (v * v + 1e-6) ** -0.5
    assert abs(float(rstd) / want - 1) <= ROOM
    assert float((y.double() / (v * want * 1.5) - 1).abs().max()) <= ROOM

    # dx = rstd (u - n mean(u n)): the two terms nearly cancel, their sizes bound the error
    dy, dx, dgain = torch.full_like(x, 0.9), torch.empty_like(x), torch.empty_like(gain)
    workspace = torch.empty(fs.fsdp_rmsnorm_backward_workspace(1, COLS), dtype=torch.uint8, device="cuda")
    fs.fsdp_rmsnorm_backward(dy, x, gain, rstd, dx, dgain, workspace)
    u, r = float(dy[0, 0]) * 1.5, float(rstd)
    n = v * r
    assert float((dx.double() - r * (u - n * u * n)).abs().max()) <= ROOM * r * (u + n * u * n)


def test_special_values_in_long_rows():
    x = torch.ones(3, 20001, device="cuda")
    x[1, 15000], x[2, 15000] = float("inf"), float("nan")
    y, rstd = torch.empty_like(x), torch.empty(3, device="cuda")
    fs.fsdp_rmsnorm(x, torch.ones(20001, device="cuda"), y, rstd=rstd)
    assert float((y[0] - 1).abs().max()) < 1e-5
    assert float(rstd[1]) == 0 and bool((y[1, :15000] == 0).all()) and bool(y[1, 15000].isnan())
    assert bool(rstd[2].isnan()) and bool(y[2].isnan().all())
