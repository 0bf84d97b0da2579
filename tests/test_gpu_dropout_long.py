"""Dropout of matrices whose elements' indexes, and whose counters, pass 32 bits, against the host's draws."""
import pytest

pytestmark = pytest.mark.gpu

fs = pytest.importorskip("fully_sharded_gb300")
np = pytest.importorskip("numpy")
torch = pytest.importorskip("torch")

from test_gpu_dropout import draws  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    torch.cuda.empty_cache()


def check_rows(x, rows, cols, p, seed, offset):
    """Some rows of dropout(ones): 1 / (1 - p) where the draw of the element's place is large enough, else 0."""
    t = round(65536 * p)
    kept = torch.tensor(65536 / (65536 - t), device="cuda").to(x.dtype)
    for r in rows:
        keep = torch.from_numpy(draws(r * cols, cols, seed, offset) >= t).cuda()
        assert torch.equal(x[r], torch.where(keep, kept, torch.zeros_like(kept))), r


@pytest.mark.parametrize("cols,pad", [(4096, 0), (4096, 8), (4095, 0), (4095, 2)])
def test_elements_beyond_32_bits(cols, pad):
    """In place, 2^32 elements and some rows: one long row, rows by vectors, one element after another (8.6 GB)."""
    rows = (1 << 32) // cols + 3
    whole = torch.full((rows * (cols + pad),), 1.0, dtype=BF16, device="cuda")
    x = torch.as_strided(whole, (rows, cols), (cols + pad, 1))
    fs.fsdp_dropout(x, x, 0.25, 2 ** 50 + 2, 3)
    half = (1 << 31) // cols
    check_rows(x, (0, half - 1, half, half + 1, rows - 4, rows - 3, rows - 2, rows - 1), cols, 0.25, 2 ** 50 + 2, 3)
    if pad:
        assert bool((torch.as_strided(whole, (rows, pad), (cols + pad, 1), cols) == 1.0).all())


def test_counters_beyond_32_bits():
    """2^35 elements and some rows, so that the last groups of eight have counters of 33 bits (69 GB, in place)."""
    cols, rows = 4096, (1 << 23) + 2
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free memory")
    x = torch.full((rows, cols), 1.0, dtype=BF16, device="cuda")
    fs.fsdp_dropout(x, x, 0.25, 5, 2 ** 40 + 7)
    check_rows(x, (0, rows - 4, rows - 3, rows - 2, rows - 1), cols, 0.25, 5, 2 ** 40 + 7)
