"""Cross entropy where rows need more care than the plain exponentials: confident rows, rows far from zero, both in
batches of many rows (a warp each) and of few (a block each)."""
import pytest

pytestmark = pytest.mark.gpu

fs = pytest.importorskip("fully_sharded_gb300")
torch = pytest.importorskip("torch")

from test_gpu_cross_entropy import HALF, call, check, inputs  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("rows", [1, 600, 2100])
@pytest.mark.parametrize("others,scale", [(-30.0, 1.0), (-39.0, 1.0), (-90.0, 1.0), (-90.0, 4.0)])
def test_no_loss_is_below_zero(rows, others, scale):
    """Rows whose target has all of the probability: logits 5 to 32 (times `scale`) against `others`. The target's element of G
    is p - 1 <= 0, and is the first column of dhidden here, whose weight is 0 in all other rows of the vocabulary.

    Tolerance: the loss itself is below 300 exp(others - 5) < 1e-12; the logit's two products are exact and their sum rounds
    once, the exponential is off by 2^-23 of its argument's size (at most 1.5 times the logit) and 2^-22, and the
    sum, the logarithm and the difference round once each: 8 roundings of the logit's size in all."""
    weight = torch.zeros(300, 8, device="cuda")
    weight[1:, 2] = others
    weight[0, :2] = torch.tensor([1.0, 2.0 ** -9])
    hidden = torch.zeros(rows, 8, device="cuda")
    hidden[:, 0] = scale * torch.linspace(5, 32, rows, device="cuda")
    hidden[:, 1] = torch.arange(rows, device="cuda") * 37 % 256 / 8
    hidden[:, 2] = 1
    hidden, weight = hidden.to(BF16), weight.to(BF16)
    targets = torch.zeros(rows, dtype=torch.int64, device="cuda")
    logit = hidden[:, 0].double() + hidden[:, 1].double() * 2.0 ** -9
    loss, lse, dh, dw = call(hidden, weight, targets)
    off = 8 * 2.0 ** -23 * logit + 2.0 ** -22
    assert bool((loss >= 0).all()) and bool((loss.double() <= off).all())
    assert bool(((lse.double() - logit).abs() <= off).all())
    assert bool((dh[:, 0] <= 0).all()) and bool((dh[:, 0].double().abs() <= off * (1 + 2 * HALF)).all())
