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


@pytest.mark.parametrize("rows", [1, 200, 2100])
@pytest.mark.parametrize("shift", [-88.0, -50.0, 0.0, 44.0, 96.0])
def test_exponentials_are_rounded_once(rows, shift):
    """Entries of the vocabulary that are the same have the same gradient, in whatever span of columns they lie: what is kept
    of a row is exp(x) rounded once, although spans have units of their own. In fp32 two such exponentials differ by at most
    2^-19 of themselves (2^-22 each by the instruction, 2^-19.5 by the rounding of an argument below 64), so their roundings
    to bf16 differ where a boundary, at least 2^-8 from the next, lies between: for 2^-11 of the pairs, with room 2^-9, and by one
    step, 2 h for h = 2^-8, which the results' own rounding may make 4 h."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    half, row = 128 * 100, rows // 2
    weight = torch.randn(half, 16, generator=gen, device="cuda") * 0.3
    weight[:, :8] = shift / 8
    weight = torch.cat([weight, weight])
    weight[half::128, 8:] = 0.05 * torch.arange(100, device="cuda")[:, None]  # the spans' largest: 0 to 40 above the others
    hidden = torch.randn(rows, 16, generator=gen, device="cuda") * 0.1
    hidden[row] = 1
    hidden, weight = hidden.to(BF16), weight.to(BF16)
    dloss = torch.zeros(rows, device="cuda")
    dloss[row] = 1
    targets = torch.full((rows,), half, device="cuda")
    _, _, _, dw = call(hidden, weight, targets, dloss)
    first, second = dw[:half], dw[half:]
    pairs = torch.ones(half, dtype=torch.bool, device="cuda")
    pairs[::128] = False
    first, second = first[pairs, 0].double(), second[pairs, 0].double()
    assert bool((first > 0).all())
    assert float((first != second).double().mean()) <= 2.0 ** -9
    assert bool(((first - second).abs() <= 4 * HALF * first).all())


def far_inputs(rows, cols, vocab, shifts):
    """Rows whose logits are all shifted by one of `shifts`, in turn."""
    hidden, weight, targets, dloss = inputs(rows, cols, vocab)
    by = torch.tensor(shifts, device="cuda")[torch.arange(rows, device="cuda") % len(shifts)]
    hidden = torch.cat([hidden, (by / 8)[:, None].expand(rows, 8).to(BF16)], 1)
    weight = torch.cat([weight, torch.ones(vocab, 8, device="cuda", dtype=BF16)], 1)
    return hidden, weight, targets, dloss


@pytest.mark.parametrize("rows", [140, 2050])
@pytest.mark.parametrize("shifts", [(-80.0,), (64.0,), (0.0, 90.0, -90.0), (-39.0, -41.0, 39.0, 41.0), (-128.0, 240.0)])
@pytest.mark.parametrize("vocab,index", [(700, torch.int64), (4097, torch.int32)])
def test_rows_far_from_zero(rows, shifts, vocab, index):
    hidden, weight, targets, dloss = far_inputs(rows, 64, vocab, shifts)
    targets = targets.to(index)
    check(hidden, weight, targets, dloss, 1.0, *call(hidden, weight, targets, dloss))
    for piece in (128, 1000):
        check(hidden, weight, targets, dloss, 1.0, *call(hidden, weight, targets, dloss, piece=piece))


@pytest.mark.parametrize("rows", [140, 2050])
def test_wide_rows(rows):
    """Logits spread over some hundreds, so that spans of the vocabulary have units of their own."""
    hidden, weight, targets, dloss = inputs(rows, 64, 1000)
    weight = (weight.float() * torch.linspace(1, 60, 1000, device="cuda")[:, None]).to(BF16)
    check(hidden, weight, targets, dloss, 1.0, *call(hidden, weight, targets, dloss))


@pytest.mark.parametrize("rows", [140, 2050])
@pytest.mark.parametrize("shift", [0.0, 70.0])
def test_bad_rows_among_rows_far_from_zero(rows, shift):
    hidden, weight, targets, _ = far_inputs(rows, 64, 700, (shift, -70.0))
    targets = targets.clamp(min=0)
    hidden[9, 3] = float("nan")       # a row with a target: loud, and alone
    targets[17], targets[18] = 700, 1 << 40
    hidden[20, 5], targets[20] = float("nan"), -1   # one without: nothing
    hidden[21, 5], targets[21] = float("inf"), -100
    loss, lse, dh, dw = call(hidden, weight, targets)
    loud = [9, 17, 18]
    assert torch.isnan(loss).nonzero()[:, 0].tolist() == loud and torch.isnan(dh).any(1).nonzero()[:, 0].tolist() == loud
    assert bool(torch.isnan(dh[loud]).all()) and bool(torch.isnan(dw).all())
    assert bool((dh[[20, 21]] == 0).all()) and bool((loss[[20, 21]] == 0).all())
    targets[loud] = -1
    hidden[[9, 20, 21]] = 0
    loss2, lse, dh2, dw2 = call(hidden, weight, targets)
    check(hidden, weight, targets, None, 1.0, loss2, lse, dh2, dw2)
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[loud] = False
    assert torch.equal(loss[rest], loss2[rest]) and torch.equal(dh[rest], dh2[rest])
