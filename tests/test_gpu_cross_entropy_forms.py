"""Cross entropy: the forms of a call together (pieces whose products are cut along the vocabulary, 32-bit targets with
gradients, a weight's rows far apart), against the formulas in 64 bits with the tolerances of test_gpu_cross_entropy.py."""
import pytest

pytestmark = pytest.mark.gpu

fs = pytest.importorskip("fully_sharded_gb300")
torch = pytest.importorskip("torch")

from test_gpu_cross_entropy import call, check, inputs  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("rows,cols,vocab,piece", [(300, 64, 50257, 128), (700, 200, 4097, 300), (513, 72, 9000, 256), (130, 40, 20000, 1),
                                                   (260, 131, 6000, 100)])
def test_pieces_of_a_product_cut_along_the_vocabulary(rows, cols, vocab, piece):
    if piece == 1:
        rows = 5
    hidden, weight, targets, dloss = inputs(rows, cols, vocab)
    got = call(hidden, weight, targets, dloss, 2.0, piece=piece)
    check(hidden, weight, targets, dloss, 2.0, *got)
    again = call(hidden, weight, targets, dloss, 2.0, piece=piece)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("rows,cols,vocab,piece", [(37, 64, 1000, 0), (300, 72, 4097, 128), (2050, 24, 300, 0)])
def test_targets_of_32_bits(rows, cols, vocab, piece):
    hidden, weight, targets, dloss = inputs(rows, cols, vocab)
    want = call(hidden, weight, targets, dloss, piece=piece)
    check(hidden, weight, targets, dloss, 1.0, *want)
    got = call(hidden, weight, targets.to(torch.int32), dloss, piece=piece)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_rows_and_a_weight_whose_rows_are_far_apart():
    """The zeros of dweight's rows, 2^31 bytes and more apart."""
    stride = (1 << 30) + 8
    whole = torch.full((2 * stride + 80,), 3.0, dtype=BF16, device="cuda")  # 4.3 GB
    dw = torch.as_strided(whole, (3, 72), (stride, 1))
    empty = torch.empty(0, 72, dtype=BF16, device="cuda")
    fs.fsdp_cross_entropy(empty, torch.zeros(3, 72, dtype=BF16, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"),
                          torch.empty(0, device="cuda"), None, dhidden=empty, dweight=dw)
    assert bool((dw == 0).all())
    for r in range(3):
        assert bool((whole[r * stride + 72:r * stride + 80] == 3).all())
    assert bool((whole[stride - 100:stride] == 3).all())


def test_a_single_row_beside_the_weight():
    """One row of a buffer whose other columns are the weight: its gradient goes beside it, into the same buffer."""
    hidden, weight, targets, _ = inputs(1, 64, 300, without=0)
    whole = torch.full((300, 192), 7.0, dtype=BF16, device="cuda")
    whole[:, :64] = weight
    whole[5, 64:128] = hidden[0]
    h, dh = whole[5:6, 64:128], whole[5:6, 128:192]
    dw, loss = torch.empty_like(weight), torch.empty(1, device="cuda")
    ws = torch.empty(fs.fsdp_cross_entropy_workspace(1, 64, 300), dtype=torch.uint8, device="cuda")
    fs.fsdp_cross_entropy(h, whole[:, :64], targets, loss, ws, dhidden=dh, dweight=dw)
    want = call(hidden, weight, targets)
    assert torch.equal(loss, want[0]) and torch.equal(dh, want[2]) and torch.equal(dw, want[3])
    whole[5, 64:] = 7.0
    assert bool((whole[:, 64:] == 7.0).all()) and torch.equal(whole[:, :64], weight)
