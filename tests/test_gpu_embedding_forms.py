"""The embedding's gradient in the forms that small cases do not reach: rows of several column tiles by vectors, and the
zeros of a large table behind each of the three ways to put the tokens in order. Tolerances of test_gpu_embedding.py."""
import pytest

pytestmark = pytest.mark.gpu

fs = pytest.importorskip("fully_sharded_gb300")
torch = pytest.importorskip("torch")

from test_gpu_embedding import check_gradient, guarded, rand, untouched  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("rows,cols,vocab", [(500, 2056, 100), (500, 4096, 1000), (40, 5000, 3), (300, 2053, 60)])
@pytest.mark.parametrize("dtype,table", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)], ids=["bb", "ff", "bf", "fb"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_wide_rows(rows, cols, vocab, dtype, table, accumulate):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    dout = rand(gen, rows, cols, dtype=dtype)
    tokens = torch.randint(-1, vocab, (rows,), generator=gen, device="cuda")
    tokens[torch.rand(rows, generator=gen, device="cuda") < 0.3] = vocab // 2
    check_gradient(tokens, dout, rand(gen, vocab, cols, dtype=table), 1.7, accumulate)


@pytest.mark.parametrize("rows", [900, 9000, 70000])
@pytest.mark.parametrize("cols,table,pad,offset", [(128, BF16, 0, 0), (128, BF16, 8, 3), (129, F32, 0, 1), (72, F32, 0, 0)])
def test_zeros_of_a_large_table(rows, cols, table, pad, offset):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    vocab = 150001
    dout = rand(gen, rows, cols, dtype=BF16)
    tokens = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    tokens[:8] = torch.tensor([0, vocab - 1, 31, 32, 33, -1, vocab, vocab - 2], device="cuda")
    tokens[100:500] = 4096
    for accumulate in (False, True):
        whole, dtable = guarded(vocab, cols, table, cols + pad, offset)
        check_gradient(tokens, dout, dtable, 1.5, accumulate)
        assert untouched(whole, dtable)


@pytest.mark.parametrize("rows", [9000, 70000])
def test_one_token_for_all_rows(rows):
    """A run through all chunks, in all column tiles; besides, runs that begin and end at the chunks' borders."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    dout = rand(gen, rows, 1032, dtype=BF16)
    for tokens in (torch.full((rows,), 7, device="cuda"), torch.arange(rows, device="cuda") // 16 % 50, torch.arange(rows, device="cuda") // 272):
        dtable = rand(gen, 400, 1032)
        first = check_gradient(tokens, dout, dtable.clone(), 1.0, True)
        assert torch.equal(first, check_gradient(tokens, dout, dtable.clone(), 1.0, True))


def test_a_single_row_beside_the_table():
    """The lookup's row in the buffer that holds the table, beside its columns."""
    whole = torch.full((40, 96), 7.0, dtype=BF16, device="cuda")
    whole[:, :32] = torch.randn(40, 32, device="cuda").to(BF16)
    before = whole.clone()
    tokens = torch.tensor([9], device="cuda")
    fs.fsdp_embedding(tokens, whole[:, :32], whole[5:6, 64:])
    assert torch.equal(whole[5, 64:96], before[9, :32])
    whole[5, 64:96] = 7.0
    assert torch.equal(whole, before)
