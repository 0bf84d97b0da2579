"""Embedding lookup and its gradient by sorted tokens against the formulas in 64 bits.

Tolerances: the lookup's product and sum round in fp32 (2 * 2^-24 of the terms) and once to the output's type;
a gradient's sum of n rows is off by at most (64 + n / 128) 2^-24 of the sum of the terms' absolute values (16 rows in
sequence, then their n / 16 sums in sequence in eight shares or more, then the shares), two more roundings for the scale
and the table's own value, and one to the output's type.
"""
import pytest

pytestmark = pytest.mark.gpu

fs = pytest.importorskip("fully_sharded_gb300")
torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32
ROUND = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def rand(gen, *shape, dtype=F32):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def guarded(rows, cols, dtype, stride=None, offset=0):
    """A matrix in a buffer of 7s: (whole, view)."""
    stride = stride or cols
    whole = torch.full((offset + max(1, rows) * stride + 70,), 7.0, dtype=dtype, device="cuda")
    return whole, torch.as_strided(whole, (rows, cols), (stride, 1), offset)


def untouched(whole, view):
    rest = whole.clone()
    torch.as_strided(rest, view.shape, view.stride(), view.storage_offset()).fill_(7.0)
    return bool((rest == 7.0).all())


SIZES = [(1, 1, 1), (1, 4096, 10), (9000, 1024, 40), (5000, 520, 9), (5, 8, 3), (33, 769, 100), (300, 24, 1000), (70, 1000, 17), (2, 5000, 7), (1000, 33, 4)]


@pytest.mark.parametrize("rows,cols,vocab", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1), (8, 8)])
def test_lookup(rows, cols, vocab, dtype, pad, offset):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    table, addend = guarded(vocab, cols, dtype, cols + pad, offset)[1], rand(gen, rows, cols, dtype=dtype)
    table.copy_(rand(gen, vocab, cols))
    tokens = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    if rows > 2:
        tokens[1] = -1
    rowsof = torch.where(tokens[:, None] >= 0, table.double()[tokens.clamp(min=0)], 0.0)
    for index in (torch.int64, torch.int32):
        for scale, add in ((1.0, None), (3.3, None), (0.7, addend)):
            whole, out = guarded(rows, cols, dtype, cols + pad, offset)
            fs.fsdp_embedding(tokens.to(index), table, out, scale=scale, addend=add)
            want = scale * rowsof + (add.double() if add is not None else 0)
            size = scale * rowsof.abs() + (add.double().abs() if add is not None else 0)
            assert bool(((out.double() - want).abs() <= 3 * U * size + ROUND[dtype] * want.abs()).all())
            assert untouched(whole, out)
    out = addend.clone()
    fs.fsdp_embedding(tokens, table, out, scale=0.7, addend=out)
    again = torch.empty_like(out)
    fs.fsdp_embedding(tokens, table, again, scale=0.7, addend=addend)
    assert torch.equal(out, again)


def test_lookup_of_a_row_that_does_not_exist():
    table = torch.ones(10, 40, dtype=BF16, device="cuda")
    tokens = torch.tensor([0, 10, -5, 9, 1 << 40], device="cuda")
    out = torch.empty(5, 40, dtype=BF16, device="cuda")
    fs.fsdp_embedding(tokens, table, out)
    assert bool((out[[0, 3]] == 1).all()) and bool((out[2] == 0).all()) and bool(torch.isnan(out[[1, 4]]).all())


def want_gradient(tokens, dout, dtable, scale, accumulate):
    """(values, sum of the terms' absolute values, number of terms of each row)"""
    vocab = dtable.shape[0]
    t = tokens.long()
    there = (t >= 0) & (t < vocab)
    base = dtable.double() if accumulate else torch.zeros_like(dtable, dtype=torch.float64)
    total, size = base.clone(), base.abs()
    total.index_add_(0, t[there], scale * dout[there].double())
    size.index_add_(0, t[there], abs(scale) * dout[there].double().abs())
    return total, size, torch.bincount(t[there], minlength=vocab)[:, None]


def check_gradient(tokens, dout, dtable, scale, accumulate):
    want, size, n = want_gradient(tokens, dout, dtable, scale, accumulate)
    before = dtable.clone()
    rows, cols = dout.shape
    ws = torch.full((fs.fsdp_embedding_backward_workspace(rows, cols, dtable.shape[0]) + 5,), 0xFF, dtype=torch.uint8, device="cuda")
    fs.fsdp_embedding_backward(tokens, dout, dtable, ws[5:], scale=scale, accumulate=accumulate)
    assert bool(((dtable.double() - want).abs() <= (64 + n / 128 + 3) * U * size + ROUND[dtable.dtype] * want.abs()).all())
    if accumulate:
        rest = (n == 0)[:, 0]
        assert torch.equal(dtable[rest], before[rest])
    return dtable


GRADIENT = [(1, 1, 1), (1, 64, 5), (31, 8, 3), (32, 24, 1), (33, 769, 100), (700, 40, 1000), (64, 1000, 2), (5000, 48, 300),
            (3000, 17, 70000), (40000, 8, 50257), (20000, 128, 3), (70000, 3, 500), (300, 2, (1 << 24) + 10)]


@pytest.mark.parametrize("rows,cols,vocab", GRADIENT)
@pytest.mark.parametrize("dtype,table", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)], ids=["bb", "ff", "bf", "fb"])
def test_gradient(rows, cols, vocab, dtype, table):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    dout = rand(gen, rows, cols, dtype=dtype)
    tokens = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    tokens[torch.rand(rows, generator=gen, device="cuda") < 0.3] = vocab // 2  # one token much more often
    tokens[torch.rand(rows, generator=gen, device="cuda") < 0.05] = -1
    results = []
    for accumulate in (False, True, True):
        dtable = rand(torch.Generator(device="cuda").manual_seed(1), vocab, cols, dtype=table)
        results.append(check_gradient(tokens.to(torch.int32) if accumulate else tokens, dout, dtable, 1.7, accumulate))
    assert torch.equal(results[1], results[2])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (8, 8), (5, 3)])
@pytest.mark.parametrize("cols", [40, 77])
def test_gradient_in_a_flat_row(dtype, pad, offset, cols):
    """dtable anywhere in a buffer, dout's rows apart: what is between stays."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    dout = guarded(200, cols, dtype, cols + pad, offset)[1]
    dout.copy_(rand(gen, 200, cols))
    tokens = torch.randint(-1, 50, (200,), generator=gen, device="cuda")
    for accumulate in (False, True):
        whole, dtable = guarded(60, cols, dtype, cols + pad, offset)
        check_gradient(tokens, dout, dtable, 1.0, accumulate)
        assert untouched(whole, dtable)


@pytest.mark.parametrize("cols,dtype,pad,offset", [(256, BF16, 0, 0), (256, BF16, 8, 3), (129, F32, 0, 1), (131, F32, 2, 0)])
def test_gradient_of_a_large_table(cols, dtype, pad, offset):
    """Tables whose other rows are set to zero beside the sums: every row, those next to a named one included."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    dout = rand(gen, 900, cols, dtype=dtype)
    tokens = torch.randint(0, 70000, (900,), generator=gen, device="cuda")
    tokens[:8] = torch.tensor([0, 69999, 31, 32, 33, -1, 70000, 69998], device="cuda")
    tokens[100:300] = 4096
    whole, dtable = guarded(70000, cols, dtype, cols + pad, offset)
    check_gradient(tokens, dout, dtable, 1.5, False)
    assert untouched(whole, dtable)


@pytest.mark.parametrize("tokens", [[-1] * 100, [500] * 100, [-7, 500] * 50, [3] * 100, [0] * 50 + [9] * 50, list(range(9, -1, -1)) * 10],
                         ids=["none", "beyond", "neither", "one", "ends", "falling"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_of_special_tokens(tokens, accumulate):
    gen = torch.Generator(device="cuda").manual_seed(4)
    check_gradient(torch.tensor(tokens, device="cuda"), rand(gen, 100, 72, dtype=BF16), rand(gen, 10, 72, dtype=BF16), 2.0, accumulate)


def test_gradient_ignores_what_padding_rows_hold():
    gen = torch.Generator(device="cuda").manual_seed(5)
    dout, dtable = rand(gen, 100, 72, dtype=BF16), rand(gen, 10, 72, dtype=BF16)
    tokens = torch.randint(0, 10, (100,), generator=gen, device="cuda")
    tokens[::4] = -1
    dout[::4] = float("nan")
    fs.fsdp_embedding_backward(tokens, dout, dtable, torch.empty(fs.fsdp_embedding_backward_workspace(100, 72, 10), dtype=torch.uint8, device="cuda"))
    assert bool(torch.isfinite(dtable).all())


def test_no_rows():
    dtable = torch.ones(5, 9, device="cuda")
    dout, tokens = torch.empty(0, 9, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    fs.fsdp_embedding_backward(tokens, dout, dtable, None, accumulate=True)
    assert bool((dtable == 1).all())
    fs.fsdp_embedding_backward(tokens, dout, dtable, None)
    assert bool((dtable == 0).all())
    fs.fsdp_embedding(tokens, dtable, dout)


def test_gradient_is_the_lookups():
    """<dout, lookup(table + d) - lookup(table)> = <dtable, d>: both sides in 64 bits from fp32 results."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    tokens = torch.randint(-1, 30, (400,), generator=gen, device="cuda")
    table, dout, d = rand(gen, 30, 52), rand(gen, 400, 52), rand(gen, 30, 52)
    a, b, dtable = torch.empty_like(dout), torch.empty_like(dout), torch.empty_like(table)
    fs.fsdp_embedding(tokens, table + d, a, scale=1.5)
    fs.fsdp_embedding(tokens, table, b, scale=1.5)
    ws = torch.empty(fs.fsdp_embedding_backward_workspace(400, 52, 30), dtype=torch.uint8, device="cuda")
    fs.fsdp_embedding_backward(tokens, dout, dtable, ws, scale=1.5)
    left = (dout.double() * (a.double() - b.double())).sum()
    right = (dtable.double() * d.double()).sum()
    size = (dtable.double() * d.double()).abs().sum() + (dout.double() * a.double()).abs().sum()
    assert abs(float(left - right)) <= 16 * U * float(size)


@pytest.mark.parametrize("rows", [500, 20000, 70000])
def test_on_a_stream_and_in_a_graph(rows):
    gen = torch.Generator(device="cuda").manual_seed(7)
    tokens = torch.randint(0, 50, (rows,), generator=gen, device="cuda")
    dout, dtable = rand(gen, rows, 64, dtype=BF16), torch.empty(50, 64, dtype=BF16, device="cuda")
    ws = torch.empty(fs.fsdp_embedding_backward_workspace(rows, 64, 50), dtype=torch.uint8, device="cuda")
    out = torch.empty(rows, 64, dtype=BF16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fs.fsdp_embedding_backward(tokens, dout, dtable, ws)
        fs.fsdp_embedding(tokens, dtable, out, scale=0.5)
    for _ in range(2):
        tokens.copy_(tokens.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        other, looked = torch.empty_like(dtable), torch.empty_like(out)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        fs.fsdp_embedding_backward(tokens, dout, other, torch.empty_like(ws), stream=side)
        fs.fsdp_embedding(tokens, other, looked, scale=0.5, stream=side)
        side.synchronize()
        assert torch.equal(other, dtable) and torch.equal(looked, out)
