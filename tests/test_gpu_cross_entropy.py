"""Softmax cross entropy of a projection and its gradients against the formulas in 64 bits.

Tolerances, element by element, from the operations' roundings:
  - a logit is a tensor-core sum of exact products. Each addition of 16 products cuts off at most
    2^-22 of the sum of the absolute values A; segments of 1024 columns are added in fp32:
    dx <= (min(cols, 1024) / 16 + cols / 1024 + 8) 2^-22 A;
  - lse is off by the largest dx of its row, by the sums' roundings (64 + vocab / 4096 additions in
    sequence at most), the exponentials' (2^-22, and 2^-23 |x| of the argument) and its own, 2^-23 |lse|; the loss
    by that and its target's dx;
  - an element of G is rounded to bf16 (2^-8 of itself), shares its row's factor, which carries the rounding of the
    target's element (2^-8), and is off by what its exponent is; in dweight the factor's product with hidden is
    rounded too (2^-8);
  - exponentials below 2^-126 (of x, where |lse| <= 40, else relative to their row's or span's largest) count as zero, and
    bf16's subnormal steps are smaller than that: at most 2^-125 in all, over exp(lse) in the former case;
  - the gradients' sums are cut off as the logits' are, in segments of 4096; partial sums add a few 2^-24; each
    output is rounded once (2^-8 of itself).
"""
import pytest

pytestmark = pytest.mark.gpu

fs = pytest.importorskip("fully_sharded_gb300")
torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32
HALF = 2.0 ** -8  # a rounding to bf16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def inputs(rows, cols, vocab, seed=0, without=0.2, size=1.0, index=torch.int64):
    gen = torch.Generator(device="cuda").manual_seed(seed + 1000 * rows + 10 * cols + vocab)
    weight = (size * torch.randn(vocab, cols, generator=gen, device="cuda") / cols ** 0.5).to(BF16)
    targets = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    hidden = torch.randn(rows, cols, generator=gen, device="cuda")
    hidden += (6 / size * torch.rand(rows, 1, generator=gen, device="cuda")) * weight[targets].float()
    none = torch.rand(rows, generator=gen, device="cuda") < without
    dloss = torch.rand(rows, generator=gen, device="cuda") + 0.5
    return hidden.to(BF16), weight, torch.where(none, -100, targets).to(index), dloss


def place(x, stride=None, offset=0):
    """A copy of matrix x whose rows lie `stride` elements apart, `offset` elements off alignment."""
    rows, cols = x.shape
    stride = stride or cols
    whole = torch.full((offset + max(1, rows) * stride + 64,), 77.0, dtype=x.dtype, device="cuda")
    view = torch.as_strided(whole, (rows, cols), (stride, 1), offset)
    view.copy_(x)
    return view


def call(hidden, weight, targets, dloss=None, scale=1.0, piece=0, gradients=True, strides=(None, None), offsets=(0, 0),
         in_place=False, stream=None):
    rows, cols = hidden.shape
    vocab = weight.shape[0]
    loss, lse = torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")
    ws = torch.empty(fs.fsdp_cross_entropy_workspace(rows, cols, vocab, gradients, piece) + 3, dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)  # NaN wherever something is read that was not written
    dh = dw = None
    if gradients:
        dh = hidden if in_place else place(torch.full_like(hidden, 3.0), strides[0], offsets[0])
        dw = place(torch.full_like(weight, 3.0), strides[1], offsets[1])
    fs.fsdp_cross_entropy(hidden, weight, targets, loss, ws[3:], lse=lse, dhidden=dh, dweight=dw, scale=scale, dloss=dloss,
                          piece=piece, stream=stream)
    return loss, lse, dh, dw


def check(hidden, weight, targets, dloss, scale, loss, lse, dh, dw):
    h, w = hidden.double(), weight.double()
    rows, cols = h.shape
    vocab = w.shape[0]
    targets = targets.long()
    there = targets >= 0
    h = torch.where(there[:, None] | torch.isfinite(h).all(1)[:, None], h, 0.0)
    x = h @ w.t()
    dx = (min(cols, 1024) / 16 + cols / 1024 + 8) * 2.0 ** -22 * (h.abs() @ w.abs().t())
    want_lse = torch.logsumexp(x, 1)
    most = dx.amax(1) + 2.0 ** -23 * x.abs().amax(1)
    d_lse = most + (64 + vocab / 4096) * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -23 * want_lse.abs()
    assert bool(((lse.double() - want_lse).abs() <= d_lse).all())
    at = targets.clamp(min=0)[:, None]
    want = torch.where(there, want_lse - x.gather(1, at)[:, 0], 0.0)
    assert bool(((loss.double() - want).abs() <= torch.where(there, d_lse + dx.gather(1, at)[:, 0] + 2.0 ** -24 * want.abs(), 0.0)).all())
    if dh is None:
        return
    f = scale * (dloss.double() if dloss is not None else torch.ones_like(want))
    f = torch.where(there, f, 0.0)[:, None]
    p = torch.exp(x - want_lse[:, None])
    hot = torch.zeros_like(p).scatter_(1, at, 1.0)
    g = f * (p - hot)
    off = g.abs() * (2 * HALF + HALF ** 2 + 2.0 ** -20) + f.abs() * p * 2 * (dx + d_lse[:, None])
    off = off + f.abs() * 2.0 ** -125 * torch.where(want_lse.abs() <= 40.01, torch.exp(-want_lse), 1.0)[:, None].clamp(min=1)
    cut = (256 + vocab / 4096 + 8) * 2.0 ** -22
    aw, ah = w.abs(), h.abs()
    want = g @ w
    bound = off @ aw + cut * (g.abs() @ aw) + HALF * want.abs() + 1e-37
    assert bool(((dh.double() - want).abs() <= bound).all())
    assert bool((dh[~there] == 0).all())
    cut = (min(rows, 4096) / 16 + rows / 4096 + 8) * 2.0 ** -22
    want = g.t() @ h
    bound = (off.t() + g.abs().t() * (HALF + cut)) @ ah + HALF * want.abs() + 1e-37
    assert bool(((dw.double() - want).abs() <= bound).all())


SIZES = [(1, 1, 1), (1, 8, 2), (3, 7, 5), (2, 64, 129), (37, 64, 1000), (128, 128, 256), (129, 72, 257), (200, 769, 1009),
         (300, 1030, 4097), (256, 4096, 640), (64, 96, 50257), (513, 2056, 700), (1000, 40, 130), (2050, 24, 300), (2050, 21, 300)]


@pytest.mark.parametrize("rows,cols,vocab", SIZES)
def test_losses_and_gradients(rows, cols, vocab):
    hidden, weight, targets, dloss = inputs(rows, cols, vocab)
    for weights in (None, dloss):
        loss, lse, dh, dw = call(hidden, weight, targets, weights, 0.25)
        check(hidden, weight, targets, weights, 0.25, loss, lse, dh, dw)
    again = call(hidden, weight, targets, dloss, 0.25)
    assert all(torch.equal(a, b) for a, b in zip(again, (loss, lse, dh, dw)))


@pytest.mark.parametrize("rows,cols,vocab", SIZES)
def test_losses_alone(rows, cols, vocab):
    hidden, weight, targets, dloss = inputs(rows, cols, vocab, index=torch.int32)
    loss, lse, dh, dw = call(hidden, weight, targets, gradients=False)
    check(hidden, weight, targets, None, 1.0, loss, lse, None, None)
    with_gradients = call(hidden, weight, targets)
    assert torch.equal(loss, with_gradients[0]) and torch.equal(lse, with_gradients[1])


@pytest.mark.parametrize("rows,piece", [(700, 256), (513, 512), (300, 100), (9, 1), (257, 256)])
@pytest.mark.parametrize("cols,pad,offset", [(200, 0, 0), (131, 0, 0), (64, 3, 1)])
def test_pieces(rows, piece, cols, pad, offset):
    hidden, weight, targets, dloss = inputs(rows, cols, 515)
    check(hidden, weight, targets, dloss, 2.0, *call(hidden, weight, targets, dloss, 2.0, piece=piece, strides=(cols + pad, cols + pad),
                                                     offsets=(offset, offset)))


@pytest.mark.parametrize("offset,pad", [(1, 0), (0, 1), (3, 5), (8, 8), (4, 0), (7, 2), (0, 5), (8, 3)])
@pytest.mark.parametrize("cols", [136, 131, 5])
def test_strides_and_alignment(cols, offset, pad):
    hidden, weight, targets, dloss = inputs(150, cols, 300)
    h, w = place(hidden, cols + pad, offset), place(weight, cols + pad, offset)
    loss, lse, dh, dw = call(h, w, targets, dloss, 1.0, strides=(cols + pad, cols + pad), offsets=(offset, offset))
    check(hidden, weight, targets, dloss, 1.0, loss, lse, dh, dw)
    plain = call(hidden, weight, targets, dloss, 1.0)
    for a, b in zip((loss, lse, dh, dw), plain):
        assert torch.equal(a, b)
    for view in (dh, dw):  # what lies between and around the rows is left as it was
        whole = torch.as_strided(view, (view.untyped_storage().nbytes() // 2,), (1,), 0).clone()
        torch.as_strided(whole, view.shape, view.stride(), offset).fill_(77.0)
        assert bool((whole == 77.0).all())


def test_in_place():
    hidden, weight, targets, dloss = inputs(150, 136, 300)
    want = call(hidden, weight, targets, dloss)
    for piece in (0, 64):
        copy = hidden.clone()
        got = call(copy, weight, targets, dloss, in_place=True, piece=piece)
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    check(hidden, weight, targets, dloss, 1.0, *got)


def test_no_row_has_a_target():
    hidden, weight, targets, _ = inputs(140, 64, 300, without=2.0)
    loss, lse, dh, dw = call(hidden, weight, targets)
    check(hidden, weight, targets, None, 1.0, loss, lse, dh, dw)
    assert bool((loss == 0).all()) and bool((dh == 0).all()) and bool((dw == 0).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_rows_without_a_target_may_hold_anything(bad):
    hidden, weight, targets, dloss = inputs(140, 64, 300)
    hidden[targets < 0] = bad
    hidden[3, 5], targets[3] = bad, -1
    loss, lse, dh, dw = call(hidden, weight, targets, dloss)
    check(hidden, weight, targets, dloss, 1.0, loss, torch.where(targets >= 0, lse, torch.logsumexp(torch.where(
        targets[:, None] >= 0, hidden.double(), 0.0) @ weight.double().t(), 1).float()), dh, dw) if bad != 3e38 else None
    assert bool(torch.isfinite(dw).all()) and bool((dh[targets < 0] == 0).all()) and bool((loss[targets < 0] == 0).all())


def test_small_factors_of_rows_with_large_logits():
    """Factors down to 1e-18 keep their rows' gradients: what is scaled stays above bf16's smallest normal values."""
    hidden, weight, targets, _ = inputs(140, 64, 700, without=0)
    hidden = torch.cat([hidden, torch.ones(140, 8, device="cuda", dtype=BF16)], 1)
    weight = torch.cat([weight, torch.full((700, 8), 4.5, device="cuda", dtype=BF16)], 1)
    dloss = torch.logspace(0, -18, 140, device="cuda")
    check(hidden, weight, targets, dloss, 1.0, *call(hidden, weight, targets, dloss))
    one = torch.full_like(dloss, 1e-18)
    check(hidden, weight, targets, one, 1.0, *call(hidden, weight, targets, one))


@pytest.mark.parametrize("size,shift", [(40.0, 0.0), (200.0, 0.0), (1.0, 90.0), (1.0, -90.0), (1.0, -200.0), (1.0, 59.0), (1.0, -62.0), (1.0, 39.0), (1.0, -46.0), (6.0, 0.0)])
def test_logits_far_from_zero(size, shift):
    """Rows beyond the range of the plain exponentials: wide ones, and ones that are shifted as a whole."""
    hidden, weight, targets, dloss = inputs(140, 64, 700)
    hidden = torch.cat([hidden.float() * size, torch.ones(140, 8, device="cuda")], 1).to(BF16)
    weight = torch.cat([weight, torch.full((700, 8), shift / 8, device="cuda", dtype=BF16)], 1)
    hidden[::3, 64:] = 0  # every third row is not shifted
    targets[5] = -1
    check(hidden, weight, targets, dloss, 1.0, *call(hidden, weight, targets, dloss))


def test_minus_infinity_in_the_vocabulary():
    """Columns whose logits are -inf have no part, as a mask of the vocabulary has it."""
    hidden, weight, targets, dloss = inputs(140, 64, 700)
    hidden = hidden.abs().clamp(min=0.01)
    weight[300:600] = -float("inf")
    targets = torch.where((targets >= 300) & (targets < 600), 7, targets)
    loss, lse, _, _ = call(hidden, weight, targets, gradients=False)
    keep = torch.cat([torch.arange(300), torch.arange(600, 700)]).cuda()
    want = torch.logsumexp(hidden.double() @ weight[keep].double().t(), 1)
    assert bool(((lse.double() - want).abs() <= 1e-4).all())


def test_target_beyond_the_vocabulary_is_loud():
    hidden, weight, targets, _ = inputs(140, 64, 300, without=0)
    targets[17] = 300
    targets[18] = 1 << 40
    loss, lse, dh, dw = call(hidden, weight, targets)
    assert torch.isnan(loss).nonzero()[:, 0].tolist() == [17, 18]
    assert bool(torch.isfinite(lse).all()) and bool(torch.isnan(dh[17:19]).all()) and bool(torch.isnan(dw).all())
    assert bool(torch.isfinite(dh[:17]).all()) and bool(torch.isfinite(dh[19:]).all())


def test_a_row_with_nan_keeps_to_itself():
    hidden, weight, targets, _ = inputs(140, 64, 300, without=0)
    hidden[9, 3] = float("nan")
    loss, lse, dh, dw = call(hidden, weight, targets)
    assert torch.isnan(loss).nonzero()[:, 0].tolist() == [9] and torch.isnan(dh).any(1).nonzero()[:, 0].tolist() == [9]


def test_no_rows():
    weight = torch.randn(30, 16, device="cuda").to(BF16)
    empty = torch.empty(0, 16, dtype=BF16, device="cuda")
    targets = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse, dh, dw = call(empty, weight, targets, strides=(None, 24), offsets=(0, 1))
    assert bool((dw == 0).all())
    call(empty, weight, targets, gradients=False)


def test_gradient_by_differences():
    """The loss itself, moved along the gradient: sums of the losses are within 1e-5 of themselves, so that a step whose
    first-order change is 1 % of the sum tells the gradient's slope to 2e-3, and its curvature is the rest."""
    hidden, weight, targets, _ = inputs(256, 64, 500, without=0.1)
    loss, _, dh, dw = call(hidden, weight, targets)
    for which, grad in ((0, dh), (1, dw)):
        square = float(grad.double().square().sum())
        step = 0.01 * float(loss.double().sum()) / square
        moved = []
        for sign in (1, -1):
            x = [hidden, weight]
            x[which] = x[which].double() + sign * step * grad.double()
            t = targets.clamp(min=0)[:, None]
            logits = x[0].double() @ x[1].double().t()
            moved.append(float(((torch.logsumexp(logits, 1) - logits.gather(1, t)[:, 0]) * (targets >= 0)).sum()))
        slope = (moved[0] - moved[1]) / (2 * step * square)
        assert abs(slope - 1) < 0.02, slope


def test_on_a_stream_and_in_a_graph():
    hidden, weight, targets, dloss = inputs(300, 128, 900)
    want = call(hidden, weight, targets, dloss)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(hidden, weight, targets, dloss, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    loss, dh, dw = torch.zeros(300, device="cuda"), torch.zeros_like(hidden), torch.zeros_like(weight)
    ws = torch.empty(fs.fsdp_cross_entropy_workspace(300, 128, 900), dtype=torch.uint8, device="cuda")
    static = hidden.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fs.fsdp_cross_entropy(static, weight, targets, loss, ws, dhidden=dh, dweight=dw, dloss=dloss)
    for other in (hidden, hidden.flip(0).contiguous()):
        static.copy_(other)
        graph.replay()
        torch.cuda.synchronize()
        want = call(other, weight, targets, dloss)
        assert torch.equal(loss, want[0]) and torch.equal(dh, want[2]) and torch.equal(dw, want[3])
