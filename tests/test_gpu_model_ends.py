"""The operators at a model's two ends used together: a tied unit trained on W virtual ranks, and calls side by side.

The model is embedding (scaled, added to its positions' rows) -> dropout -> RMS norm -> tied head with the softmax
cross entropy; every gradient goes to its tensor's place in the rank's flat bf16 row, the lookup's on top of the
head's, and the fused step reduces the rows, updates the state and gathers the parameters that the next forward reads.

Tolerance of a gradient, of its norm: the path from a parameter to its gradient rounds at most 12 arrays to bf16 (the
activations out, normalised and back, E, the scaled rows, the gradient itself, twice for the tied table), each by at
most 2^-8 of each element, so of its norm; the logits, at most 8 here (a row of the table is about 0.05 sqrt(104) long, a
normalised one sqrt(104): 5.2 where they point the same way), carry the
roundings of the normalised rows into the probabilities: 8 * 2^-8 more. 20 * 2^-8 in all.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

fs = pytest.importorskip("fully_sharded_gb300")
torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32
WORLD, ROWS, WIDTH, VOCAB, PLACES = 2, 192, 104, 515, 64
SHAPES = [(VOCAB, WIDTH), (PLACES, WIDTH), (WIDTH,)]
P, SEED = 0.25, 77


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def views(flat, places):
    return [flat[a:a + math.prod(s)].view(s) for a, s in zip(places, SHAPES)]


def workspace(n):
    return torch.empty(max(1, n), dtype=torch.uint8, device="cuda")


def gradients(full, places, row, tokens, targets, offset):
    """The rank's losses; its gradients are written to their places in `row`."""
    table, positions, gain = views(full, places)
    dtable, dpositions, dgain = views(row, places)
    at = torch.arange(ROWS, device="cuda") % PLACES
    scale = math.sqrt(WIDTH)
    h = torch.empty(ROWS, WIDTH, dtype=BF16, device="cuda")
    fs.fsdp_embedding(at, positions, h)
    fs.fsdp_embedding(tokens, table, h, scale=scale, addend=h)
    fs.fsdp_dropout(h, h, P, SEED, offset)
    y, rstd = torch.empty_like(h), torch.empty(ROWS, device="cuda")
    fs.fsdp_rmsnorm(h, gain, y, rstd=rstd)
    loss, dy = torch.empty(ROWS, device="cuda"), torch.empty_like(y)
    fs.fsdp_cross_entropy(y, table, targets, loss, workspace(fs.fsdp_cross_entropy_workspace(ROWS, WIDTH, VOCAB)), dhidden=dy,
                          dweight=dtable, scale=1.0 / ROWS)
    dh = torch.empty_like(h)
    fs.fsdp_rmsnorm_backward(dy, h, gain, rstd, dh, dgain, workspace(fs.fsdp_rmsnorm_backward_workspace(ROWS, WIDTH)))
    fs.fsdp_dropout(dh, dh, P, SEED, offset)
    ws = workspace(fs.fsdp_embedding_backward_workspace(ROWS, WIDTH, VOCAB))
    fs.fsdp_embedding_backward(tokens, dh, dtable, ws, scale=scale, accumulate=True)
    fs.fsdp_embedding_backward(at, dh, dpositions, ws)
    return loss


def wanted(full, places, tokens, targets, offset):
    """Losses and gradients by automatic differentiation of the formulas in 64 bits."""
    table, positions, gain = (v.double().requires_grad_() for v in views(full, places))
    at = torch.arange(ROWS, device="cuda") % PLACES
    keep = torch.empty(ROWS, WIDTH, device="cuda")
    fs.fsdp_dropout(torch.ones_like(keep), keep, P, SEED, offset)  # the mask and its factor, tested elsewhere
    there = tokens >= 0
    h = math.sqrt(WIDTH) * table[tokens.clamp(min=0)] * there[:, None] + positions[at]
    h = h * keep.double()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6) * gain
    logits = y @ table.t()
    assert float(logits.detach().abs().max()) < 8
    loss = torch.where(targets >= 0, torch.logsumexp(logits, 1) - logits.gather(1, targets.clamp(min=0)[:, None])[:, 0], 0.0)
    return loss.detach(), torch.autograd.grad(loss.sum() / ROWS, (table, positions, gain))


def test_a_tied_unit_is_trained():
    gen = torch.Generator(device="cuda").manual_seed(0)
    layout, offsets = fs.fsdp_flatten_layout([3] + [math.prod(s) for s in SHAPES], WORLD)  # an odd place for the table
    places = offsets[1:]
    shard, padded = layout.shard_numel, layout.padded_numel
    master = 0.05 * torch.randn(padded, generator=gen, device="cuda")
    master[layout.numel:] = 0
    master[places[2]:places[2] + WIDTH] = 1
    full = master.to(BF16)
    state = {k: list(torch.zeros(WORLD, shard, device="cuda")) for k in ("exp_avg", "exp_avg_sq")}
    masters = list(master.view(WORLD, shard).clone())
    batches = []
    for _ in range(WORLD):
        tokens = torch.randint(-1, VOCAB, (ROWS,), generator=gen, device="cuda")
        batches.append((tokens, torch.roll(tokens, -1)))
    for step in (1, 2):
        rows = torch.zeros(WORLD, padded, dtype=BF16, device="cuda")
        for rank, (tokens, targets) in enumerate(batches):
            loss = gradients(full, places, rows[rank], tokens, targets, 10 * step + rank)
            want_loss, want = wanted(full, places, tokens, targets, 10 * step + rank)
            assert float((loss.double() - want_loss).norm()) <= 20 * 2.0 ** -8 * float(want_loss.norm())
            for got, ref in zip(views(rows[rank], places), want):
                assert float((got.double() - ref).norm()) <= 20 * 2.0 ** -8 * float(ref.norm())
            assert bool((rows[rank, :places[0]] == 0).all()) and bool((rows[rank, layout.numel:] == 0).all())
        before = full.clone()
        fs.fsdp_shard_step(list(rows), layout, 0, WORLD, masters, state["exp_avg"], state["exp_avg_sq"], None, [full],
                           fs.AdamHyper(lr=1e-3, step=step))
        mean = rows.float().mean(0)
        moved = (full.float() - before.float())[:layout.numel]
        clear = mean[:layout.numel].abs() > 1e-4  # steps of about the learning rate against the gradient
        if step == 1:
            assert bool((torch.sign(moved[clear]) * torch.sign(mean[:layout.numel][clear]) <= 0).all()) and float(moved.abs().max()) > 0


def test_calls_side_by_side():
    """Two streams, each with workspaces of its own, give what one after the other gives."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    hidden = torch.randn(700, 256, generator=gen, device="cuda").to(BF16)
    weight = (torch.randn(3000, 256, generator=gen, device="cuda") / 16).to(BF16)
    targets = torch.randint(0, 3000, (700,), generator=gen, device="cuda")

    def both():
        loss, dh, dw = torch.empty(700, device="cuda"), torch.empty_like(hidden), torch.empty_like(weight)
        return (loss, dh, dw, torch.zeros_like(weight),
                workspace(fs.fsdp_cross_entropy_workspace(700, 256, 3000)), workspace(fs.fsdp_embedding_backward_workspace(700, 256, 3000)))

    def go(loss, dh, dw, dt, ws, ws2):
        fs.fsdp_cross_entropy(hidden, weight, targets, loss, ws, dhidden=dh, dweight=dw)
        fs.fsdp_embedding_backward(targets, hidden, dt, ws2)

    want = both()
    go(*want)
    torch.cuda.synchronize()
    sets = [both() for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, args in zip(streams, sets):
            with torch.cuda.stream(s):
                go(*args)
    torch.cuda.synchronize()
    for args in sets:
        assert all(torch.equal(a, b) for a, b in zip(args[:4], want[:4]))


def test_offsets_beyond_32_bits():
    """Rows so far apart that their offsets pass 2^32 elements."""
    rows, stride, cols = 2200, 1 << 21, 72
    whole = torch.empty(rows * stride, dtype=BF16, device="cuda")  # 9.2 GB
    gen = torch.Generator(device="cuda").manual_seed(2)
    wide = torch.as_strided(whole, (rows, cols), (stride, 1))
    narrow = torch.randn(rows, cols, generator=gen, device="cuda").to(BF16)
    wide.copy_(narrow)
    tokens = torch.randint(0, rows, (rows,), generator=gen, device="cuda")
    tokens[:2] = rows - 1
    targets = torch.randint(0, rows, (rows,), generator=gen, device="cuda")
    a, b = torch.empty_like(narrow), torch.empty_like(narrow)
    fs.fsdp_embedding(tokens, wide, a)
    fs.fsdp_embedding(tokens, narrow, b)
    assert torch.equal(a, b)
    fs.fsdp_dropout(wide, a, 0.5, 1)
    fs.fsdp_dropout(narrow, b, 0.5, 1)
    assert torch.equal(a, b)
    ws = workspace(fs.fsdp_embedding_backward_workspace(rows, cols, rows))
    fs.fsdp_embedding_backward(tokens, wide, a, ws)
    fs.fsdp_embedding_backward(tokens, narrow, b, ws)
    assert torch.equal(a, b)
    ws = workspace(fs.fsdp_cross_entropy_workspace(rows, cols, rows))
    results = []
    for h, w in ((wide, narrow), (narrow, wide), (narrow, narrow)):
        loss, dh, dw = torch.empty(rows, device="cuda"), torch.empty_like(narrow), torch.empty_like(narrow)
        fs.fsdp_cross_entropy(h, w, targets, loss, ws, dhidden=dh, dweight=dw)
        results.append((loss, dh, dw))
    for r in results[:2]:
        assert all(torch.equal(x, y) for x, y in zip(r, results[2]))
    fs.fsdp_cross_entropy(narrow, narrow, targets, loss, ws, dhidden=dh, dweight=wide)
    assert torch.equal(wide, results[2][2])
    fs.fsdp_embedding_backward(tokens, narrow, wide, workspace(fs.fsdp_embedding_backward_workspace(rows, cols, rows)))
    fs.fsdp_embedding_backward(tokens, narrow, b, workspace(fs.fsdp_embedding_backward_workspace(rows, cols, rows)))
    assert torch.equal(wide, b)
