"""The Muon step of a unit against its formulas in 64 bits.

Tolerances: momentum and Adam state are fp32 with a few roundings of terms of the same
size, 1e-6 of the largest value. The orthogonalised update is off by 0.4 % of its
norm at most, as in the operator's own tests, and the master by lr * scale times that.
"""
import math

import pytest

import gpu_util as gu

pytestmark = pytest.mark.gpu

fs = pytest.importorskip("fully_sharded_gb300")
torch = pytest.importorskip("torch")

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def orthogonal(g):
    x = g.double()
    if x.shape[0] > x.shape[1]:
        return orthogonal(g.t()).t()
    x = x / (x.norm() + 1e-7)
    for _ in range(5):
        gram = x @ x.t()
        x = 3.4445 * x + (-4.7750 * gram + 2.0315 * gram @ gram) @ x
    return x


class Unit:
    def __init__(self, shapes, world, seed=0, odd=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.shapes, self.world = shapes, world
        self.layout, self.offsets = fs.fsdp_flatten_layout([math.prod(s) for s in shapes], world)
        padded, shard, numel = self.layout.padded_numel, self.layout.shard_numel, self.layout.numel

        def flat(scale):
            t = torch.zeros(padded, device="cuda")
            t[:numel] = scale * torch.randn(numel, generator=gen, device="cuda")
            return t

        def place(t):  # each in an allocation of its own, `odd` elements off alignment
            out = torch.empty(t.numel() + odd, dtype=t.dtype, device="cuda")[odd:]
            return out.copy_(t)

        self.grads = [place(flat(1e-2).to(BF16)) for _ in range(world)]
        state = {"master": flat(0.02), "exp_avg": flat(1e-2), "exp_avg_sq": flat(1e-3).abs()}
        self.state = {k: [place(t[r * shard:(r + 1) * shard]) for r in range(world)] for k, t in state.items()}
        self.full = place(torch.zeros(padded, dtype=BF16, device="cuda"))
        self.tensors = [fs.MuonTensor(s[0], s[1], 0.2 * math.sqrt(max(s))) if len(s) == 2 else fs.MuonTensor(s[0])
                        for s in shapes]
        self.unit = fs.MuonUnit(self.layout, self.tensors, self.grads, full_out=self.full, **self.state)

    def flat(self, name):
        return torch.cat(self.state[name]).double()

    def step(self, muon, stream=None):
        workspace = torch.empty(fs.fsdp_muon_workspace(self.unit, muon) + 1, dtype=torch.uint8, device="cuda")[1:]
        fs.fsdp_muon_step(self.unit, muon, workspace, stream=stream)
        torch.cuda.synchronize()

    def want(self, muon):
        g = torch.stack([t.double() for t in self.grads]).mean(0)
        out = {k: self.flat(k) for k in self.state}
        room = torch.zeros_like(g)
        for shape, at, end, tensor in zip(self.shapes, self.offsets, self.offsets[1:], self.tensors):
            if end == at:
                continue
            s = slice(at, end)
            p, m, v = (out[k][s] for k in ("master", "exp_avg", "exp_avg_sq"))
            if len(shape) == 2:
                m.mul_(muon.momentum).add_(g[s])
                u = g[s] + muon.momentum * m if muon.nesterov else m
                o = orthogonal(u.view(shape)).reshape(-1)
                p.mul_(1 - muon.lr * muon.weight_decay).sub_(muon.lr * tensor.scale * o)
                rms = float(o.norm()) / o.numel() ** 0.5
                room[s] = muon.lr * tensor.scale * 0.03 * o.abs().clamp(min=rms)
            else:
                a = muon.adam
                m.mul_(a.beta1).add_((1 - a.beta1) * g[s])
                v.mul_(a.beta2).add_((1 - a.beta2) * g[s] ** 2)
                p.sub_(a.lr * (m / (1 - a.beta1 ** a.step)) / ((v / (1 - a.beta2 ** a.step)).sqrt() + a.eps))
        return out, room

    def check(self, want, room):
        for name in ("exp_avg", "exp_avg_sq"):
            top = 1e-6 * float(want[name].abs().max())
            assert bool(((self.flat(name) - want[name]).abs() <= top).all()), name
        master = self.flat("master")
        assert bool(((master - want["master"]).abs() <= room + 1e-6 * want["master"].abs() + 1e-8).all())
        assert torch.equal(self.full, torch.cat(self.state["master"]).to(BF16))
        assert bool((master[self.layout.numel:] == 0).all())


TINY_MLP = [(64, 32), (32,), (32, 16), (16,)]
UNITS = {
    "tiny_mlp": (TINY_MLP, 4, 0),
    "one_rank": (TINY_MLP, 1, 0),
    "three_ranks_odd": ([(37, 53), (5,), (300, 257), (1, 9), (9, 1), (0,), (0, 4), (7,)], 3, 1),
    "matrices_only": ([(260, 300), (300, 260)], 8, 0),
    "vectors_only": ([(1000,), (33,)], 8, 0),
    "shards_inside_rows": ([(3, 2000)], 16, 3),
    "sixty_four_ranks": ([(40, 50), (11,), (5, 5)], 64, 0),
    "gpt2_block": ([(768,), (768,), (768, 2304), (2304,), (768, 768), (768,)], 8, 0),
}


@pytest.mark.parametrize("name", list(UNITS))
@pytest.mark.parametrize("nesterov,decay", [(True, 0.1), (False, 0.0)])
def test_step(name, nesterov, decay):
    shapes, world, odd = UNITS[name]
    unit = Unit(shapes, world, odd=odd)
    for step in (1, 2):
        muon = fs.Muon(lr=3e-3, momentum=0.9, nesterov=nesterov, weight_decay=decay,
                       adam=fs.AdamHyper(lr=1e-3, beta1=0.9, beta2=0.95, step=step))
        want, room = unit.want(muon)
        unit.step(muon)
        unit.check(want, room)


def test_adam_tensors_equal_the_shard_step_bit_for_bit():
    """What Adam updates is what fsdp_shard_step would have made of it."""
    a, b = Unit(TINY_MLP, 4, seed=3), Unit(TINY_MLP, 4, seed=3)
    hyper = gu.adam_hyper(5)
    a.step(fs.Muon(adam=hyper))
    fs.fsdp_shard_step(b.grads, b.layout, 0, 4, b.state["master"], b.state["exp_avg"], b.state["exp_avg_sq"], None,
                       [b.full], hyper)
    torch.cuda.synchronize()
    for i in (1, 3):
        s = slice(a.offsets[i], a.offsets[i + 1])
        assert torch.equal(a.full[s], b.full[s])
        for k in a.state:
            assert torch.equal(torch.cat(a.state[k])[s], torch.cat(b.state[k])[s])


def test_matrix_leaves_its_second_moment_alone():
    unit = Unit([(300, 280)], 2)
    before = unit.flat("exp_avg_sq")
    unit.step(fs.Muon())
    assert torch.equal(before, unit.flat("exp_avg_sq"))


def test_repeatable_on_another_stream_and_in_a_graph():
    shapes, muon = [(300, 260), (40,), (20, 30)], fs.Muon(lr=1e-3)
    a, b, c = (Unit(shapes, 3, seed=4) for _ in range(3))
    a.step(muon)
    torch.cuda.synchronize()
    b.step(muon, stream=torch.cuda.Stream())
    workspace = torch.empty(fs.fsdp_muon_workspace(c.unit, muon), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fs.fsdp_muon_step(c.unit, muon, workspace)
    graph.replay()
    torch.cuda.synchronize()
    for other in (b, c):
        assert torch.equal(a.full, other.full)
        assert all(torch.equal(x, y) for k in a.state for x, y in zip(a.state[k], other.state[k]))
