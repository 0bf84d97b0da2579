"""The example block: the operators together, as a training loop calls them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

fs = pytest.importorskip("fully_sharded_gb300")
torch = pytest.importorskip("torch")

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "muon_block.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    spec = importlib.util.spec_from_file_location("muon_block", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("world,width,inner", [(4, 320, 800), (3, 33, 70), (1, 64, 64)])
def test_the_block_learns(example, world, width, inner):
    losses, eight = example.run(world=world, steps=30, width=width, inner=inner, rows=128, say=None)
    assert losses[-1] < 0.5 * losses[0]
    assert eight < 0.7 * losses[0]


def test_gradients_reach_their_places(example):
    """The flat gradient row equals what autograd makes of the same block in 64 bits, to bf16's rounding
    of the forward and backward products (a few times 2^-8 of each gradient's largest value)."""
    block = example.Block(48, 96, 2, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, residual, target = (torch.randn(64, 48, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3))
    block.loss(x, residual, target, 1).backward()
    wide = [t.detach().double().requires_grad_() for t in block.views(block.full)]
    h = (x.detach() + residual).double()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * wide[0]
    out = h + torch.nn.functional.silu(y @ wide[1].t()) @ wide[2].t()
    (out - target.double()).square().mean().backward()
    for got, want in zip(block.views(block.grads[1]), wide):
        top = float(want.grad.abs().max())
        assert float((got.double() - want.grad).abs().max()) < 8 * 2.0 ** -8 * top
    assert bool((block.grads[0] == 0).all())
