"""Trains a small block on W virtual ranks with the operators around the FlatParameter step.

The block is out = h + W2 silu(W1 rmsnorm(h)), h = x + residual: one FSDP unit
of a norm gain and two matrices. Each rank runs forward and backward on its own
batch; the norm's gradient of its gain goes straight to the gain's place in the
rank's flat bf16 gradient row, the matrices' gradients to theirs. One
fsdp_muon_step then reduces the rows, updates the matrices along their
orthogonalised momentum and the gain by Adam, and gathers the new bf16
parameters, which the next forward reads in place. The trained block is then
evaluated with the norm's output in 8 bits.

    python examples/muon_block.py --world 4 --steps 40
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fully_sharded_gb300 as fs  # noqa: E402


class Norm(torch.autograd.Function):
    """(h, y) = (x + residual, rmsnorm(h) gain); the gain's gradient is written to `dgain`."""

    @staticmethod
    def forward(ctx, x, residual, gain, dgain):
        h, y = torch.empty_like(x), torch.empty_like(x)
        rstd = torch.empty(x.shape[0], device=x.device)
        fs.fsdp_rmsnorm(x, gain, y, residual=residual, h_out=h, rstd=rstd)
        ctx.save_for_backward(h, gain, rstd)
        ctx.dgain = dgain
        return h, y

    @staticmethod
    def backward(ctx, dh, dy):
        h, gain, rstd = ctx.saved_tensors
        dx = torch.empty_like(h)
        workspace = torch.empty(fs.fsdp_rmsnorm_backward_workspace(*h.shape), dtype=torch.uint8, device=h.device)
        fs.fsdp_rmsnorm_backward(dy.contiguous(), h, gain, rstd, dx, ctx.dgain, workspace, dh=dh.contiguous())
        return dx, dx, None, None


class Block:
    """The unit's flat parameters, gradients and sharded state on one GPU."""

    def __init__(self, width: int, inner: int, world: int, seed: int):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.shapes = [(width,), (inner, width), (width, inner)]
        self.layout, offsets = fs.fsdp_flatten_layout([math.prod(s) for s in self.shapes], world)
        padded = self.layout.padded_numel
        master = torch.zeros(padded, device="cuda")
        master[:width] = 1
        matrices = slice(width, self.layout.numel)
        master[matrices] = 0.02 * torch.randn(self.layout.numel - width, generator=gen, device="cuda")
        self.state = {"master": master, "exp_avg": torch.zeros_like(master), "exp_avg_sq": torch.zeros_like(master)}
        self.full = master.to(torch.bfloat16)
        self.grads = torch.zeros(world, padded, dtype=torch.bfloat16, device="cuda")
        self.places = list(zip(offsets, offsets[1:], self.shapes))
        tensors = [fs.MuonTensor(*s, 0.2 * math.sqrt(max(s))) if len(s) == 2 else fs.MuonTensor(s[0]) for s in self.shapes]
        self.unit = fs.MuonUnit(self.layout, tensors, list(self.grads), full_out=self.full,
                                **{k: list(v.view(world, -1)) for k, v in self.state.items()})
        self.workspace = torch.empty(fs.fsdp_muon_workspace(self.unit), dtype=torch.uint8, device="cuda")

    def views(self, flat):
        return [flat[a:b].view(s) for a, b, s in self.places]

    def loss(self, x, residual, target, rank: int):
        """The rank's loss; after backward() its gradients stand in its flat row."""
        gain, w1, w2 = self.views(self.full)
        dgain, dw1, dw2 = self.views(self.grads[rank])
        w1, w2 = w1.detach().requires_grad_(), w2.detach().requires_grad_()
        dw1.zero_(), dw2.zero_()
        w1.grad, w2.grad = dw1, dw2
        h, y = Norm.apply(x.requires_grad_(), residual, gain, dgain)
        out = h + torch.nn.functional.silu(y @ w1.t()) @ w2.t()
        return (out.float() - target.float()).square().mean()

    def eight_bit(self, x, residual, target, group: int):
        """The loss with the norm's output quantised in groups, as an 8-bit product would take it."""
        gain, w1, w2 = self.views(self.full)
        rows, cols = x.shape
        h, y = torch.empty_like(x), torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty(rows, -(-cols // group), device="cuda")
        fs.fsdp_rmsnorm(x, gain, y, residual=residual, h_out=h, scales=scales, group=group)
        wide = (y.float() * scales.repeat_interleave(group, 1)[:, :cols]).to(torch.bfloat16)
        out = h + torch.nn.functional.silu(wide @ w1.t()) @ w2.t()
        return (out.float() - target.float()).square().mean()


def run(world: int = 4, steps: int = 40, width: int = 320, inner: int = 800, rows: int = 512, seed: int = 0, say=print):
    """Trains the block; returns the losses by step and the 8-bit evaluation's."""
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    block = Block(width, inner, world, seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)

    teacher = [0.5 / math.sqrt(s[1]) * normal(*s) for s in block.shapes[1:]]
    batches = []
    for _ in range(world):
        x, residual = normal(rows, width), normal(rows, width)
        h = x + residual
        y = torch.nn.functional.rms_norm(h.float(), (width,), eps=1e-6).to(torch.bfloat16)
        batches.append((x, residual, h + torch.nn.functional.silu(y @ teacher[0].t()) @ teacher[1].t()))
    losses = []
    for step in range(1, steps + 1):
        total = 0.0
        for rank, (x, residual, target) in enumerate(batches):
            loss = block.loss(x.detach(), residual, target, rank)
            loss.backward()
            total += loss.detach()
        muon = fs.Muon(lr=0.01, adam=fs.AdamHyper(lr=0.003, beta1=0.9, beta2=0.95, step=step))
        fs.fsdp_muon_step(block.unit, muon, block.workspace)
        losses.append(float(total) / world)
        if say and (step == 1 or step % 10 == 0):
            say("step %3d  loss %.6f" % (step, losses[-1]))
    with torch.no_grad():
        eight = sum(float(block.eight_bit(*b, group=64)) for b in batches) / world
    if say:
        say("after the last step, with 8-bit norm outputs: loss %.6f" % eight)
    return losses, eight


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--world", type=int, default=4)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--width", type=int, default=320)
    ap.add_argument("--inner", type=int, default=800)
    ap.add_argument("--rows", type=int, default=512)
    args = ap.parse_args()
    run(args.world, args.steps, args.width, args.inner, args.rows)
