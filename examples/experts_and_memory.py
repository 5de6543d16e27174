"""A block of a language model: a gated matrix memory over packed sequences,
then experts for each token.

    attend     linear attention with a decay per head, heads sharing queries and keys
    route      tokens sorted by expert
    dispatch   rows to their experts
    experts    two products with an activation between them
    combine    rows back to their tokens, weighted by the router

Trains the block to follow another one, then continues its sequences token by
token on the states that the memory left.

    python examples/experts_and_memory.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from examples.routed_recurrence import Combine, Dispatch, batch  # noqa: E402
from laplace_matvec_amd import laplex as lx  # noqa: E402


class Attend(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, offsets, scale):
        r = lx.laplex_attend(q, k, v, g, offsets=offsets, scale=scale, final=True, keep=True)
        ctx.save_for_backward(q, k, v, g, r.states, offsets)
        ctx.scale = scale
        ctx.mark_non_differentiable(r.final)
        return r.y, r.final

    @staticmethod
    def backward(ctx, dy, _):
        q, k, v, g, states, offsets = ctx.saved_tensors
        d = lx.laplex_attend_backward(q, k, v, g, dy.contiguous(), states, offsets=offsets, scale=ctx.scale,
                                      want=("dq", "dk", "dv", "dg"))
        return d["dq"], d["dk"], d["dv"], d["dg"], None, None


class Experts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(x, w, offsets)
        return lx.laplex_experts(x, w, offsets)

    @staticmethod
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        d = lx.laplex_experts_backward(x, w, dy.contiguous(), offsets)
        return d["dx"], d["dw"], None


class Block(torch.nn.Module):
    def __init__(self, width, heads, shared, dk, dv, experts, slots, inner):
        super().__init__()
        self.parts = (shared * dk, shared * dk, heads * dv)
        self.dk, self.dv, self.experts, self.slots = dk, dv, experts, slots
        self.qkv = torch.nn.Linear(width, sum(self.parts), bias=False)
        self.gate = torch.nn.Linear(width, heads)
        self.out = torch.nn.Linear(heads * dv, width, bias=False)
        self.router = torch.nn.Linear(width, experts, bias=False)
        self.up = torch.nn.Parameter(torch.randn(experts, inner, width) * width ** -0.5)
        self.down = torch.nn.Parameter(torch.randn(experts, width, inner) * inner ** -0.5)

    def project(self, x):
        """q, k and v as parts of one projection's rows, and the decays."""
        q, k, v = self.qkv(x).split(self.parts, -1)
        g = -torch.nn.functional.softplus(self.gate(x).float())
        return q.unflatten(-1, (-1, self.dk)), k.unflatten(-1, (-1, self.dk)), v.unflatten(-1, (-1, self.dv)), g

    def mix(self, x):
        """The experts' part: each token to its best experts and back."""
        best, ids = self.router(x).float().topk(self.slots, -1)
        route = lx.laplex_route(ids, self.experts)
        rows = torch.nn.functional.silu(Experts.apply(Dispatch.apply(x, route), self.up, route.offsets))
        return Combine.apply(Experts.apply(rows, self.down, route.offsets), torch.softmax(best, -1), route)

    def forward(self, x, offsets):
        """x [tokens, width] of the sequences offsets; returns y and the memory's states."""
        y, states = Attend.apply(*self.project(x), offsets, self.dk ** -0.5)
        x = x + self.out(y.flatten(1))
        return x + self.mix(x), states

    @torch.no_grad()
    def step(self, x, states):
        """One more token for each sequence; states are updated."""
        y = lx.laplex_attend_step(*self.project(x), states, scale=self.dk ** -0.5)
        x = x + self.out(y.flatten(1))
        return x + self.mix(x)


def starts(lengths, device):
    return torch.tensor([0, *lengths], device=device).cumsum(0).to(torch.int32)


def main(width=128, heads=8, shared=2, dk=32, dv=24, experts=8, slots=2, inner=96, lengths=(300, 17, 1, 482), steps=40):
    """Returns the first and last training loss, and how far the token-by-token
    form is from the packed one."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(0)
    torch.manual_seed(0)
    sizes = (width, heads, shared, dk, dv, experts, slots, inner)
    teacher, block = Block(*sizes).to(dev), Block(*sizes).to(dev)
    block.router.load_state_dict(teacher.router.state_dict())  # the choice itself has no gradient
    opt = torch.optim.Adam(block.parameters(), 2e-3)
    offsets = starts(lengths, dev)
    losses = []
    for _ in range(steps):
        x, _ = batch(lengths, width, gen, dev)
        with torch.no_grad():
            want, _ = teacher(x, offsets)
        y, _ = block(x, offsets)
        loss = (y - want).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())

    x, seq = batch(lengths, width, gen, dev)
    with torch.no_grad():
        whole, _ = block(x, offsets)
        first = torch.cat([(seq == q).nonzero()[:-1, 0] for q in range(len(lengths))])  # all but the last tokens
        _, states = block(x[first], starts([n - 1 for n in lengths], dev))
    last = offsets[1:].long() - 1
    y = block.step(x[last], states)
    off = float((y - whole[last]).abs().max() / whole[last].abs().max())
    return losses[0], losses[-1], off


if __name__ == "__main__":
    first, last, off = main()
    print(f"loss {first:.4f} -> {last:.4f}; token by token against packed: {off:.1e}")
