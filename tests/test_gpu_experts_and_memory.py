"""The block of the example: memory, routing and experts together, its
gradients against the same block of plain operations in float64."""
import pytest
import torch

from examples.experts_and_memory import Block, main, starts

pytestmark = pytest.mark.gpu


def test_the_example_runs(gpu):
    _, last, off = main(steps=4)
    assert last == last
    # the same token in two ways: float32 sums over up to 482 rows and 128 values, one after the other,
    # (482 + 3 * 128) 2^-23 of sums of absolute terms, which are at most some 16 times the largest result here
    assert off <= 16 * 866 * 2.0 ** -23


def plain(block, x, offsets, ids):
    """The block in float64, token by token; ids: the experts that were chosen."""
    p = {name: t.detach().cpu().double().requires_grad_() for name, t in block.named_parameters()}
    x = x.detach().cpu().double().requires_grad_()
    heads, dk, dv = p["gate.weight"].shape[0], block.dk, block.dv
    q, k, v = (x @ p["qkv.weight"].t()).split(block.parts, -1)
    q, k, v = q.unflatten(-1, (-1, dk)), k.unflatten(-1, (-1, dk)), v.unflatten(-1, (-1, dv))
    q, k = (t.repeat_interleave(heads // t.shape[1], 1) for t in (q, k))
    g = -torch.nn.functional.softplus(x @ p["gate.weight"].t() + p["gate.bias"])
    rows = []
    for a, b in zip(offsets, offsets[1:]):
        h = torch.zeros(heads, dk, dv, dtype=torch.float64)
        for t in range(a, b):
            h = g[t].exp()[:, None, None] * h + k[t][:, :, None] * v[t][:, None, :]
            rows.append(dk ** -0.5 * (q[t][:, :, None] * h).sum(1))
    x1 = x + torch.stack(rows).flatten(1) @ p["out.weight"].t()
    logits = (x1 @ p["router.weight"].t()).gather(1, ids)
    weights = torch.softmax(logits, -1)
    mixed = sum(weights[:, s, None] * torch.einsum("tio,to->ti", p["down"][ids[:, s]], torch.nn.functional.silu(
        torch.einsum("tio,to->ti", p["up"][ids[:, s]], x1))) for s in range(ids.shape[1]))
    return x1 + mixed, x, p


def test_gradients_of_the_block(gpu):
    torch.manual_seed(0)
    lengths, width = (70, 1, 33), 40
    block = Block(width, 4, 2, 16, 24, 5, 2, 56).to(gpu)
    x = torch.randn(sum(lengths), width, device=gpu, requires_grad=True)
    offsets = starts(lengths, gpu)
    chosen = []
    block.router.register_forward_hook(lambda m, i, o: chosen.append(o.detach().topk(block.slots, -1).indices.cpu()))
    y, _ = block(x, offsets)
    dy = torch.randn(y.shape, device=gpu)
    (y * dy).sum().backward()
    want, wx, p = plain(block, x, offsets.tolist(), chosen[0])
    (want * dy.cpu().double()).sum().backward()
    # a float32 chain of at most 12 sums of up to 104 terms, each off by 104 2^-24 of its absolute terms, which for sums of
    # random terms are some sqrt(104) times the result
    bound = 12 * 104 * 104 ** 0.5 * 2.0 ** -24
    pairs = [(y, want), (x.grad, wx.grad)] + [(t.grad, p[name].grad) for name, t in block.named_parameters()]
    for got, ref in pairs:
        assert float((got.detach().cpu().double() - ref.detach()).norm()) <= bound * float(ref.detach().norm())
