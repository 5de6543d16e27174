"""The routed-recurrence example: its gradients against float64 autograd on
plain operations, and the example itself; refusals of the binding on the GPU."""
import importlib.util
import os

import pytest
import torch

import tokens_ref as ref
from laplace_matvec_amd import laplex as lx

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("routed_recurrence",
                                                  os.path.join(ROOT, "examples", "routed_recurrence.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(layer, x, seq, seqs):
    """The layer in float64 on the host, token by token."""
    w = {k: v.detach().cpu().double().requires_grad_() for k, v in layer.named_parameters()}
    x = x.detach().cpu().double().requires_grad_()
    best, memory = (x @ w["router.weight"].T).topk(layer.slots, -1)
    weights = torch.softmax(best, -1)
    g = -torch.nn.functional.softplus(x @ w["gate.weight"].T + w["gate.bias"])
    v = x @ w["value.weight"].T
    per = v.shape[1] // g.shape[1]
    state, rows = {}, []
    for t in range(x.shape[0]):
        y = 0
        for k in range(layer.slots):
            key = int(seq[t]), int(memory[t, k])
            h = v[t] + (torch.exp(g[t]).repeat_interleave(per) * state[key] if key in state else 0)
            state[key] = h
            y = y + weights[t, k] * h
        rows.append(y)
    return torch.stack(rows), x, w


def test_layer_gradients(gpu, example):
    torch.manual_seed(1)
    layer = example.RoutedRecurrence(24, 6, 3, 2).to(gpu)
    lengths = (70, 1, 9)
    gen = torch.Generator(device=gpu).manual_seed(2)
    x, seq = example.batch(lengths, 24, gen, gpu)
    x.requires_grad_()
    y, _ = layer(x, seq, 3)
    dy = torch.randn(y.shape, device=gpu, generator=gen)
    (y * dy).sum().backward()
    want, xd, w = plain(layer, x, seq.cpu(), 3)
    (want * ref.d(dy)).sum().backward()
    # sums of some 80 terms of order 1 in float32, projections among them
    near = lambda a, b: float((ref.d(a) - b).norm() / b.norm()) < 1e-5  # noqa: E731
    assert near(y, want.detach()) and near(x.grad, xd.grad)
    for name, p in layer.named_parameters():
        assert near(p.grad, w[name].grad), name


def test_example(gpu, example):
    first, last, off = example.main(steps=40)
    assert last < 0.5 * first
    assert off < 1e-4


def test_refusals(gpu):
    x, g = torch.zeros(6, 8, device=gpu), torch.zeros(6, 2, device=gpu)
    ids = torch.zeros(6, 2, dtype=torch.int64, device=gpu)
    route = lx.laplex_route(ids, 4)
    at = torch.tensor([0, 6], dtype=torch.int32, device=gpu)
    state = torch.zeros(6, 8, device=gpu)
    wrong = {
        TypeError: [
            lambda: lx.laplex_route(ids.float(), 4),
            lambda: lx.laplex_route(ids.T, 4),
            lambda: lx.laplex_dispatch(route, x.double()),
            lambda: lx.laplex_combine(route, torch.zeros(12, 8, device=gpu), torch.zeros(6, 2, device=gpu).half()),
            lambda: lx.laplex_combine(route, torch.zeros(12, 8, device=gpu), torch.zeros(6, 2)),
            lambda: lx.laplex_combine_backward(route, x, torch.zeros(12, 8, device=gpu), None),
            lambda: lx.laplex_combine_backward(route, x, torch.zeros(12, 8, device=gpu).half(),
                                               torch.zeros(6, 2, device=gpu)),
            lambda: lx.laplex_recur(x.bfloat16(), g.half()),
            lambda: lx.laplex_recur(x, g, offsets=at.long()),
            lambda: lx.laplex_recur(x, g, offsets=at[:1]),
            lambda: lx.laplex_recur(x, g, h0=torch.zeros(1, 8, device=gpu).half()),
            lambda: lx.laplex_recur_backward(x, g, x, None),
            lambda: lx.laplex_recur_backward(x, g, x.half(), torch.zeros(0, device=gpu)),
            lambda: lx.laplex_recur_step(x, g, state.half()),
            lambda: lx.laplex_recur_step(x, g, state, slots=torch.zeros(6, dtype=torch.int64, device=gpu)),
        ],
        ValueError: [
            lambda: lx.laplex_route(ids, 0),
            lambda: lx.laplex_route(ids, 5000),
            lambda: lx.laplex_dispatch(route, x[:5]),
            lambda: lx.laplex_combine(route, torch.zeros(11, 8, device=gpu)),
            lambda: lx.laplex_combine(route, torch.zeros(12, 8, device=gpu), torch.zeros(12, device=gpu)),
            lambda: lx.laplex_combine_backward(route, x, torch.zeros(12, 7, device=gpu), torch.zeros(6, 2, device=gpu)),
            lambda: lx.laplex_recur(x, g[:5]),
            lambda: lx.laplex_recur(x, torch.zeros(6, 3, device=gpu)),
            lambda: lx.laplex_recur(x[0], g[0]),
            lambda: lx.laplex_recur(x[:1].expand(6, 8), g),                     # rows on top of each other
            lambda: lx.laplex_recur(x.T.contiguous().T, g),                     # no unit stride
            lambda: lx.laplex_recur(x.view(2, 3, 8), g.view(2, 3, 2), offsets=at),
            lambda: lx.laplex_recur(torch.zeros(2, 5, 8, device=gpu)[:, :3], g.view(2, 3, 2)),  # uneven rows
            lambda: lx.laplex_recur(x, g, h0=torch.zeros(2, 8, device=gpu)),
            lambda: lx.laplex_recur(x, g, h0=torch.zeros(1, 4, device=gpu)),
            lambda: lx.laplex_recur_backward(x, g, x[:5], torch.zeros(0, device=gpu)),
            lambda: lx.laplex_recur_backward(x, g, x, torch.zeros(3, device=gpu)),
            lambda: lx.laplex_recur_backward(x, g, x, torch.zeros(0, device=gpu), dfinal=torch.zeros(2, 8, device=gpu)),
            lambda: lx.laplex_recur_step(x, g, torch.zeros(6, 7, device=gpu)),
            lambda: lx.laplex_recur_step(x, g[:, :1].expand(6, 3), state),
            lambda: lx.laplex_recur_step(x, g, state, slots=torch.zeros(5, dtype=torch.int32, device=gpu)),
        ],
        lx.LaplexError: [
            lambda: lx.laplex_recur_step(x, g, state[:5]),                      # fewer states than requests
            lambda: lx.laplex_recur_step(x, g, state[:0]),
        ],
    }
    for kind, calls in wrong.items():
        for i, call in enumerate(calls):
            with pytest.raises(kind):
                call()
                pytest.fail(f"{kind.__name__} {i} was not refused")
