"""Token routing, dispatch, combine and its gradient against plain float64."""
import pytest
import torch

import tokens_ref as ref
from laplace_matvec_amd import laplex as lx

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def ids_of(tokens, slots, experts, seed, dropped=0.1, dtype=torch.int64):
    gen = torch.Generator().manual_seed(seed)
    ids = (torch.rand(tokens, slots, generator=gen).pow(2) * experts).to(dtype)
    if dropped:
        ids[torch.rand(tokens, slots, generator=gen) < dropped] = -1
    return ids


def check_route(r, ids, experts):
    flat = ids.reshape(-1).to(torch.int64)
    valid = (flat >= 0) & (flat < experts)
    key = torch.where(valid, flat, experts)
    srt, order = torch.sort(key, stable=True)
    kept = int(valid.sum())
    want = torch.full((flat.numel(),), -1, dtype=torch.int32)
    want[:kept] = order[:kept].to(torch.int32)
    place = torch.full((flat.numel(),), -1, dtype=torch.int32)
    place[order[:kept]] = torch.arange(kept, dtype=torch.int32)
    offsets = torch.searchsorted(srt, torch.arange(experts + 1)).to(torch.int32)
    assert torch.equal(r.order.cpu(), want)
    assert torch.equal(r.place.cpu().reshape(-1), place)
    assert torch.equal(r.offsets.cpu(), offsets)


# one wave, one tile's edges, several tiles, more than 256 tiles of the scan
@pytest.mark.parametrize("tokens,slots", [(1, 1), (63, 1), (64, 1), (65, 2), (1365, 3), (1024, 4), (4097, 1),
                                          (12289, 1), (30000, 8), (1100000, 1)])
@pytest.mark.parametrize("experts", [1, 2, 16, 17, 256, 257, 4096])
def test_route(gpu, tokens, slots, experts):
    ids = ids_of(tokens, slots, experts, tokens + experts)
    check_route(lx.laplex_route(ids.to(gpu), experts), ids, experts)


def test_route_small_against_lists(gpu):
    ids = torch.tensor([[3, 0], [7, 3], [-1, 8], [2, 3], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32)
    for dtype in (torch.int32, torch.int64):
        r = lx.laplex_route(ids.to(gpu, dtype), 8)
        for got, want in zip(r, ref.route(ids, 8)):
            assert torch.equal(got.cpu(), want)
    wide = torch.tensor([2 ** 32, 2 ** 32 + 3, 1, -2 ** 63], dtype=torch.int64)  # not folded into 32 bits
    r = lx.laplex_route(wide.to(gpu), 8)
    assert r.order.tolist() == [2, -1, -1, -1] and r.place.reshape(-1).tolist() == [-1, -1, 0, -1]


@pytest.mark.parametrize("tokens", [0, 5, 5000])
def test_route_all_dropped_or_one_expert(gpu, tokens):
    for value in (-1, 5, 9):
        ids = torch.full((tokens, 2), value, dtype=torch.int32)
        check_route(lx.laplex_route(ids.to(gpu), 7), ids, 7)


def test_route_keeps_no_state_between_calls(gpu):
    a, b = ids_of(20000, 2, 100, 1), ids_of(20000, 2, 100, 2, dropped=0)
    for _ in range(3):
        check_route(lx.laplex_route(a.to(gpu), 100), a, 100)
        check_route(lx.laplex_route(b.to(gpu), 100), b, 100)


SHAPES = [(1, 1, 1), (3, 2, 7), (5, 3, 8), (130, 4, 64), (67, 1, 1001), (33, 8, 2049), (20, 11, 516), (2, 2, 16640)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,slots,width", SHAPES)
def test_dispatch_combine(gpu, dtype, tokens, slots, width):
    gen = torch.Generator().manual_seed(width)
    experts = 6
    route = lx.laplex_route(ids_of(tokens, slots, experts, width, 0.3).to(gpu), experts)
    x = torch.randn(tokens, width, generator=gen).to(dtype)
    xs = lx.laplex_dispatch(route, x.to(gpu)).cpu()
    order = route.order.cpu().long()
    want = torch.where((order >= 0)[:, None], x[order.clamp(min=0) // slots], torch.zeros((), dtype=dtype))
    assert torch.equal(xs, want)

    ys = torch.randn(tokens * slots, width, generator=gen).to(dtype)
    kept = int(route.offsets[-1])
    ys[kept:] = float("nan")  # rows of no slot
    weights = torch.rand(tokens, slots, generator=gen)
    weights[route.place.cpu() < 0] = float("inf")  # weights of dropped slots
    for w in (None, weights):
        y = lx.laplex_combine(route, ys.to(gpu), None if w is None else w.to(gpu))
        ref.assert_within(y, *ref.combine(route.place, ys, w))

    dy = torch.randn(tokens, width, generator=gen).to(dtype)
    dys, dw = lx.laplex_combine_backward(route, dy.to(gpu), ys.to(gpu), weights.to(gpu))
    (rys, eys), (rw, ew) = ref.combine_backward(route.place, dy, torch.nan_to_num(ys), weights)
    ref.assert_within(dys, rys, eys)
    ref.assert_within(dw, rw, ew)


def test_combine_gradient_by_differences(gpu):
    gen = torch.Generator().manual_seed(0)
    route = lx.laplex_route(ids_of(9, 3, 4, 0).to(gpu), 4)
    ys = torch.randn(27, 12, generator=gen).to(gpu)
    w, dy = torch.rand(9, 3, generator=gen).to(gpu), torch.randn(9, 12, generator=gen).to(gpu)
    dys, dw = lx.laplex_combine_backward(route, dy, ys, w)
    loss = lambda ys, w: float((lx.laplex_combine(route, ys, w).double() * dy.double()).sum())  # noqa: E731
    # the map is linear in each input: a unit step is exact up to rounding
    tol = 1e-4
    for i in (0, 5, 13, 26):
        step = torch.zeros_like(ys)
        step[i, i % 12] = 1.0
        assert abs(loss(ys + step, w) - loss(ys, w) - float(dys[i, i % 12])) < tol
    for t, k in ((0, 0), (4, 2), (8, 1)):
        step = torch.zeros_like(w)
        step[t, k] = 1.0
        assert abs(loss(ys, w + step) - loss(ys, w) - float(dw[t, k])) < tol


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,lead", [(0, 0), (3, 1), (8, 8)])
def test_row_pitch_and_alignment(gpu, dtype, pad, lead):
    """Rows inside a wider array, starting anywhere in it."""
    gen = torch.Generator().manual_seed(3)
    tokens, slots, width = 37, 2, 48
    route = lx.laplex_route(ids_of(tokens, slots, 5, 4).to(gpu), 5)
    part = lambda rows: torch.randn(rows, width + pad + lead, generator=gen).to(dtype).to(gpu)[:, lead:lead + width]  # noqa: E731,E501
    x, ys, dy = part(tokens), part(tokens * slots), part(tokens)
    w = torch.rand(tokens, slots, generator=gen).to(gpu)
    assert torch.equal(lx.laplex_dispatch(route, x), lx.laplex_dispatch(route, x.contiguous()))
    assert torch.equal(lx.laplex_combine(route, ys, w), lx.laplex_combine(route, ys.contiguous(), w))
    got = lx.laplex_combine_backward(route, dy, ys, w)
    (rys, eys), (rw, ew) = ref.combine_backward(route.place, dy, ys, w)
    ref.assert_within(got[0], rys, eys)
    ref.assert_within(got[1], rw, ew)


def test_places_outside_the_rows_are_skipped(gpu):
    place = torch.tensor([[0, 99], [-7, 1]], dtype=torch.int32, device=gpu)
    route = lx.Route(torch.zeros(4, dtype=torch.int32, device=gpu), place,
                     torch.tensor([0, 2], dtype=torch.int32, device=gpu))
    x = torch.tensor([[1.0], [2.0]], device=gpu)
    assert lx.laplex_dispatch(route, x).reshape(-1).tolist() == [1.0, 2.0, 0.0, 0.0]
    ys = torch.tensor([[10.0], [20.0], [30.0], [40.0]], device=gpu)
    assert lx.laplex_combine(route, ys).reshape(-1).tolist() == [10.0, 20.0]


def test_rows_past_32_bit_offsets(gpu):
    """Expert rows whose last element is past 2^31 values."""
    tokens, slots, width = 2, 1, 64
    big = torch.empty(2, 2 ** 31 + 64, dtype=torch.bfloat16, device=gpu)
    ys = big[:, :width]
    assert ys.stride(0) > 2 ** 31
    ys.copy_(torch.arange(2 * width, device=gpu).reshape(2, width))
    route = lx.laplex_route(torch.tensor([[1], [0]], device=gpu), 2)
    y = lx.laplex_combine(route, ys)
    assert torch.equal(y, ys.flip(0))
    del big


def test_another_stream(gpu):
    side = torch.cuda.Stream()
    ids = ids_of(50000, 2, 64, 8)
    x = torch.randn(50000, 64).to(gpu)
    want = lx.laplex_route(ids.to(gpu), 64)
    on = ids.to(gpu)
    torch.cuda.synchronize()
    route = lx.laplex_route(on, 64, stream=side)
    xs = lx.laplex_dispatch(route, x, stream=side)
    y = lx.laplex_combine(route, xs, stream=side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(route, want))
    kept = (route.place >= 0).sum(1, keepdim=True)
    assert torch.allclose(y, x * kept)
