"""Decays whose products leave float32's range while the states do not:
growth, and infinities and NaN that only a decay of 0 forgets."""
import math

import pytest
import torch

import tokens_ref as ref
from laplace_matvec_amd import laplex as lx

pytestmark = pytest.mark.gpu

# (channels, decays) of a call with few tiles, of one with many, of one channel per thread; float32 rows
FORMS = [(64, 64), (64, 8), (5120, 5120), (5120, 80), (66, 22)]
FORMS_IDS = ["few-own", "few-shared", "many-own", "many-shared", "single"]
N = 1100  # five row tiles


def look(width):
    """Channels that are compared: tiles' borders and a few between."""
    return sorted({c % width for c in (0, 1, 2, 63, 64, 65, width // 2, width - 2, width - 1)})


def check(gpu, x, g, dy, offsets, h0=None, dfinal=None):
    """x, dy [n, width], g [n, heads] on the host; all outputs against float64 on some channels."""
    width, heads = x.shape[1], g.shape[1]
    per, cols = width // heads, look(width)
    at = torch.tensor(offsets, dtype=torch.int32, device=gpu)
    to = lambda t: None if t is None else t.to(gpu)  # noqa: E731
    r = lx.laplex_recur(to(x), to(g), offsets=at, h0=to(h0), final=True, keep=True)
    d = lx.laplex_recur_backward(to(x), to(g), to(dy), r.states, offsets=at, h0=to(h0), dfinal=to(dfinal))
    pick = lambda t: None if t is None else t[:, cols]  # noqa: E731
    want = ref.Recur(x[:, cols], g[:, [c // per for c in cols]], offsets, pick(h0), dy[:, cols], pick(dfinal))
    ref.assert_within(r.y[:, cols], want.y, want.ey)
    ref.assert_within(r.final[:, cols], want.final, want.efinal)
    ref.assert_within(d["dx"][:, cols], want.dx, want.edx)
    ref.assert_within(d["dh0"][:, cols], want.dh0, want.edh0)
    # dg of a head: the sum over its channels, here all alike
    ref.assert_within(d["dg"][:, [c // per for c in cols]], want.dg * per, (want.edg + per * ref.U32 * want.dg.abs()) * per)
    return r, d


def alike(n, width):
    """A column for all channels: heads' sums are then known from one of them."""
    return lambda col: col.reshape(n, 1).expand(n, width).contiguous()


@pytest.mark.parametrize("width,heads", FORMS, ids=FORMS_IDS)
def test_growth_from_nothing(gpu, width, heads):
    """e^550 times a state of 0 is 0, both ways."""
    x, g = torch.zeros(N, width), torch.full((N, heads), 0.5)
    r, d = check(gpu, x, g, x, [0, N])
    assert not r.y.any() and not d["dx"].any() and not d["dg"].any() and not d["dh0"].any()


@pytest.mark.parametrize("width,heads", FORMS, ids=FORMS_IDS)
def test_growth_of_small_values(gpu, width, heads):
    """Values from 1e-20 to 1e32 and back; the products within a tile reach e^102 and e^-102."""
    t = torch.arange(N)
    g = torch.where(t % 512 < 256, 0.4, -0.4)
    g[0] = 0.0
    h0 = torch.full((1, width), 1e-20)
    x, dy = torch.zeros(N), torch.zeros(N)
    x[513] = 1e-12
    dy[768:1024] = 1e-25  # no gradient is subnormal: its products with states of 1e32 would not be within the bounds
    dy[700], dy[N - 1] = 1e-9, 1e-15
    check(gpu, alike(N, width)(x), alike(N, heads)(g), alike(N, width)(dy), [0, N], h0, torch.full((1, width), 1e-16))


@pytest.mark.parametrize("width,heads", FORMS, ids=FORMS_IDS)
@pytest.mark.parametrize("rate", [5.0, 7.0, 12.0])
@pytest.mark.parametrize("large", ["states", "gradients"])
def test_decay_of_large_values(gpu, width, heads, rate, large):
    """Values of 1e35 that fall by e^-rate a row: the product of 16 such rows is no float32, its effect is."""
    n = 600
    some, other = torch.zeros(n), torch.full((n,), 1e-2 if large == "states" else 1.0)
    some[[0, 14, 15, 30, 31, 250, 255, 256, 300, 511]] = 1e35
    edge, far = torch.full((1, width), 3e37), torch.full((1, width), 1.0)
    some, other = alike(n, width)(some), alike(n, width)(other)
    g = alike(n, heads)(torch.full((n,), -rate))
    if large == "states":
        check(gpu, some, g, other, [0, n], edge, far)
    else:
        check(gpu, other, g, some, [0, n], far, edge)


@pytest.mark.parametrize("width,heads", FORMS, ids=FORMS_IDS)
def test_up_and_down_within_a_few_rows(gpu, width, heads):
    """Single decays up to e^95 and down to e^-100, neither a normal float32, between values of 1e-35 and 1e29."""
    n = 300
    g = torch.tensor([0.0, 80.0, -80.0, -40.0, 40.0, -45.0, 95.0, -100.0, 30.0, 20.0]).repeat(n // 10)  # 0 in all
    x, dy = torch.zeros(n), torch.zeros(n)
    x[0::10], x[3::10], x[5::10] = 1e-10, 1e-26, 1e-27
    dy[1::10], dy[2::10], dy[9::10] = 1e-30, 1.0, 1e-9
    check(gpu, alike(n, width)(x), alike(n, heads)(g), alike(n, width)(dy), [0, n], torch.full((1, width), 1e-12), None)


def scan64(x, g, offsets, reverse=False, first=None):
    """The float64 definition on one column: states, or (reverse) gradients of x."""
    out = torch.zeros_like(x, dtype=torch.float64)
    for q in range(len(offsets) - 1):
        rows = range(offsets[q], offsets[q + 1])
        h = 0.0
        for t in reversed(rows) if reverse else rows:
            if reverse:
                out[t] = h + float(x[t])
                h = 0.0 if g[t] < -104 else math.exp(g[t]) * float(out[t])
            else:
                h = float(x[t]) + (0.0 if g[t] < -104 or t == rows[0] else math.exp(g[t]) * h)
                out[t] = h
    return out


@pytest.mark.parametrize("width,heads", FORMS, ids=FORMS_IDS)
@pytest.mark.parametrize("rate", [0.1, 1.0, 7.0, 60.0])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_only_a_decay_of_zero_forgets(gpu, width, heads, rate, value):
    """One value that is not finite stays to the end of its sequence or the next reset, however its decays multiply."""
    offsets = [0, 900, N]
    x, dy, g = torch.ones(N), torch.ones(N), torch.full((N,), -rate)
    x[3], dy[880] = value, value
    x[901], dy[N - 7] = value, value
    g[950] = -math.inf
    at = torch.tensor(offsets, dtype=torch.int32, device=gpu)
    xs, gs, dys = (alike(N, k)(t).to(gpu) for t, k in ((x, width), (g, heads), (dy, width)))
    r = lx.laplex_recur(xs, gs, offsets=at, final=True, keep=True)
    d = lx.laplex_recur_backward(xs, gs, dys, r.states, offsets=at)
    for got, want in ((r.y, scan64(x, g, offsets)), (d["dx"], scan64(dy, g, offsets, True))):
        want = want.float().to(gpu)[:, None].expand(N, width)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.isinf(got) & (got > 0), torch.isinf(want) & (want > 0))
        assert torch.equal(torch.isinf(got) & (got < 0), torch.isinf(want) & (want < 0))
    assert not torch.isfinite(r.final[0]).any() and torch.isfinite(r.final[1]).all()
    assert not torch.isfinite(d["dh0"][0]).any() and torch.isfinite(d["dh0"][1]).all()


@pytest.mark.parametrize("width,heads", FORMS, ids=FORMS_IDS)
def test_a_decay_of_nan_shows(gpu, width, heads):
    """Also where the state is 0: NaN until the next reset or the sequence's end, both ways."""
    x, g = torch.zeros(N, width, device=gpu), torch.full((N, heads), -6.0, device=gpu)
    g[[5, 700]] = math.nan
    g[[900, 300]] = -math.inf
    at = torch.tensor([0, 500, N], dtype=torch.int32, device=gpu)
    r = lx.laplex_recur(x, g, offsets=at, keep=True)
    d = lx.laplex_recur_backward(x, g, x, r.states, offsets=at)
    t = torch.arange(N, device=gpu)
    want = ((t >= 5) & (t < 300)) | ((t >= 700) & (t < 900))
    back = (t < 5) | ((t >= 500) & (t < 700))
    assert torch.equal(torch.isnan(r.y), want[:, None].expand(N, width))
    assert torch.equal(torch.isnan(d["dx"]), back[:, None].expand(N, width))


def test_step_past_the_range_of_a_decay(gpu):
    state = torch.tensor([[0.0, 1e-20, 1e-44, math.inf], [0.0, 1e-20, 3e38, 1.0]], device=gpu)
    g = torch.tensor([[100.0] * 4, [100.0, 95.0, -200.0, -103.0]], device=gpu)
    x = torch.tensor([[2.0, 0.0, 0.0, 0.0], [0.0, 0.0, 1.0, 0.0]], device=gpu)
    y = lx.laplex_recur_step(x, g, state)
    want = torch.tensor([[2.0, 2.6881171e23, 0.26881171, math.inf], [0.0, 1.811239e21, 1.0, math.exp(-103.0)]])
    # 1e-44 is 7 * 2^-149; e^-103 is a few of the smallest float32
    want[0, 2] = 7 * 2.0 ** -149 * math.exp(100.0)
    assert y[0, 3] == math.inf
    err = (y.cpu().double() - want.double()).abs()
    err[0, 3] = 0
    # the exponent's rounding, 100 u, the exponential's ulp and two roundings
    assert (err <= 256 * 2.0 ** -24 * want.double().abs().clamp(max=1e38) + 2.0 ** -149).all()
    assert torch.equal(y, state)
