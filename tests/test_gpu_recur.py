"""The gated recurrence, its gradients and its single-token form against
plain float64."""
import math

import pytest
import torch

import tokens_ref as ref
from laplace_matvec_amd import laplex as lx

pytestmark = pytest.mark.gpu

COMBOS = [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
          (torch.float16, torch.float16), (torch.float16, torch.float32)]


def inputs(n, width, heads, types, seed, resets=0.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(n, width, generator=gen).to(types[0])
    g = -torch.exp(torch.randn(n, heads, generator=gen) * 2 - 3)
    if resets:
        g[torch.rand(n, heads, generator=gen) < resets] = -math.inf
    dy = torch.randn(n, width, generator=gen).to(types[0])
    return x, g.to(types[1]), dy, gen


def check(gpu, x, g, dy, offsets, h0, dfinal, packed=True):
    seqs, width = len(offsets) - 1, x.shape[-1]
    at = torch.tensor(offsets, dtype=torch.int32, device=gpu) if packed else None
    to = lambda t: None if t is None else t.to(gpu)  # noqa: E731
    r = lx.laplex_recur(to(x), to(g), offsets=at, h0=to(h0), final=True, keep=True)
    got = lx.laplex_recur_backward(to(x), to(g), to(dy), r.states, offsets=at, h0=to(h0), dfinal=to(dfinal))
    want = ref.Recur(x, g, offsets, h0, dy, dfinal)
    ref.assert_within(r.y.reshape(-1, width), want.y, want.ey)
    ref.assert_within(r.final, want.final, want.efinal)
    ref.assert_within(got["dx"].reshape(-1, width), want.dx, want.edx)
    ref.assert_within(got["dg"].reshape(-1, g.shape[-1]), want.dg, want.edg)
    ref.assert_within(got["dh0"], want.dh0, want.edh0)
    assert r.final.shape == got["dh0"].shape == (seqs, width)
    return r, got


@pytest.mark.parametrize("types", COMBOS)
@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 300, 1025])
@pytest.mark.parametrize("width,heads", [(1, 1), (8, 8), (64, 4), (72, 72), (100, 5)])
def test_one_sequence(gpu, types, n, width, heads):
    x, g, dy, gen = inputs(n, width, heads, types, n + width)
    h0, df = torch.randn(1, width, generator=gen), torch.randn(1, width, generator=gen)
    check(gpu, x, g, dy, [0, n], h0, df, packed=False)


# decays within a channel tile, across its borders, over several tiles
@pytest.mark.parametrize("types", COMBOS[:3])
@pytest.mark.parametrize("width,heads", [(192, 3), (192, 4), (256, 2), (260, 2), (300, 1), (65, 1), (66, 22), (130, 26),
                                         (320, 4), (512, 2), (64, 64), (63, 3)])
def test_head_layouts(gpu, types, width, heads):
    x, g, dy, gen = inputs(200, width, heads, types, width)
    check(gpu, x, g, dy, [0, 90, 200], torch.randn(2, width, generator=gen), torch.randn(2, width, generator=gen))


@pytest.mark.parametrize("types", COMBOS[:3])
@pytest.mark.parametrize("width", [2, 3, 4, 5, 7, 61, 65, 66, 67, 129, 191])
def test_widths_that_four_does_not_divide(gpu, types, width):
    """A decay per channel; the last group of four of a row starts before where it would."""
    x, g, dy, gen = inputs(290, width, width, types, width, resets=0.01)
    check(gpu, x, g, dy, [0, 100, 290], torch.randn(2, width, generator=gen), torch.randn(2, width, generator=gen))


def test_odd_width_over_many_tiles(gpu):
    """More tiles than the few that take the short form, odd rows, twice the same."""
    n, width = 4200, 1027
    gen = torch.Generator(device=gpu).manual_seed(5)
    x = torch.randn(n, width, device=gpu, generator=gen).to(torch.bfloat16)
    g = -torch.rand(n, width, device=gpu, generator=gen)
    dy = torch.randn(n, width, device=gpu, generator=gen).to(torch.bfloat16)
    r = lx.laplex_recur(x, g, final=True, keep=True)
    d = lx.laplex_recur_backward(x, g, dy, r.states)
    again = lx.laplex_recur(x, g, final=True, keep=True)
    assert torch.equal(r.y, again.y) and torch.equal(r.final, again.final)
    cols = [0, 63, 64, 1022, 1023, 1024, 1025, 1026]
    want = ref.Recur(x[-600:, cols], g[-600:, cols], [0, 600], None, dy[-600:, cols])  # 0.5 a row
    ref.assert_within(r.y[-300:, cols], want.y[-300:], want.ey[-300:])
    ref.assert_within(d["dx"][-600:, cols], want.dx, want.edx)
    ref.assert_within(d["dg"][-300:, cols], want.dg[-300:], want.edg[-300:])


@pytest.mark.parametrize("types", COMBOS[1:3])
@pytest.mark.parametrize("offsets", [
    [0, 0, 1, 2, 2, 2, 60, 128, 128, 256, 257, 700, 700],  # empty ones, borders of tiles
    [0] + list(range(1, 300)) + [300] * 90 + [640],         # single rows, many empty ones
    [5, 40, 200, 333],                                      # rows of no sequence at both ends
    [130, 130, 131],                                        # tiles without a sequence
    [0, 1000],
])
@pytest.mark.parametrize("states", [False, True])
def test_packed(gpu, types, offsets, states):
    n = max(640, offsets[-1]) + (7 if offsets[0] else 0)
    x, g, dy, gen = inputs(n, 68, 17, types, len(offsets), resets=0.01)
    offsets = offsets if offsets[0] or offsets[-1] == n else offsets[:-1] + [n]
    seqs = len(offsets) - 1
    h0 = torch.randn(seqs, 68, generator=gen) if states else None
    df = torch.randn(seqs, 68, generator=gen) if states else None
    # rows of no sequence are not looked at
    for t in (x, g, dy):
        t[:offsets[0]] = float("nan")
        t[offsets[-1]:] = float("nan")
    clean = [torch.nan_to_num(t) if offsets[0] else t for t in (x, g, dy)]
    at = torch.tensor(offsets, dtype=torch.int32, device=gpu)
    to = lambda t: None if t is None else t.to(gpu)  # noqa: E731
    r = lx.laplex_recur(to(x), to(g), offsets=at, h0=to(h0), final=True, keep=True)
    got = lx.laplex_recur_backward(to(x), to(g), to(dy), r.states, offsets=at, h0=to(h0), dfinal=to(df))
    want = ref.Recur(clean[0], clean[1], offsets, h0, clean[2], df)
    ref.assert_within(r.y, want.y, want.ey)
    ref.assert_within(r.final, want.final, want.efinal)
    ref.assert_within(got["dx"], want.dx, want.edx)
    ref.assert_within(got["dg"], want.dg, want.edg)
    ref.assert_within(got["dh0"], want.dh0, want.edh0)


@pytest.mark.parametrize("seqs,length", [(1, 257), (3, 1), (5, 64), (2, 128), (7, 129), (40, 3)])
def test_equal_sequences(gpu, seqs, length):
    types = COMBOS[2]
    x, g, dy, gen = inputs(seqs * length, 96, 12, types, length)
    h0, df = torch.randn(seqs, 96, generator=gen), torch.randn(seqs, 96, generator=gen)
    split = lambda t: t.unflatten(0, (seqs, length))  # noqa: E731
    check(gpu, split(x), split(g), split(dy), [q * length for q in range(seqs + 1)], h0, df, packed=False)


def test_no_rows(gpu):
    x, g = torch.empty(0, 8, device=gpu), torch.empty(0, 2, device=gpu)
    h0 = torch.randn(3, 8, device=gpu)
    at = torch.zeros(4, dtype=torch.int32, device=gpu)
    r = lx.laplex_recur(x, g, offsets=at, h0=h0, final=True, keep=True)
    assert r.y.shape == (0, 8) and torch.equal(r.final, h0)
    d = lx.laplex_recur_backward(x, g, x, r.states, offsets=at, h0=h0, dfinal=h0)
    assert torch.equal(d["dh0"], h0) and d["dx"].shape == (0, 8) and d["dg"].shape == (0, 2)
    r = lx.laplex_recur(x.view(3, 0, 8), g.view(3, 0, 2), final=True)
    assert torch.equal(r.final, torch.zeros_like(h0))


@pytest.mark.parametrize("at", [0, 1, 126, 127, 128, 200])
def test_a_decay_of_zero_forgets_inf_and_nan(gpu, at):
    """What comes before a reset leaves no trace after it, and its gradient none before."""
    x, g, dy, gen = inputs(300, 64, 8, COMBOS[0], at)
    g[at] = -math.inf
    bad = x.clone()
    bad[:at] = torch.tensor([math.inf, math.nan, -math.inf, 1.0]).repeat(16)
    run = lambda v: lx.laplex_recur(v.to(gpu), g.to(gpu), h0=torch.full((1, 64), math.nan, device=gpu), keep=True)  # noqa: E731,E501
    r = run(bad)
    want = ref.Recur(x[at:], g[at:], [0, 300 - at])
    ref.assert_within(r.y[at:], want.y, want.ey)
    bad_dy = dy.clone()
    bad_dy[at:] = math.nan
    r = lx.laplex_recur(x.to(gpu), g.to(gpu), keep=True)
    d = lx.laplex_recur_backward(x.to(gpu), g.to(gpu), bad_dy.to(gpu), r.states)
    want = ref.Recur(x[:at], g[:at], [0, at], None, dy[:at])
    ref.assert_within(d["dx"][:at], want.dx, want.edx)
    ref.assert_within(d["dg"][:at], want.dg, want.edg)
    assert (d["dg"][at] == 0).all()


@pytest.mark.parametrize("at", [3, 150, 255])
def test_a_reset_after_an_infinite_decay(gpu, at):
    """exp(g) overflows at one row and is 0 at the next: what follows is finite."""
    x, g, dy, _ = inputs(300, 64, 8, COMBOS[0], at)
    g[at], g[at + 1] = 200.0, -math.inf
    r = lx.laplex_recur(x.to(gpu), g.to(gpu), keep=True)
    want = ref.Recur(x[at + 1:], g[at + 1:], [0, 299 - at], None, dy[at + 1:])
    ref.assert_within(r.y[at + 1:], want.y, want.ey)
    d = lx.laplex_recur_backward(x.to(gpu), g.to(gpu), dy.to(gpu), r.states)
    ref.assert_within(d["dx"][at + 1:], want.dx, want.edx)
    assert torch.isfinite(d["dg"][at + 2:]).all() and (d["dg"][at + 1] == 0).all()


def test_sequences_do_not_leak(gpu):
    """inf and NaN in one sequence stay there, both ways."""
    x, g, dy, _ = inputs(400, 64, 64, COMBOS[0], 9)
    offsets = [0, 150, 250, 400]
    bad, bad_dy = x.clone(), dy.clone()
    bad[150:250], bad_dy[150:250] = math.nan, math.inf
    at = torch.tensor(offsets, dtype=torch.int32, device=gpu)
    r = lx.laplex_recur(bad.to(gpu), g.to(gpu), offsets=at, keep=True)
    d = lx.laplex_recur_backward(bad.to(gpu), g.to(gpu), bad_dy.to(gpu), r.states, offsets=at)
    want = ref.Recur(x, g, offsets, None, dy)
    for rows in (slice(0, 150), slice(250, 400)):
        ref.assert_within(r.y[rows], want.y[rows], want.ey[rows])
        ref.assert_within(d["dx"][rows], want.dx[rows], want.edx[rows])
        ref.assert_within(d["dg"][rows], want.dg[rows], want.edg[rows])


@pytest.mark.parametrize("value", [-1e-30, -1e-4, -87.0, -104.0, -3e38, 0.0, 0.5])
def test_extreme_decays(gpu, value):
    x, _, dy, _ = inputs(40, 16, 4, COMBOS[0], 3)
    g = torch.full((40, 4), value)
    check(gpu, x, g, dy, [0, 40], None, None, packed=False)


@pytest.mark.parametrize("types", COMBOS[:2])
@pytest.mark.parametrize("lead", [0, 1, 4])
def test_parts_of_wider_rows(gpu, types, lead):
    """x, g and dy as parts of one projection's rows, at any offset."""
    n, width = 333, 64
    gen = torch.Generator().manual_seed(lead)
    both = torch.randn(n, 3 * width + lead, generator=gen).to(types[0])
    both[:, lead + width:lead + 2 * width] = -both[:, lead + width:lead + 2 * width].abs()
    dev = both.to(gpu)
    x, g, dy = (dev[:, lead + i * width:lead + (i + 1) * width] for i in range(3))
    r = lx.laplex_recur(x, g, final=True, keep=True)
    d = lx.laplex_recur_backward(x, g, dy, r.states)
    want = ref.Recur(x, g, [0, n], None, dy)
    ref.assert_within(r.y, want.y, want.ey)
    ref.assert_within(d["dx"], want.dx, want.edx)
    ref.assert_within(d["dg"], want.dg, want.edg)
    ref.assert_within(r.final, want.final, want.efinal)


def test_gradient_by_differences(gpu):
    n, width, heads = 150, 8, 2
    x, g, dy, gen = inputs(n, width, heads, COMBOS[0], 5)
    h0, df = torch.randn(2, width, generator=gen), torch.randn(2, width, generator=gen)
    at = torch.tensor([0, 70, n], dtype=torch.int32, device=gpu)
    x, g, dy, h0, df = (t.to(gpu) for t in (x, g, dy, h0, df))
    r = lx.laplex_recur(x, g, offsets=at, h0=h0, keep=True)
    d = lx.laplex_recur_backward(x, g, dy, r.states, offsets=at, h0=h0, dfinal=df)

    def loss(x, g, h0):
        r = lx.laplex_recur(x, g, offsets=at, h0=h0, final=True)
        return float((r.y.double() * dy.double()).sum() + (r.final.double() * df.double()).sum())

    for t, row, col in ((x, 0, 1), (x, 69, 3), (x, 70, 0), (x, 149, 7), (g, 0, 0), (g, 69, 1), (g, 70, 0), (g, 149, 1),
                        (h0, 0, 2), (h0, 1, 5)):
        name, eps = ("dx", 0.5) if t is x else ("dg", 0.01) if t is g else ("dh0", 0.5)
        up, down = t.clone(), t.clone()
        up[row, col] += eps
        down[row, col] -= eps
        of = lambda v: loss(v if t is x else x, v if t is g else g, v if t is h0 else h0)  # noqa: E731
        num = (of(up) - of(down)) / (2 * eps)
        # x and h0 enter linearly; g's central difference is off by eps^2 / 6 = 2e-5 of terms no
        # larger than the loss's.  The loss sums 1200 float32 outputs below 10, each off by some
        # 6e-8 of itself with either sign: 35 * 6e-7 = 2e-5, divided by 2 eps.
        assert abs(num - float(d[name][row, col])) < 5e-3 + 1e-4 * abs(num)


def test_gradients_wanted_in_part(gpu):
    x, g, dy, _ = inputs(300, 128, 1, COMBOS[0], 6)
    x, g, dy = x.to(gpu), g.to(gpu), dy.to(gpu)
    r = lx.laplex_recur(x, g, keep=True)
    every = lx.laplex_recur_backward(x, g, dy, r.states)
    assert set(every) == {"dx", "dg", "dh0"}
    for name in every:
        one = lx.laplex_recur_backward(x, g, dy, r.states, want=(name,))
        assert set(one) == {name} and torch.equal(one[name], every[name])


def test_long_rows_repeat_bit_for_bit(gpu):
    """Many tiles in flight: the same bits every time, and the float64 scan's values at the end."""
    gen = torch.Generator(device=gpu).manual_seed(1)
    n, width = 20000, 1024
    x = torch.randn(n, width, device=gpu, generator=gen).to(torch.bfloat16)
    g = (-torch.rand(n, width, device=gpu, generator=gen) * 0.02).to(torch.bfloat16)
    dy = torch.randn(n, width, device=gpu, generator=gen).to(torch.bfloat16)
    first = lx.laplex_recur(x, g, final=True, keep=True)
    d0 = lx.laplex_recur_backward(x, g, dy, first.states)
    for _ in range(4):
        r = lx.laplex_recur(x, g, final=True, keep=True)
        assert all(torch.equal(a, b) for a, b in zip(r, first))
        d1 = lx.laplex_recur_backward(x, g, dy, r.states)
        assert all(torch.equal(d1[k], d0[k]) for k in d0)
    cols = [0, 63, 64, 500, 1023]
    want = ref.Recur(x[-6000:, cols], g[-6000:, cols], [0, 6000])  # 0.01 a row: nothing older is left
    ref.assert_within(first.y[-1000:, cols], want.y[-1000:], want.ey[-1000:])
    ref.assert_within(first.final[0, cols], want.final[0], want.efinal[0])
    want = ref.Recur(x[:6000, cols], g[:6000, cols], [0, 6000], None, dy[:6000, cols])
    ref.assert_within(d0["dx"][:1000, cols], want.dx[:1000], want.edx[:1000])
    ref.assert_within(d0["dg"][:1000, cols], want.dg[:1000], want.edg[:1000])


@pytest.mark.parametrize("seqs", [1, 7])
def test_one_narrow_chain(gpu, seqs):
    """400 tiles that all hang on the ones before them, next to another such pass on a second stream."""
    gen = torch.Generator(device=gpu).manual_seed(seqs)
    n, width = 102400, 64
    x = torch.randn(n, width, device=gpu, generator=gen)
    g = -torch.rand(n, 1, device=gpu, generator=gen) - 0.1
    dy = torch.randn(n, width, device=gpu, generator=gen)
    at = torch.linspace(0, n, seqs + 1, device=gpu).to(torch.int32)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    both = []
    for stream in (None, side):
        r = lx.laplex_recur(x, g, offsets=at, final=True, keep=True, stream=stream)
        both.append((r, lx.laplex_recur_backward(x, g, dy, r.states, offsets=at, stream=stream)))
    torch.cuda.synchronize()
    (r, d), (r2, d2) = both
    assert torch.equal(r.y, r2.y) and all(torch.equal(d[k], d2[k]) for k in d)
    first = int(at[-2])
    m = min(500, n - first)  # 0.6 a row: nothing older is left after 200
    want = ref.Recur(x[-m:], g[-m:], [0, m], None, dy[-m:])
    ref.assert_within(r.y[-300:], want.y[-300:], want.ey[-300:])
    ref.assert_within(d["dx"][-m:], want.dx, want.edx)
    ref.assert_within(d["dg"][-300:], want.dg[-300:], want.edg[-300:])
    want = ref.Recur(x[:500], g[:500], [0, 500], None, dy[:500])
    ref.assert_within(r.y[:500], want.y, want.ey)
    ref.assert_within(d["dx"][:300], want.dx[:300], want.edx[:300])
    ref.assert_within(d["dg"][:300], want.dg[:300], want.edg[:300])


def test_rows_past_32_bit_offsets(gpu):
    """Rows far apart: the last ones are past 2^32 bytes and 2^31 values."""
    n, pitch, width = 140, 1 << 24, 64
    big = torch.empty(n, pitch, dtype=torch.bfloat16, device=gpu)
    x, g, _, _ = inputs(n, width, width, COMBOS[1], 2)
    xs, gs = big[:, :width], big[:, 4096:4096 + width]
    xs.copy_(x)
    gs.copy_(g)
    r = lx.laplex_recur(xs, gs)
    del big
    want = ref.Recur(x, g, [0, n])
    ref.assert_within(r.y, want.y, want.ey)


def test_graph_replays(gpu):
    n, width = 700, 256
    x, g, dy, _ = inputs(n, width, 4, COMBOS[2], 4)
    x, g, dy = x.to(gpu), g.to(gpu), dy.to(gpu)
    at = torch.tensor([0, 300, 700], dtype=torch.int32, device=gpu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        r = lx.laplex_recur(x, g, offsets=at, final=True, keep=True)
        d = lx.laplex_recur_backward(x, g, dy, r.states, offsets=at)
        return [r.y, r.final, d["dx"], d["dg"], d["dh0"]]

    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(torch.randn(n, width))
        eager = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), k


def test_another_stream(gpu):
    x, g, dy, _ = inputs(5000, 256, 256, COMBOS[1], 7)
    x, g, dy = x.to(gpu), g.to(gpu), dy.to(gpu)
    want = lx.laplex_recur(x, g, final=True, keep=True)
    dwant = lx.laplex_recur_backward(x, g, dy, want.states)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        r = lx.laplex_recur(x, g, final=True, keep=True, stream=stream)
        d = lx.laplex_recur_backward(x, g, dy, r.states, stream=stream)
        side.synchronize()
        assert torch.equal(r.y, want.y) and torch.equal(r.final, want.final)
        assert all(torch.equal(d[k], dwant[k]) for k in d)


@pytest.mark.parametrize("types", COMBOS)
@pytest.mark.parametrize("n,width,heads", [(1, 1, 1), (5, 64, 4), (7, 63, 9), (33, 128, 128), (3, 1002, 501),
                                           (300, 96, 2)])
def test_step(gpu, types, n, width, heads):
    x, g, _, gen = inputs(n, width, heads, types, n, resets=0.05)
    pool = n + 5
    state = torch.randn(pool, width, generator=gen)
    slots = torch.randperm(pool, generator=gen)[:n].to(torch.int32)
    if n > 3:
        slots[1], slots[3] = -1, pool  # requests without a state
    dev = state.to(gpu)
    y = lx.laplex_recur_step(x.to(gpu), g.to(gpu), dev, slots=slots.to(gpu))
    after = ref.d(state)
    for i in range(n):
        q = int(slots[i])
        if not 0 <= q < pool:
            assert (y[i] == 0).all()
            continue
        want = ref.Recur(x[i:i + 1], g[i:i + 1], [0, 1], state[q:q + 1])
        ref.assert_within(y[i:i + 1], want.y, want.ey)
        ref.assert_within(dev[q:q + 1], want.final, want.efinal)
        after[q] = ref.d(dev[q])
    assert torch.equal(ref.d(dev), after)  # no other state is touched


def test_steps_go_on_where_the_sequence_ended(gpu):
    x, g, _, _ = inputs(200, 64, 8, COMBOS[0], 8)
    x, g = x.to(gpu), g.to(gpu)
    r = lx.laplex_recur(x[:190], g[:190], final=True)
    state = r.final
    for t in range(190, 200):
        y = lx.laplex_recur_step(x[t:t + 1], g[t:t + 1], state)
    want = ref.Recur(x, g, [0, 200])
    ref.assert_within(y, want.y[-1:], want.ey[-1:])
    ref.assert_within(state, want.final, want.efinal)


def test_step_drops_a_forgotten_state(gpu):
    state = torch.full((2, 4), math.nan, device=gpu)
    x = torch.ones(2, 4, device=gpu)
    g = torch.full((2, 1), -math.inf, device=gpu)
    y = lx.laplex_recur_step(x, g, state)
    assert torch.equal(y, x) and torch.equal(state, x)
