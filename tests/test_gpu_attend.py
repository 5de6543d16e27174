"""The gated matrix memory against float64, at the sizes, layouts and decays where it can go wrong."""
import math

import pytest
import torch

import more_tokens_ref as ref
from laplace_matvec_amd import laplex as lx
from tokens_ref import assert_within

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
ALL = ("dq", "dk", "dv", "dg", "dh0")


def make(gpu, dtype, n, heads, dk, dv, shared=None, gates=None, seqs=1, seed=0, strong=False):
    """Inputs of one pass: q, k, v, g, h0, dy, dfinal."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    hq, hk, hv = shared or (heads, heads, heads)
    g = -torch.rand(n, heads, generator=gen) * torch.logspace(-3, 1.5 if strong else 0, heads)
    put = lambda t, kind=dtype: t.to(kind).to(gpu)  # noqa: E731
    return dict(q=put(rand(n, hq, dk)), k=put(rand(n, hk, dk)), v=put(rand(n, hv, dv)),
                g=put(g, gates or torch.float32), h0=put(rand(seqs, heads, dk, dv), torch.float32),
                dy=put(rand(n, heads, dv)), dfinal=put(rand(seqs, heads, dk, dv), torch.float32))


def passes(t, offsets, gpu, scale, h0=True, dfinal=True, want=ALL):
    at = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=gpu)
    first = t["h0"] if h0 else None
    args = (t["q"], t["k"], t["v"], t["g"])
    r = lx.laplex_attend(*args, offsets=at, h0=first, scale=scale, final=True, keep=True)
    d = lx.laplex_attend_backward(*args, t["dy"], r.states, offsets=at, h0=first, scale=scale,
                                  dfinal=t["dfinal"] if dfinal else None, want=want)
    return {"y": r.y, "final": r.final, **d}


def check(t, offsets, gpu, scale=None, h0=True, dfinal=True):
    scale = t["q"].shape[-1] ** -0.5 if scale is None else scale
    got = passes(t, offsets, gpu, scale, h0, dfinal)
    want = ref.attend(t["q"], t["k"], t["v"], t["g"], offsets or [0, t["g"].shape[0]], t["h0"] if h0 else None, scale,
                      t["dy"], t["dfinal"] if dfinal else None)
    for name, (value, bound) in want.items():
        try:
            assert_within(got[name], value, bound)
        except AssertionError as e:
            raise AssertionError(f"{name}: {e}") from e


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 128, 200])
def test_lengths(gpu, dtype, n):
    check(make(gpu, dtype, n, 2, 64, 64, seed=n), None, gpu)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [513, 700, 1100])
def test_several_segments(gpu, dtype, n):
    check(make(gpu, dtype, n, 1, 32, 48, seed=n), None, gpu)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv", [(1, 1), (7, 33), (33, 7), (64, 128), (128, 64), (128, 128), (40, 40), (72, 65),
                                   (130, 20), (200, 130), (256, 96)])
def test_widths(gpu, dtype, dk, dv):
    check(make(gpu, dtype, 150, 2, dk, dv, seed=dk + dv), None, gpu)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,shared", [(6, (2, 3, 6)), (4, (1, 1, 1)), (4, (4, 2, 1)), (6, (2, 2, 6)), (6, (6, 6, 2)),
                                          (3, (1, 1, 3))])
def test_shared_heads(gpu, dtype, heads, shared):
    check(make(gpu, dtype, 140, heads, 40, 24, shared, seed=heads), None, gpu)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_shared_heads_of_several_blocks(gpu, dtype):
    check(make(gpu, dtype, 100, 4, 150, 70, (2, 2, 1)), None, gpu)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offsets", [[0, 1, 1, 40, 200, 200], [5, 70, 134, 135, 190], [0, 64, 128, 200], [199, 200],
                                     [100, 100, 100]])
def test_packed(gpu, dtype, offsets):
    """Empty sequences, and rows of no sequence before and past them."""
    check(make(gpu, dtype, 200, 2, 40, 72, seqs=len(offsets) - 1, seed=len(offsets)), offsets, gpu)


def test_packed_of_several_segments(gpu):
    offsets = [3, 600, 600, 1300, 1310, 1900]
    check(make(gpu, torch.bfloat16, 2000, 1, 24, 16, seqs=5), offsets, gpu)


@pytest.mark.parametrize("dtype", TYPES)
def test_equal_sequences(gpu, dtype):
    t = make(gpu, dtype, 3 * 90, 2, 24, 40, seqs=3)
    want = passes(t, [0, 90, 180, 270], gpu, 0.3)
    for name in ("q", "k", "v", "g", "dy"):
        t[name] = t[name].unflatten(0, (3, 90))
    got = passes(t, None, gpu, 0.3)
    for name, value in want.items():
        assert torch.equal(got[name].reshape(value.shape), value), name


@pytest.mark.parametrize("dtype", TYPES)
def test_without_edges(gpu, dtype):
    t = make(gpu, dtype, 150, 2, 40, 40)
    check(t, None, gpu, h0=False, dfinal=False)
    check(t, None, gpu, h0=False)
    check(t, None, gpu, dfinal=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("own", [False, True])
def test_resets_and_strong_decays(gpu, dtype, own):
    """Decays of 0 at the ends of chunks, beside each other, at the first and last rows; sums of logarithms in the
    thousands followed by weak decays, where a float32 sum would lose the differences."""
    t = make(gpu, dtype, 330, 3, 48, 40, gates=dtype if own else torch.float32, strong=True)
    for row, head in ((0, 0), (63, 0), (64, 0), (65, 1), (100, 1), (101, 1), (127, 0), (128, 1), (300, 0), (329, 1)):
        t["g"][row, head] = -math.inf
    t["g"][200, 0] = -200.0  # e^g is 0 too
    t["g"][70:110, 2] = -100.0
    t["g"][110:128, 2] = -0.01
    check(t, None, gpu)


def test_all_decays_zero_and_all_one(gpu):
    t = make(gpu, torch.float32, 130, 2, 16, 16)
    t["g"][:, 0], t["g"][:, 1] = -math.inf, 0.0
    check(t, None, gpu)


def test_decays_above_one(gpu):
    t = make(gpu, torch.bfloat16, 130, 2, 16, 16)
    t["g"] = -t["g"] * 0.05
    check(t, None, gpu)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_parts_of_one_projection(gpu, dtype):
    """Rows that are parts of wider ones, from odd values on: the same results, bit for bit."""
    t = make(gpu, dtype, 150, 4, 40, 24, (2, 2, 4))
    want = passes(t, None, gpu, 0.25)
    rows = torch.full((150, 1 + 80 + 80 + 96 + 96 + 2), float("nan"), dtype=dtype, device=gpu)
    at = 1
    for name in ("q", "k", "v", "dy"):
        width = t[name].shape[1] * t[name].shape[2]
        view = rows[:, at:at + width].unflatten(1, t[name].shape[1:])
        view.copy_(t[name])
        t[name] = view
        at += width
    got = passes(t, None, gpu, 0.25)
    for name, value in want.items():
        assert torch.equal(got[name], value), name


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_of_no_sequence_are_not_used(gpu, dtype):
    t = make(gpu, dtype, 260, 2, 24, 24, seqs=3)
    offsets = [70, 100, 100, 170]
    want = passes(t, offsets, gpu, 1.0)
    for name in ("q", "k", "v", "g", "dy"):
        t[name][:70] = float("nan")
        t[name][170:] = float("inf")
    got = passes(t, offsets, gpu, 1.0)
    for name, value in want.items():
        assert torch.equal(got[name], value), name
    for name in ("y", "dq", "dk", "dv", "dg"):
        assert not got[name][:70].any() and not got[name][170:].any(), name


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_a_bad_row_reaches_no_earlier_one(gpu, dtype, bad, name):
    """Not its chunk's earlier rows, no other head or sequence, nothing past a decay of 0."""
    t = make(gpu, dtype, 300, 2, 24, 24, seqs=2)
    offsets = [0, 250, 300]
    t["g"][130, 0] = -math.inf
    at = torch.tensor(offsets, dtype=torch.int32, device=gpu)
    run = lambda: lx.laplex_attend(t["q"], t["k"], t["v"], t["g"], offsets=at, h0=t["h0"], final=True)  # noqa: E731
    y0, f0, _ = run()
    t[name][100, 0, 3] = bad
    y, f, _ = run()
    assert torch.equal(y[:100], y0[:100]) and torch.equal(y[:, 1], y0[:, 1]) and torch.equal(y[130:], y0[130:])
    assert torch.equal(f, f0)
    column = slice(3, 4) if name == "v" else slice(None)
    reached = y[100:101, 0] if name == "q" else y[100:130, 0]
    assert not torch.isfinite(reached[:, column]).any()
    if name == "v":  # other columns stay
        assert torch.equal(y[:, 0, 4:], y0[:, 0, 4:])


@pytest.mark.parametrize("dtype", TYPES)
def test_what_is_forgotten_may_hold_anything(gpu, dtype):
    t = make(gpu, dtype, 100, 2, 24, 24)
    t["g"][0] = -math.inf
    want = passes(t, None, gpu, 1.0)
    t["h0"].fill_(float("inf"))
    got = passes(t, None, gpu, 1.0)
    for name, value in want.items():
        assert torch.equal(got[name], value), name


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [1e-3, 300.0])
def test_small_and_large_rows(gpu, dtype, size):
    """Scores and states outside float16's range, results inside their type's."""
    t = make(gpu, dtype, 130, 2, 40, 40)
    t["k"], t["v"] = (t[name] * size for name in ("k", "v"))
    t["q"] = t["q"] / size
    t["dy"] = t["dy"] / size
    check(t, None, gpu)


def test_wanted_gradients_only(gpu):
    t = make(gpu, torch.bfloat16, 150, 4, 72, 40, (2, 2, 1))
    want = passes(t, None, gpu, 1.0)
    for name in ALL:
        got = passes(t, None, gpu, 1.0, want=(name,))
        assert set(got) == {"y", "final", name} and torch.equal(got[name], want[name])


@pytest.mark.parametrize("dtype", TYPES)
def test_no_rows(gpu, dtype):
    t = make(gpu, dtype, 0, 2, 8, 8, seqs=3)
    got = passes(t, [0, 0, 0, 0], gpu, 1.0)
    assert torch.equal(got["final"], t["h0"]) and torch.equal(got["dh0"], t["dfinal"])
    assert got["y"].shape == (0, 2, 8) and got["dq"].shape == (0, 2, 8)


def test_offsets_out_of_range(gpu):
    t = make(gpu, torch.bfloat16, 200, 2, 24, 24, seqs=2)
    want = passes(t, [0, 100, 200], gpu, 1.0)
    got = passes(t, [-7, 100, 2 ** 31 - 1], gpu, 1.0)
    for name, value in want.items():
        assert torch.equal(got[name], value), name


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "h0"])
def test_gradients_against_differences(gpu, name):
    """L = <y, c> + <final, e> in float32, central differences along a direction: L's own change is known to the
    float64 definition within the bounds of the kernel's outputs; what is left is the difference's third-order term."""
    t = make(gpu, torch.float32, 150, 2, 24, 16)
    scale, step = 0.2, 2.0 ** -6
    u = torch.randn(t[name].shape, generator=torch.Generator().manual_seed(5)).to(gpu)
    grads = passes(t, None, gpu, scale)
    slope = float((grads["d" + name].cpu().double() * u.cpu().double()).sum())
    ends, slack = [], 0.0
    exact = []
    for sign in (1, -1):
        moved = dict(t)
        moved[name] = t[name] + sign * step * u
        got = passes(moved, None, gpu, scale)
        r = ref.attend(moved["q"], moved["k"], moved["v"], moved["g"], [0, 150], moved["h0"], scale)
        total = true = 0.0
        for part, by in (("y", "dy"), ("final", "dfinal")):
            c = t[by].cpu().double()
            total += float((got[part].cpu().double() * c).sum())
            true += float((r[part][0] * c).sum())
            slack += float(((r[part][1] + 2.0 ** -24 * r[part][0].abs()) * c.abs()).sum())
        ends.append(total)
        exact.append(true)
    value, bound = ref.attend(t["q"], t["k"], t["v"], t["g"], [0, 150], t["h0"], scale, t["dy"], t["dfinal"])["d" + name]
    own = float(((bound + 2.0 ** -24 * value.abs()) * u.cpu().double().abs()).sum())
    third = abs((exact[0] - exact[1]) / (2 * step) - float((value * u.cpu().double()).sum()))
    assert abs((ends[0] - ends[1]) / (2 * step) - slope) <= slack / (2 * step) + own + third
    # and the definition's own difference is near its gradient, as far as the step's square goes
    assert third <= 0.02 * float((value.abs() * u.cpu().double().abs()).sum())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,heads,shared,dk,dv", [(1, 1, (1, 1, 1), 1, 1), (5, 4, (2, 1, 4), 64, 64), (3, 2, (2, 2, 1), 40, 7),
                                                  (9, 3, (3, 3, 3), 128, 130), (2, 2, (1, 2, 2), 33, 300)])
def test_step(gpu, dtype, n, heads, shared, dk, dv):
    t = make(gpu, dtype, n, heads, dk, dv, shared, seqs=n + 3)
    slots = [(i * 2 + 1) % (n + 3) for i in range(n)] if n % 2 == 0 or n == 1 else list(range(n + 2, 2, -1))
    if n > 2:
        slots[1], t["g"][2, 0] = -1, -math.inf
        t["h0"][slots[2], 0] = float("inf")
    want_y, want_state = ref.attend_step(t["q"], t["k"], t["v"], t["g"], t["h0"], slots, 0.5)
    state = t["h0"].clone()
    y = lx.laplex_attend_step(t["q"], t["k"], t["v"], t["g"], state, slots=torch.tensor(slots, dtype=torch.int32, device=gpu),
                              scale=0.5)
    assert_within(y, *want_y)
    assert_within(state, *want_state)


@pytest.mark.parametrize("slots", [[-1, 7, 2 ** 31 - 1], [3, -5, 4]])
def test_step_without_state(gpu, slots):
    t = make(gpu, torch.bfloat16, 3, 2, 16, 24, seqs=4)
    state = t["h0"].clone()
    y = lx.laplex_attend_step(t["q"], t["k"], t["v"], t["g"], state,
                              slots=torch.tensor(slots, dtype=torch.int32, device=gpu))
    none = [i for i, s in enumerate(slots) if not 0 <= s < 4]
    assert not y[none].any()
    same = [i for i in range(4) if i not in slots]
    assert torch.equal(state[same], t["h0"][same])


@pytest.mark.parametrize("dtype", TYPES)
def test_steps_continue_a_pass(gpu, dtype):
    """Token by token on the states that a pass left, against the pass over all rows."""
    n, more = 90, 20
    t = make(gpu, dtype, n + more, 2, 48, 40)
    args = [t[name] for name in "qkvg"]
    want = ref.attend(*args, [0, n + more], t["h0"], 0.4)["y"]
    state = lx.laplex_attend(*(a[:n] for a in args), h0=t["h0"], scale=0.4, final=True).final
    for i in range(n, n + more):
        y = lx.laplex_attend_step(*(a[i:i + 1] for a in args), state, scale=0.4)
        assert_within(y, want[0][i:i + 1], want[1][i:i + 1])


def test_repeats_bit_for_bit_and_in_a_graph(gpu):
    t = make(gpu, torch.bfloat16, 1200, 4, 64, 64, (2, 2, 4))
    first = passes(t, None, gpu, 0.125)
    again = passes(t, None, gpu, 0.125)
    for name, value in first.items():
        assert torch.equal(again[name], value), name
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        passes(t, None, gpu, 0.125)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = passes(t, None, gpu, 0.125)
    for _ in range(3):
        t["v"].mul_(-1)
        t["dy"].mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        want = passes(t, None, gpu, 0.125)
        for name, value in want.items():
            assert torch.equal(got[name], value), name


def test_two_graphs_that_share_nothing(gpu):
    """Scratch comes from each graph's own pool: replays in turn keep their results apart."""
    t, s = (make(gpu, torch.bfloat16, 700, 2, 64, 64, seed=i) for i in (0, 1))
    want = [passes(x, None, gpu, 0.125) for x in (t, s)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for x in (t, s):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(passes(x, None, gpu, 0.125))
    for k in (0, 1, 1, 0):
        graphs[k].replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for name, value in a.items():
            assert torch.equal(b[name], value), name


def test_another_stream(gpu):
    t = make(gpu, torch.bfloat16, 300, 2, 64, 64)
    want = passes(t, None, gpu, 1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    args = (t["q"], t["k"], t["v"], t["g"])
    for s in (side, side.cuda_stream):
        r = lx.laplex_attend(*args, h0=t["h0"], final=True, keep=True, stream=s)
        d = lx.laplex_attend_backward(*args, t["dy"], r.states, h0=t["h0"], dfinal=t["dfinal"], stream=s)
        side.synchronize()
        assert torch.equal(r.y, want["y"]) and all(torch.equal(d[name], want[name]) for name in ALL)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv", [(129, 24), (136, 64), (160, 64), (176, 40), (192, 128), (264, 8), (320, 72)])
def test_key_widths_that_end_inside_the_states_blocks(gpu, dtype, dk, dv):
    """States are padded to blocks of 128 keys; gradients of float32 and float16 rows go by blocks of 64."""
    check(make(gpu, dtype, 150, 2, dk, dv, (2, 1, 2), seed=dk), None, gpu)


def test_digits_of_float32_results_of_bfloat16_rows(gpu):
    """The relative L2 norm of the errors, which is that of independent errors and far below their worst case.

    final, dh0: a row's decay is off by at most 2^-23 + 2^-24 (rms below 1e-7); the product with it and its three terms
    by 2.5e-8 rms each (half a step of 2^-24, uniform, mean significand).  Over 300 rows the sums take 6 products for
    each of 5 chunks, of at most 4 additions each, and 5 products with decays: 125 roundings of 2.5e-8 of partial
    results whose squares grow in proportion, sqrt(125 / 2) * 2.5e-8 = 2e-7.  Together 2.3e-7; the bound is twice that.
    Two terms leave 2^-17 of the binade at most, 1.6e-6 to 2.3e-6 rms, and do not pass.
    dg: both states in two terms, 2.3e-6 each, meet in one product: 3.3e-6, and the bound is 1.5 times that.  One term
    (2^-9 and more) does not pass."""
    t = make(gpu, torch.bfloat16, 300, 4, 64, 64)
    got = passes(t, None, gpu, 0.125)
    want = ref.attend(t["q"], t["k"], t["v"], t["g"], [0, 300], t["h0"], 0.125, t["dy"], t["dfinal"])
    off = {name: float((got[name].cpu().double() - want[name][0]).norm() / want[name][0].norm()) for name in got}
    print(off)
    assert off["final"] < 5e-7 and off["dh0"] < 5e-7 and off["dg"] < 5e-6, off


@pytest.mark.parametrize("dtype", TYPES)
def test_a_sequence_in_parts(gpu, dtype):
    """A long sequence part by part, as where scratch is short: last states are the next part's first ones, and the
    gradient of a part's first states is that of the part before's last ones.  Three parts have 7 chunks instead of 5,
    three roundings each: 6 of the 270 and more that the bounds count, 3 in 100."""
    t = make(gpu, dtype, 300, 2, 24, 24)
    want = ref.attend(t["q"], t["k"], t["v"], t["g"], [0, 300], t["h0"], 0.2, t["dy"], t["dfinal"])
    parts, first, passed = [slice(0, 130), slice(130, 131), slice(131, 300)], t["h0"], []
    for at in parts:
        r = lx.laplex_attend(*(t[x][at] for x in "qkvg"), h0=first, scale=0.2, final=True, keep=True)
        passed.append((at, first, r))
        first = r.final
    assert_within(first, want["final"][0], 1.03 * want["final"][1])
    got, last = {"y": torch.cat([r.y for _, _, r in passed])}, t["dfinal"]
    grads = []
    for at, h0, r in reversed(passed):
        d = lx.laplex_attend_backward(*(t[x][at] for x in "qkvg"), t["dy"][at], r.states, h0=h0, scale=0.2, dfinal=last)
        last = d["dh0"]
        grads.insert(0, d)
    got.update({name: torch.cat([d[name] for d in grads]) for name in ("dq", "dk", "dv", "dg")}, dh0=last)
    for name, x in got.items():
        assert_within(x, want[name][0], 1.03 * want[name][1])


@pytest.mark.parametrize("gates", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv,shared", [(128, 128, (3, 3, 3)), (128, 64, (1, 1, 3)), (64, 128, (3, 3, 3)), (64, 64, (3, 3, 1)),
                                          (40, 72, (3, 3, 3)), (101, 100, (3, 1, 3)), (200, 256, (1, 3, 3))])
def test_results_of_bfloat16_rows_are_rounded_once(gpu, gates, dk, dv, shared):
    """y's error against float64 is that of rounding: what enters a product is off by 2^-17 of the binade at most in two
    terms, 2.3e-6 rms for scores and states each, 3.3e-6 together beside 1.7e-3, which adds 2e-6 of it to the norm; the
    bound is one in 1000.  One term of either, 1.6e-3 rms, adds up to 0.4 of it."""
    t = make(gpu, torch.bfloat16, 300, 3, dk, dv, shared, gates=gates, seed=dk)
    scale = dk ** -0.5
    y = lx.laplex_attend(t["q"], t["k"], t["v"], t["g"], h0=t["h0"], scale=scale).y.cpu()
    exact = ref.attend(t["q"], t["k"], t["v"], t["g"], [0, 300], t["h0"], scale)["y"][0]
    own = (exact.bfloat16().double() - exact).norm()
    assert (y.double() - exact).norm() < 1.001 * own


@pytest.mark.parametrize("gates", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv,shared", [(128, 128, (3, 3, 3)), (128, 64, (1, 1, 3)), (64, 128, (3, 3, 3)), (64, 64, (3, 3, 1)),
                                          (40, 72, (3, 3, 3)), (101, 100, (3, 1, 3)), (200, 256, (1, 3, 3))])
def test_gradients_of_bfloat16_rows_are_rounded_once(gpu, gates, dk, dv, shared):
    """dq, dk and dv like y: scores and their gradients in two terms.  dg (float32 gates): states in three terms, to the
    last digits of float32, sums of 64 pairs and of dk + dv products: below the 2.3e-6 / 2 that even one state in two
    terms leaves."""
    t = make(gpu, torch.bfloat16, 300, 3, dk, dv, shared, gates=gates, seed=dk)
    scale = dk ** -0.5
    got = passes(t, None, gpu, scale)
    want = ref.attend(t["q"], t["k"], t["v"], t["g"], [0, 300], t["h0"], scale, t["dy"], t["dfinal"])
    off = {name: float((got[name].cpu().double() - want[name][0]).norm()) for name in ALL}
    print({name: x / float(want[name][0].norm()) for name, x in off.items()})
    for name in ("dq", "dk", "dv") + (("dg",) if gates is torch.bfloat16 else ()):
        exact = want[name][0]
        assert off[name] < 1.001 * float((exact.bfloat16().double() - exact).norm()), name
    if gates is torch.float32:
        assert off["dg"] < 1.0e-6 * float(want["dg"][0].norm())
