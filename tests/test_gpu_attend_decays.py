"""The matrix memory's decays where they leave the ordinary: inf and NaN among them."""
import math

import pytest
import torch

import more_tokens_ref as ref
from laplace_matvec_amd import laplex as lx
from test_gpu_attend import ALL, TYPES, make
from tokens_ref import assert_within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("row,reset", [(100, 110), (64, 127), (0, 63), (126, 127), (10, 100), (100, 128), (10, 300), (0, 549)])
def test_a_bad_decay_reaches_nothing_past_a_decay_of_zero(gpu, dtype, own, bad, row, reset):
    """Segments are 128 rows and chunks 64: the reset is in the same chunk, in the segment's next one, or in a later
    segment.  Rows before the bad one, and the other head and sequence, keep their results and gradients."""
    t = make(gpu, dtype, 600, 2, 24, 24, gates=dtype if own else torch.float32, seqs=2)
    at = torch.tensor([0, 550, 600], dtype=torch.int32, device=gpu)
    t["g"][reset, 0] = -math.inf

    def run():
        args = (t["q"], t["k"], t["v"], t["g"])
        r = lx.laplex_attend(*args, offsets=at, h0=t["h0"], final=True, keep=True)
        return r, lx.laplex_attend_backward(*args, t["dy"], r.states, offsets=at, h0=t["h0"], dfinal=t["dfinal"])

    r0, d0 = run()
    want = ref.attend(t["q"], t["k"], t["v"], t["g"], [0, 550, 600], t["h0"])
    t["g"][row, 0] = bad
    r, d = run()
    assert torch.equal(r.y[:row], r0.y[:row]) and torch.equal(r.y[:, 1], r0.y[:, 1])
    assert_within(r.y[reset:550], want["y"][0][reset:550], want["y"][1][reset:550])
    assert torch.equal(r.y[550:], r0.y[550:])
    assert_within(r.final, *want["final"])
    assert torch.equal(r.final[1], r0.final[1]) and torch.equal(r.final[:, 1], r0.final[:, 1])
    assert not torch.isfinite(r.y[row:reset, 0]).any()
    for name in ALL:
        if name == "dh0":
            assert torch.equal(d[name][1], d0[name][1]) and torch.equal(d[name][0, 1], d0[name][0, 1])
        else:
            assert torch.equal(d[name][550:], d0[name][550:]) and torch.equal(d[name][:, 1], d0[name][:, 1]), name


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_decay_that_itself_is_forgotten_leaves_no_trace(gpu, dtype, bad):
    """Documents packed by decays of 0, one with a bad decay in each of its rows: token by token, and in one pass."""
    t = make(gpu, dtype, 400, 1, 16, 16)
    starts = [0, 70, 128, 200, 333]
    t["g"][starts] = -math.inf
    t["g"][71:128] = bad
    y = lx.laplex_attend(t["q"], t["k"], t["v"], t["g"], h0=t["h0"], final=True)
    state = t["h0"].clone()
    for i in range(400):
        step = lx.laplex_attend_step(*(t[x][i:i + 1] for x in "qkvg"), state)
        assert torch.isfinite(step).all() == torch.isfinite(y.y[i]).all(), i
    assert torch.isfinite(y.y[128:]).all() and torch.isfinite(y.final).all() and torch.isfinite(state).all()


def decayed(name):
    """Logarithms of decays of 300 rows (segments of 128) whose product is e^-96, float32 2.03e-42, the first row
    with one and the first that has seen them all."""
    g = torch.zeros(300, 1)
    if name.startswith("one"):
        row = int(name[3:])
        g[row] = -96.0
        return g, row, row
    if name == "several":
        g[[70, 75, 80]] = -32.0
        return g, 70, 80
    if name == "a chunk":
        g[64:128] = -1.5
        return g, 64, 127
    g[:128] = -0.75
    return g, 0, 127


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("large", ["rows before", "rows past"])
@pytest.mark.parametrize("name", ["one5", "one64", "one127", "one128", "several", "a chunk", "a segment"])
def test_decays_below_the_smallest_normal_number(gpu, dtype, large, name):
    """e^-96 of values of 1e36 is about 1e-6, not 0, in what has passed through the decays: results of the rows past them,
    or gradients of the rows before them.

    Slack beside the usual bounds: a decay below 2^-126 is a float32 multiple of 2^-149, so each of the factors that
    make one (two and one for each of 5 chunks, and the product with scale = 1/4) adds at most 2^-150, with the scale
    taken out four times as much: 8 * 5 * 2^-150 < 2^-144 for each pair of rows.  Only what is large all the way is
    compared: where the row that such a decay is multiplied with is of ordinary size, their product (and the state that
    it goes into) is itself below 2^-126, where bfloat16 has no digits left (2^-133 is its smallest number, the product
    about 2^-138)."""
    g, first, past = decayed(name)
    t = make(gpu, dtype, 300, 1, 16, 16, seed=past)
    t["g"] = g.to(gpu)
    rows = torch.arange(300, device=gpu).view(-1, 1, 1)
    big = 1.0 if dtype is torch.float16 else 1e17  # float16 rows stay small beside large first or last states
    before, after = (big, 1.0) if large == "rows before" else (1.0, big)
    t["k"], t["v"] = (torch.where(rows < first, before * t[x].float(), 0.0).to(dtype) for x in "kv")
    t["q"], t["dy"] = (torch.where(rows < past, 0.0, after * t[x].float()).to(dtype) for x in ("q", "dy"))
    edge = "h0" if large == "rows before" else "dfinal"
    t[edge] = t[edge] * (1e36 if dtype is torch.float16 else 1e35)
    scale = 0.25
    want = ref.attend(t["q"], t["k"], t["v"], t["g"], [0, 300], t["h0"], scale, t["dy"], t["dfinal"])
    size = ref._attend(*(ref.d(t[x]).abs() for x in "qkv"), torch.zeros(300, 1, dtype=torch.float64), [0, 300],
                       ref.d(t["h0"]).abs(), scale, ref.d(t["dy"]).abs(), ref.d(t["dfinal"]).abs(), False)
    r = lx.laplex_attend(t["q"], t["k"], t["v"], t["g"], h0=t["h0"], scale=scale, final=True, keep=True)
    got = lx.laplex_attend_backward(t["q"], t["k"], t["v"], t["g"], t["dy"], r.states, h0=t["h0"], scale=scale,
                                    dfinal=t["dfinal"])
    got.update(y=r.y, final=r.final)
    assert all(torch.isfinite(x).all() for x in got.values())
    for part in ("y", "dq", "final") if large == "rows before" else ("dk", "dv", "dh0"):
        value, bound = want[part]
        assert_within(got[part], value, bound + 2.0 ** -144 * size[part])
        off = (got[part].cpu().double() - value).norm()
        assert off < 0.1 * value.norm() or first == 0 and part in ("dk", "dv") and not got[part].any(), part  # no rows before


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gate", [-87.0, -88.0, -95.0, -103.0, -103.9720764, -103.9720841, -104.0])
def test_one_row_as_a_step(gpu, dtype, gate):
    """The pass over one row and the single-token form keep, or forget, the same state: e^g is 0 in float32 below
    -103.97208, and a multiple of 2^-149 above it."""
    t = make(gpu, dtype, 1, 2, 16, 16)
    t["k"] = t["k"] * 0
    t["g"].fill_(gate)
    t["h0"] *= 1e36
    r = lx.laplex_attend(t["q"], t["k"], t["v"], t["g"], h0=t["h0"], final=True)
    state = t["h0"].clone()
    y = lx.laplex_attend_step(t["q"], t["k"], t["v"], t["g"], state)
    slack = 2.0 ** -148 * t["h0"].cpu().double().abs() + 200 * 2.0 ** -23 * state.cpu().double().abs()
    assert ((r.final - state).cpu().double().abs() <= slack).all()
    assert bool(r.final.any()) == bool(state.any()) == (gate > -103.97208)
    assert bool(r.y.any()) == bool(y.any())
    if dtype is not torch.float16:  # whose smallest number is 6e-8; sums of states of 1e-9 are not
        assert bool(y.any()) == (gate > -103.97208)
