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
