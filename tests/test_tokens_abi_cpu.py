"""Refusals of the token operators' C entry points, on the host before any
HIP call, and of their binding."""
import ctypes

import pytest
import torch

from laplace_matvec_amd import laplex as lx

BAD = lx.ERR_INVALID_ARGUMENT


def at(i):
    """A fake, aligned address; never followed: the checks run first."""
    return ctypes.c_void_p((i + 1) << 40)


def bad(name, args):
    assert getattr(lx.load(), name)(*args) == BAD
    assert lx.load().laplex_last_error()


def changed(base, **kw):
    d = dict(base)
    d.update(kw)
    return list(d.values())


ROUTE = dict(experts=at(0), wide=0, tokens=100, slots=2, n_experts=8, order=at(1), place=at(2), offsets=at(3),
             ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("kw", [
    dict(experts=None), dict(order=None), dict(place=None), dict(offsets=None), dict(wide=2), dict(wide=-1),
    dict(tokens=-1), dict(slots=0), dict(n_experts=0), dict(n_experts=4097),
    dict(tokens=1 << 30, slots=2), dict(tokens=(1 << 30) + 1, slots=1),
    dict(tokens=1 << 62, slots=1 << 62),                     # no overflow on the way
    dict(tokens=10000),                                      # needs scratch
    dict(tokens=10000, ws=ctypes.c_void_p(8), ws_bytes=1 << 30),  # misaligned
    dict(tokens=10000, ws=at(4), ws_bytes=100),              # too small
    dict(tokens=10000, ws=at(1), ws_bytes=1 << 30),          # overlaps order
    dict(place=at(1)), dict(order=at(0)), dict(offsets=ctypes.c_void_p((4 << 40) + 1)),
    dict(experts=ctypes.c_void_p((1 << 40) + 2)),
])
def test_route_refuses(kw):
    bad("laplex_route", changed(ROUTE, **kw))


def test_route_workspace():
    f = lx.load().laplex_route_workspace
    assert f(0, 1, 1) == 0 and f(48, 2, 8) == 0
    assert f(1 << 20, 1, 256) >= 4 * 256 * ((1 << 20) // 4096)
    assert f(-1, 1, 1) == f(1, 0, 1) == f(1, 1, 0) == f(1, 1, 4097) == f(1 << 30, 2, 1) == -1


DISPATCH = dict(tokens=10, slots=2, n_experts=8, place=at(0), offsets=at(1), type=1, width=64, x=at(2), ldx=64,
                xs=at(3), ldxs=64, stream=None)


@pytest.mark.parametrize("kw", [
    dict(place=None), dict(offsets=None), dict(x=None), dict(xs=None), dict(type=3), dict(type=-1), dict(width=0),
    dict(width=(1 << 24) + 1), dict(tokens=-1), dict(slots=0), dict(n_experts=0), dict(ldx=63), dict(ldxs=63),
    dict(xs=at(2)), dict(x=ctypes.c_void_p((3 << 40) + 1)), dict(xs=at(0)), dict(tokens=1 << 40),
    dict(ldx=1 << 50),
])
def test_dispatch_refuses(kw):
    bad("laplex_dispatch", changed(DISPATCH, **kw))


COMBINE = dict(tokens=10, slots=2, place=at(0), type=0, width=64, ys=at(1), ldys=64, weights=at(2), y=at(3), ldy=64,
               stream=None)


@pytest.mark.parametrize("kw", [
    dict(place=None), dict(ys=None), dict(y=None), dict(type=9), dict(width=0), dict(tokens=-5), dict(slots=0),
    dict(ldys=1), dict(ldy=1), dict(y=at(1)), dict(y=at(2)), dict(y=ctypes.c_void_p((4 << 40) + 2)),
])
def test_combine_refuses(kw):
    bad("laplex_combine", changed(COMBINE, **kw))


COMBINE_GRAD = dict(tokens=10, slots=2, n_experts=8, place=at(0), offsets=at(1), type=2, width=64, dy=at(2), lddy=64,
                    ys=at(3), ldys=64, weights=at(4), dys=at(5), lddys=64, dw=at(6), stream=None)


@pytest.mark.parametrize("kw", [
    dict(place=None), dict(dy=None), dict(weights=None), dict(offsets=None), dict(ys=None), dict(type=3),
    dict(lddy=3), dict(ldys=3), dict(lddys=3), dict(dys=at(3)), dict(dw=at(5)), dict(dw=at(4)), dict(n_experts=5000),
])
def test_combine_backward_refuses(kw):
    bad("laplex_combine_backward", changed(COMBINE_GRAD, **kw))


def test_nothing_to_do_is_ok():
    lib = lx.load()
    assert lib.laplex_combine_backward(*changed(COMBINE_GRAD, dys=None, dw=None)) == lx.OK
    assert lib.laplex_dispatch(*changed(DISPATCH, tokens=0)) == lx.OK
    assert lib.laplex_combine(*changed(COMBINE, tokens=0)) == lx.OK
    assert lib.laplex_recur_backward(*changed(RECUR_GRAD, dx=None, dg=None, dh0=None)) == lx.OK
    assert lib.laplex_recur_step(*changed(STEP, n=0)) == lx.OK


RECUR = dict(n=1000, seqs=1, offsets=None, width=64, heads=8, type=1, gate_type=0, x=at(0), ldx=64, g=at(1), ldg=8,
             h0=at(2), y=at(3), ldy=64, final=at(4), states=at(5), ws=at(6), ws_bytes=1 << 30, stream=None)
RECUR_GRAD = dict(n=1000, seqs=1, offsets=None, width=64, heads=8, type=1, gate_type=0, x=at(0), ldx=64, g=at(1),
                  ldg=8, h0=at(2), states=at(3), dy=at(4), lddy=64, dfinal=at(5), dx=at(6), lddx=64, dg=at(7), lddg=8,
                  dh0=at(8), ws=at(9), ws_bytes=1 << 30, stream=None)
SIZES = [dict(n=-1), dict(n=1 << 31), dict(seqs=0), dict(seqs=-1), dict(seqs=3), dict(width=0), dict(heads=0),
         dict(heads=7), dict(heads=128), dict(width=(1 << 24) + 8), dict(type=3), dict(type=1, gate_type=2),
         dict(type=0, gate_type=1), dict(x=None), dict(g=None), dict(ldx=60), dict(ldg=7), dict(ldx=(1 << 24) + 1),
         dict(ws=None), dict(ws_bytes=1000), dict(ws=ctypes.c_void_p((7 << 40) + 8)),
         dict(x=ctypes.c_void_p((1 << 40) + 1)), dict(g=ctypes.c_void_p((2 << 40) + 2)),
         dict(n=(1 << 31) - 1, width=1 << 24, heads=1 << 24, ldx=1 << 24, ldg=1 << 24)]


@pytest.mark.parametrize("kw", SIZES + [
    dict(y=None), dict(ldy=60), dict(ldy=(1 << 24) + 64), dict(y=at(0)), dict(y=at(1)), dict(final=at(2)),
    dict(final=at(3)), dict(states=ctypes.c_void_p((6 << 40) + 4)), dict(ws=at(5)), dict(states=at(3)),
])
def test_recur_refuses(kw):
    bad("laplex_recur", changed(RECUR, **kw))


@pytest.mark.parametrize("kw", SIZES + [
    dict(dy=None), dict(states=None), dict(lddy=60), dict(lddx=60), dict(lddg=7), dict(dx=at(0)), dict(dx=at(4)),
    dict(dg=at(1)), dict(dg=at(6)), dict(dh0=at(5)), dict(dh0=at(2)), dict(ws=at(3)),
])
def test_recur_backward_refuses(kw):
    bad("laplex_recur_backward", changed(RECUR_GRAD, **kw))


def test_recur_sizes():
    lib = lx.load()
    assert lib.laplex_recur_workspace(0, 64, 8, 0) == lib.laplex_recur_workspace(1, 64, 8, 0) == 0
    assert lib.laplex_recur_states(1, 64) == 0 and lib.laplex_recur_states(0, 64) == 0
    assert lib.laplex_recur_states(100000, 65) >= 65
    assert lib.laplex_recur_workspace(100000, 64, 8, 0) > 4 * lib.laplex_recur_states(100000, 64)
    # decays that span channel tiles take partial sums
    assert lib.laplex_recur_workspace(1000, 256, 2, 1) >= 4 * 1000 * 2
    for args in ((-1, 64, 8, 0), (1 << 31, 64, 8, 0), (10, 0, 1, 0), (10, 64, 7, 0), (10, 64, 8, 2)):
        assert lib.laplex_recur_workspace(*args) == -1
    assert lib.laplex_recur_states(-1, 64) == lib.laplex_recur_states(5, 0) == -1


STEP = dict(n=10, pool=20, slots=at(0), width=64, heads=8, type=2, gate_type=2, x=at(1), ldx=64, g=at(2), ldg=8,
            state=at(3), y=at(4), ldy=64, stream=None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(pool=-1), dict(pool=1 << 31), dict(slots=None, n=21), dict(width=0), dict(heads=5),
    dict(type=2, gate_type=1), dict(type=4), dict(x=None), dict(g=None), dict(state=None), dict(y=None), dict(ldx=63),
    dict(ldy=63), dict(ldg=7), dict(y=at(3)), dict(y=at(1)), dict(state=at(2)), dict(state=at(0)),
    dict(state=ctypes.c_void_p((4 << 40) + 2)),
])
def test_step_refuses(kw):
    bad("laplex_recur_step", changed(STEP, **kw))


def test_rows_may_interleave():
    """Outputs beside each other in wider rows are no overlap; the call gets as far as the device."""
    wide = dict(x=at(0), ldx=128, g=ctypes.c_void_p(at(0).value + 128), ldg=128, gate_type=1, heads=64)
    grads = dict(dx=at(6), lddx=128, dg=ctypes.c_void_p(at(6).value + 128), lddg=128)
    if torch.cuda.is_available():
        pytest.skip("the addresses are fake")
    assert lx.load().laplex_recur_backward(*changed(RECUR_GRAD, **wide, **grads)) == lx.ERR_NO_DEVICE
    grads["dg"] = ctypes.c_void_p(at(6).value + 126)
    bad("laplex_recur_backward", changed(RECUR_GRAD, **wide, **grads))


def test_binding_refuses_host_tensors_and_types():
    x, g = torch.zeros(4, 8), torch.zeros(4, 2)
    ids = torch.zeros(4, 2, dtype=torch.int64)
    for call in (lambda: lx.laplex_route(ids, 4), lambda: lx.laplex_route([[1]], 4), lambda: lx.laplex_recur(x, g),
                 lambda: lx.laplex_recur_step(x, g, torch.zeros(4, 8)), lambda: lx.laplex_recur([1.0], g),
                 lambda: lx.laplex_recur_backward(x, g, x, torch.zeros(0)),
                 lambda: lx.laplex_dispatch(lx.Route(ids, ids, ids), x),
                 lambda: lx.laplex_combine(lx.Route(ids, ids, ids), x),
                 lambda: lx.laplex_combine_backward(lx.Route(ids, ids, ids), x, x, x)):
        with pytest.raises(TypeError):
            call()
