"""Refusals of the experts' and the matrix memory's C entry points, on the
host before any HIP call, and of their binding; the float64 forms that the GPU
tests compare with, against differences and the recurrence itself."""
import ctypes
import math

import pytest
import torch

import more_tokens_ref as ref
from laplace_matvec_amd import laplex as lx
from test_tokens_abi_cpu import at, bad, changed

EXPERTS = dict(n=100, n_experts=8, offsets=at(0), inner=64, out=32, type=1, transpose=0, x=at(1), ldx=64, w=at(2),
               ldw=64, pitch=2048, y=at(3), ldy=32, stream=None)
EXPERTS_GRAD = dict(n=100, n_experts=8, offsets=at(0), inner=64, out=32, type=1, transpose=0, x=at(1), ldx=64, w=at(2),
                    ldw=64, pitch=2048, dy=at(3), lddy=32, dx=at(4), lddx=64, dw=at(5), lddw=64, pitch_dw=2048,
                    stream=None)
EXPERT_SIZES = [dict(n=-1), dict(n=1 << 31), dict(n_experts=0), dict(n_experts=4097), dict(inner=0), dict(out=0),
                dict(inner=(1 << 24) + 1), dict(out=(1 << 24) + 1), dict(type=3), dict(transpose=2),
                dict(transpose=-1), dict(offsets=None), dict(x=None), dict(w=None), dict(ldx=63), dict(ldw=63),
                dict(transpose=1, ldw=31), dict(pitch=-1), dict(pitch=1 << 47), dict(ldw=1 << 41), dict(ldx=1 << 50),
                dict(x=ctypes.c_void_p((1 << 41) + 1)), dict(w=ctypes.c_void_p((1 << 41) + 1)),
                dict(offsets=ctypes.c_void_p((1 << 40) + 2))]


@pytest.mark.parametrize("kw", EXPERT_SIZES + [dict(y=None), dict(ldy=31), dict(y=at(1)), dict(y=at(2)), dict(y=at(0))])
def test_experts_refuses(kw):
    bad("laplex_experts", changed(EXPERTS, **kw))


@pytest.mark.parametrize("kw", EXPERT_SIZES + [
    dict(dy=None), dict(lddy=31), dict(lddx=63), dict(lddw=63), dict(pitch_dw=2047), dict(pitch_dw=0), dict(dx=at(1)),
    dict(dx=at(3)), dict(dw=at(2)), dict(dw=at(4)), dict(dw=at(0)), dict(dw=ctypes.c_void_p((6 << 40) + 1)),
])
def test_experts_backward_refuses(kw):
    bad("laplex_experts_backward", changed(EXPERTS_GRAD, **kw))


ATTEND = dict(n=1000, seqs=1, offsets=None, heads=8, hq=4, hk=4, hv=8, dk=16, dv=24, type=1, gate_type=0, scale=1.0,
              q=at(0), ldq=64, k=at(1), ldk=64, v=at(2), ldv=192, g=at(3), ldg=8, h0=at(4), y=at(5), ldy=192,
              final=at(6), states=at(7), ws=at(8), ws_bytes=1 << 40, stream=None)
ATTEND_GRAD = dict(n=1000, seqs=1, offsets=None, heads=8, hq=4, hk=4, hv=8, dk=16, dv=24, type=1, gate_type=0,
                   scale=1.0, q=at(0), ldq=64, k=at(1), ldk=64, v=at(2), ldv=192, g=at(3), ldg=8, h0=at(4),
                   states=at(5), dy=at(6), lddy=192, dfinal=at(7), dq=at(8), lddq=64, dk_out=at(9), lddk=64,
                   dv_out=at(10), lddv=192, dg=at(11), lddg=8, dh0=at(12), ws=at(13), ws_bytes=1 << 39, stream=None)
SIZES = [dict(n=-1), dict(n=1 << 31), dict(seqs=0), dict(seqs=3), dict(seqs=(1 << 24) + 1, offsets=at(20)),
         dict(heads=0), dict(heads=4097), dict(hq=3), dict(hk=0), dict(hv=16), dict(dk=0), dict(dk=1025), dict(dv=0),
         dict(dv=1025), dict(type=3), dict(type=1, gate_type=2), dict(type=0, gate_type=1), dict(q=None), dict(k=None),
         dict(v=None), dict(g=None), dict(ldq=63), dict(ldk=63), dict(ldv=191), dict(ldg=7), dict(ws=None),
         dict(ws_bytes=1000), dict(ws=ctypes.c_void_p((9 << 40) + 8)), dict(q=ctypes.c_void_p((1 << 40) + 1)),
         dict(g=ctypes.c_void_p((4 << 40) + 2)), dict(offsets=ctypes.c_void_p((20 << 40) + 2)),
         dict(n=(1 << 31) - 1, heads=4096, hv=4096, dk=1024, dv=1024), dict(ldq=1 << 50)]


@pytest.mark.parametrize("kw", SIZES + [
    dict(y=None), dict(ldy=191), dict(y=at(0)), dict(y=at(3)), dict(final=at(4)), dict(final=at(5)),
    dict(states=ctypes.c_void_p((8 << 40) + 4)), dict(ws=at(5)), dict(states=at(2)),
])
def test_attend_refuses(kw):
    bad("laplex_attend", changed(ATTEND, **kw))


@pytest.mark.parametrize("kw", SIZES + [
    dict(dy=None), dict(states=None), dict(lddy=191), dict(lddq=63), dict(lddk=63), dict(lddv=191), dict(lddg=7),
    dict(dq=at(0)), dict(dk_out=at(8)), dict(dv_out=at(6)), dict(dg=at(3)), dict(dh0=at(7)), dict(dh0=at(4)),
    dict(ws=at(5)), dict(states=ctypes.c_void_p((6 << 40) + 4)),
])
def test_attend_backward_refuses(kw):
    bad("laplex_attend_backward", changed(ATTEND_GRAD, **kw))


STEP = dict(n=10, pool=20, slots=at(0), heads=8, hq=4, hk=2, hv=8, dk=16, dv=24, type=2, gate_type=2, scale=1.0,
            q=at(1), ldq=64, k=at(2), ldk=32, v=at(3), ldv=192, g=at(4), ldg=8, state=at(5), y=at(6), ldy=192,
            stream=None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=1 << 31), dict(pool=-1), dict(pool=1 << 31), dict(slots=None, n=21), dict(heads=0), dict(hq=3),
    dict(dk=0), dict(dv=2000), dict(type=2, gate_type=1), dict(type=4), dict(q=None), dict(k=None), dict(v=None),
    dict(g=None), dict(state=None), dict(y=None), dict(ldq=63), dict(ldk=31), dict(ldv=191), dict(ldg=7),
    dict(ldy=191), dict(y=at(5)), dict(y=at(1)), dict(state=at(0)), dict(state=ctypes.c_void_p((6 << 40) + 2)),
])
def test_attend_step_refuses(kw):
    bad("laplex_attend_step", changed(STEP, **kw))


def test_nothing_to_do_is_ok():
    lib = lx.load()
    assert lib.laplex_experts(*changed(EXPERTS, n=0)) == lx.OK
    assert lib.laplex_experts_backward(*changed(EXPERTS_GRAD, dx=None, dw=None)) == lx.OK
    assert lib.laplex_attend_backward(*changed(ATTEND_GRAD, dq=None, dk_out=None, dv_out=None, dg=None, dh0=None)) == lx.OK
    assert lib.laplex_attend_step(*changed(STEP, n=0)) == lx.OK


def test_attend_sizes():
    lib = lx.load()
    states, need = lib.laplex_attend_states, lib.laplex_attend_workspace
    assert states(1, 1, 4, 64, 64) == states(0, 1, 4, 64, 64) == 0
    assert states(100000, 1, 4, 64, 64) >= 4 * 64 * 64
    assert need(10, 1, 4, 4, 4, 4, 64, 64, 1, 0) == 0
    # states between chunks in both directions
    assert need(128, 1, 4, 4, 4, 4, 64, 64, 1, 1) >= 2 * 4 * 2 * 4 * 64 * 64
    # heads that share values take partial sums
    assert need(128, 1, 4, 4, 4, 1, 64, 64, 1, 1) >= need(128, 1, 4, 4, 4, 4, 64, 64, 1, 1) + 4 * 4 * 128 * 64
    for args in ((-1, 1, 4, 4, 4, 4, 64, 64, 1, 0), (10, 0, 4, 4, 4, 4, 64, 64, 1, 0), (10, 1, 0, 1, 1, 1, 64, 64, 1, 0),
                 (10, 1, 4, 3, 4, 4, 64, 64, 1, 0), (10, 1, 4, 4, 4, 4, 0, 64, 1, 0), (10, 1, 4, 4, 4, 4, 64, 1025, 1, 0),
                 (10, 1, 4, 4, 4, 4, 64, 64, 3, 0), (10, 1, 4, 4, 4, 4, 64, 64, 1, 2)):
        assert need(*args) == -1
    assert states(-1, 1, 4, 64, 64) == states(5, 1, 0, 64, 64) == states(5, 1 << 25, 4, 64, 64) == -1


def test_binding_refuses_host_tensors_and_types():
    x, w, o = torch.zeros(4, 8), torch.zeros(2, 6, 8), torch.zeros(3, dtype=torch.int32)
    q, g = torch.zeros(4, 2, 8), torch.zeros(4, 2)
    for call in (lambda: lx.laplex_experts(x, w, o), lambda: lx.laplex_experts([1.0], w, o),
                 lambda: lx.laplex_experts_backward(x, w, x, o), lambda: lx.laplex_attend(q, q, q, g),
                 lambda: lx.laplex_attend([1.0], q, q, g), lambda: lx.laplex_attend(q, q, q, [1.0]),
                 lambda: lx.laplex_attend_backward(q, q, q, g, q, torch.zeros(0)),
                 lambda: lx.laplex_attend_step(q, q, q, g, torch.zeros(4, 2, 8, 8)),
                 lambda: lx.laplex_attend_step(q, q, q, [1.0], torch.zeros(4, 2, 8, 8))):
        with pytest.raises(TypeError):
            call()


# ---- the float64 forms


def small(n=23, heads=4, shared=(2, 1, 4), dk=3, dv=5, seqs=3):
    gen = torch.Generator().manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    g = -torch.rand(n, heads, generator=gen, dtype=torch.float64)
    g[7, 1], g[0, 2], g[11, 0] = -math.inf, -math.inf, -150.0
    hq, hk, hv = shared
    return [rand(n, hq, dk), rand(n, hk, dk), rand(n, hv, dv), g], [2, 9, 9, 21], rand(seqs, heads, dk, dv), \
        rand(n, heads, dv), rand(seqs, heads, dk, dv)


def recurrence(q, k, v, g, offsets, h0, scale):
    """The definition, one token after the other."""
    n, heads = g.shape
    rep = lambda t: t.repeat_interleave(heads // t.shape[1], 1)  # noqa: E731
    q, k, v = rep(q), rep(k), rep(v)
    y, final = [torch.zeros(heads, v.shape[-1], dtype=torch.float64)] * n, []
    for s in range(len(offsets) - 1):
        h = h0[s]
        for t in range(offsets[s], offsets[s + 1]):
            kept = g[t].detach().float().exp() != 0
            a = torch.where(kept, g[t], 0.0).exp()
            h = torch.where(kept[:, None, None], a[:, None, None] * h, 0.0) + k[t][:, :, None] * v[t][:, None, :]
            y[t] = scale * (q[t][:, :, None] * h).sum(1)
        final.append(h)
    return torch.stack(y), torch.stack(final)


def test_reference_is_the_recurrence_and_its_gradient():
    args, offsets, h0, dy, dfinal = small()
    leaves = [t.clone().requires_grad_() for t in (*args, h0)]
    y, final = recurrence(*leaves[:4], offsets, leaves[4], 0.7)
    ((y * dy).sum() + (final * dfinal).sum()).backward()
    got = ref._attend(*args, offsets, h0, 0.7, dy, dfinal, False)
    assert torch.allclose(got["y"], y.detach(), atol=1e-12) and torch.allclose(got["final"], final.detach(), atol=1e-12)
    for name, leaf in zip(("dq", "dk", "dv", "dg", "dh0"), leaves):
        want = torch.zeros_like(leaf) if leaf.grad is None else leaf.grad
        assert torch.allclose(got[name], want, atol=1e-12), name


def test_reference_gradient_against_differences():
    args, offsets, h0, dy, dfinal = small()
    grads = ref._attend(*args, offsets, h0, 0.7, dy, dfinal, False)
    gen = torch.Generator().manual_seed(2)

    def loss(parts):
        r = ref._attend(*parts[:4], offsets, parts[4], 0.7, None, None, False)
        return float((r["y"] * dy).sum() + (r["final"] * dfinal).sum())

    for i, name in enumerate(("dq", "dk", "dv", "dg", "dh0")):
        parts = [*args, h0]
        u = torch.randn(parts[i].shape, generator=gen, dtype=torch.float64)
        ends = []
        for sign in (1, -1):
            moved = list(parts)
            moved[i] = parts[i] + sign * 1e-5 * u
            ends.append(loss(moved))
        slope = float((grads[name] * u).sum())
        assert abs((ends[0] - ends[1]) / 2e-5 - slope) <= 1e-6 * max(1.0, float((grads[name] * u).abs().sum()))


def test_step_reference_is_the_recurrence():
    args, _, h0, _, _ = small()
    one = [a[:3] for a in args]
    y, final = recurrence(*one, [0, 1, 2, 3], h0, 0.7)
    (got, _), (state, _) = ref.attend_step(*one, h0, [0, 1, 2], 0.7)
    assert torch.allclose(got, y, atol=1e-12) and torch.allclose(state, final, atol=1e-12)


def test_experts_reference_gradient():
    gen = torch.Generator().manual_seed(3)
    for transpose in (False, True):
        x = torch.randn(9, 4, generator=gen, dtype=torch.float64).requires_grad_()
        w = torch.randn(3, *((4, 5) if transpose else (5, 4)), generator=gen, dtype=torch.float64).requires_grad_()
        dy, offsets = torch.randn(9, 5, generator=gen, dtype=torch.float64), [1, 4, 4, 8]
        y = torch.stack([sum((w[e].t() if transpose else w[e]) @ x[r] * (offsets[e] <= r < offsets[e + 1]) for e in range(3))
                         for r in range(9)])
        (y * dy).sum().backward()
        got = ref.experts(x, w, offsets, transpose, dy)
        for (value, _), want in zip(got, (y.detach(), x.grad, w.grad)):
            assert torch.allclose(value, want, atol=1e-12)


def test_gradients_take_no_planes_for_blocks_past_the_keys():
    """float32 and float16 gradients go by key blocks of 64.  Between widths of the same padded states the scratch
    grows by what a block takes: a plane of dv and one of dg."""
    n, heads, dv = 4096, 2, 40
    size = lambda dk, kind: lx.load().laplex_attend_workspace(n, 1, heads, heads, heads, heads, dk, dv, kind, 1)  # noqa: E731
    plane = n * heads * dv * 4 + n * heads * 4
    for kind in (0, 2):
        assert size(256, kind) - size(192, kind) == size(512, kind) - size(448, kind) == plane
        assert size(129, kind) == size(136, kind) == size(192, kind)
    assert size(256, 1) == size(192, 1) == size(136, 1)  # bfloat16: blocks of 128
