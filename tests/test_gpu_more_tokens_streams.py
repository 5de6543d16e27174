"""Inputs of the experts' products and the matrix memory on a stream that is
not their own, and outputs behind which other memory lies."""
import pytest
import torch

from laplace_matvec_amd import laplex as lx

pytestmark = pytest.mark.gpu

ROWS, HEADS, DK, DV = 3000, 4, 48, 40


def inputs(gpu):
    """Tensors of the calls below, none of a size that any other has, so that
    a block of one that is given out again shows."""
    gen = torch.Generator(device=gpu).manual_seed(0)
    rand = lambda *s: torch.randn(*s, device=gpu, generator=gen)  # noqa: E731
    at = lambda *v: torch.tensor(v, dtype=torch.int32, device=gpu)  # noqa: E731
    return dict(x=rand(ROWS, 96), w=rand(3, 80, 96), dy=rand(ROWS, 80), offsets=at(0, 900, 900, ROWS),
                q=rand(ROWS, 2, DK), k=rand(ROWS, 1, DK), v=rand(ROWS, HEADS, DV), g=-rand(ROWS, HEADS).abs(),
                h0=rand(2, HEADS, DK, DV), da=rand(ROWS, HEADS, DV), two=at(0, 1000, ROWS),
                dfinal=rand(2, HEADS, DK, DV), pool=rand(ROWS + 7, HEADS, 8, 8), q8=rand(ROWS, HEADS, 8),
                slots=torch.arange(ROWS - 1, -1, -1, dtype=torch.int32, device=gpu))


CALLS = {
    "experts": (("x", "w", "offsets"), lambda t, s: lx.laplex_experts(t["x"], t["w"], t["offsets"], stream=s)),
    "experts_backward": (("x", "w", "dy", "offsets"),
                         lambda t, s: lx.laplex_experts_backward(t["x"], t["w"], t["dy"], t["offsets"], stream=s)),
    "attend": (("q", "k", "v", "g", "h0", "two"),
               lambda t, s: lx.laplex_attend(t["q"], t["k"], t["v"], t["g"], t["two"], t["h0"], final=True, keep=True,
                                             stream=s)),
    "attend_backward": (("q", "k", "v", "g", "da", "kept", "h0", "dfinal", "two"),
                        lambda t, s: lx.laplex_attend_backward(t["q"], t["k"], t["v"], t["g"], t["da"], t["kept"],
                                                               t["two"], t["h0"], dfinal=t["dfinal"], stream=s)),
    "attend_step": (("q8", "g", "pool", "slots"),
                    lambda t, s: lx.laplex_attend_step(t["q8"], t["q8"], t["q8"], t["g"], t["pool"], slots=t["slots"],
                                                       stream=s)),
}


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_inputs_outlive_a_call_on_another_stream(gpu, name, raw):
    """Their memory is not given out again while the stream still has the call before it."""
    used, call = CALLS[name]
    t = inputs(gpu)
    t["kept"] = lx.laplex_attend(t["q"], t["k"], t["v"], t["g"], t["two"], t["h0"], keep=True).states
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # some tenths of a second of work before the call
    out = call(t, side.cuda_stream if raw else side)
    sizes = {k: (t[k].data_ptr(), t[k].shape, t[k].dtype) for k in used}
    t.clear()  # the last references
    for k, (ptr, shape, dtype) in sizes.items():
        again = [torch.empty(shape, dtype=dtype, device=gpu) for _ in range(3)]
        assert all(a.data_ptr() != ptr for a in again), k
    busy = not side.query()
    torch.cuda.synchronize()
    assert busy, "the stream was done too early for the test to say anything"
    del out


def at(t):
    return None if t is None else t.data_ptr()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("counts", [[3, 0, 5], [300, 0, 131]])
@pytest.mark.parametrize("transpose", [0, 1])
def test_experts_write_their_rows_alone(gpu, dtype, counts, transpose):
    """y, dx and dw as parts of wider arrays: what lies between and behind stays."""
    lib, kind = lx.load(), lx._DTYPES[dtype]
    n, inner, outer, E = sum(counts) + 9, 88, 56, len(counts)
    offsets = torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32, device=gpu)
    gen = torch.Generator(device=gpu).manual_seed(1)
    rand = lambda *s: torch.randn(*s, device=gpu, generator=gen).to(dtype)  # noqa: E731
    x, dy = rand(n, inner), rand(n, outer)
    rw, cw = (inner, outer) if transpose else (outer, inner)
    w = rand(E, rw, cw)
    y = torch.full((n + 1, outer + 5), 7.0, dtype=dtype, device=gpu)
    dx = torch.full((n + 1, inner + 3), 7.0, dtype=dtype, device=gpu)
    dw = torch.full((E, rw + 2, cw + 3), 7.0, dtype=dtype, device=gpu)
    s = torch.cuda.current_stream().cuda_stream
    lx._check(lib.laplex_experts(n, E, at(offsets), inner, outer, kind, transpose, at(x), inner, at(w), cw, rw * cw,
                                 at(y), outer + 5, s), "experts")
    lx._check(lib.laplex_experts_backward(n, E, at(offsets), inner, outer, kind, transpose, at(x), inner, at(w), cw,
                                          rw * cw, at(dy), outer, at(dx), inner + 3, at(dw), cw + 3,
                                          (rw + 2) * (cw + 3), s), "experts_backward")
    assert torch.equal(y[:n, :outer], lx.laplex_experts(x, w, offsets, transpose=bool(transpose)))
    want = lx.laplex_experts_backward(x, w, dy, offsets, transpose=bool(transpose))
    assert torch.equal(dx[:n, :inner], want["dx"]) and torch.equal(dw[:, :rw, :cw], want["dw"])
    for t, rows, cols in ((y, n, outer), (dx, n, inner)):
        assert bool((t[rows:] == 7).all()) and bool((t[:, cols:] == 7).all())
    assert bool((dw[:, rw:] == 7).all()) and bool((dw[:, :, cw:] == 7).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", [(40, 72), (33, 7), (160, 64)])
def test_attend_writes_its_rows_alone(gpu, dtype, dk, dv):
    """Results as parts of wider rows, scratch exactly as large as asked for."""
    lib, kind = lx.load(), lx._DTYPES[dtype]
    n, heads = 333, 2
    gen = torch.Generator(device=gpu).manual_seed(1)
    rand = lambda *s: torch.randn(*s, device=gpu, generator=gen).to(dtype)  # noqa: E731
    q, k, v, dy = rand(n, heads, dk), rand(n, heads, dk), rand(n, heads, dv), rand(n, heads, dv)
    g = -torch.rand(n, heads, device=gpu, generator=gen)
    r = lx.laplex_attend(q, k, v, g, keep=True)
    want = lx.laplex_attend_backward(q, k, v, g, dy, r.states)
    wide = lambda width, like: torch.full((n + 1, width + 3), 7.0, dtype=like.dtype, device=gpu)  # noqa: E731
    y, dq, dkey, dval, dg = (wide(heads * d, t) for d, t in ((dv, q), (dk, q), (dk, q), (dv, q), (1, g)))
    sizes = (heads, heads, heads, heads, dk, dv)
    need = [lib.laplex_attend_workspace(n, 1, *sizes, kind, b) for b in (0, 1)]
    ws = [torch.full((b + 4096,), 7, dtype=torch.uint8, device=gpu) for b in need]
    s = torch.cuda.current_stream().cuda_stream
    ins = (n, 1, None, *sizes, kind, 0, 1.0, at(q), heads * dk, at(k), heads * dk, at(v), heads * dv, at(g), heads, None)
    lx._check(lib.laplex_attend(*ins, at(y), heads * dv + 3, None, None, at(ws[0]), need[0], s), "attend")
    lx._check(lib.laplex_attend_backward(*ins, at(r.states), at(dy), heads * dv, None, at(dq), heads * dk + 3, at(dkey),
                                         heads * dk + 3, at(dval), heads * dv + 3, at(dg), heads + 3, None, at(ws[1]),
                                         need[1], s), "attend_backward")
    for t, width, value in ((y, heads * dv, r.y), (dq, heads * dk, want["dq"]), (dkey, heads * dk, want["dk"]),
                            (dval, heads * dv, want["dv"]), (dg, heads, want["dg"])):
        assert torch.equal(t[:n, :width], value.reshape(n, width))
        assert bool((t[n:] == 7).all()) and bool((t[:, width:] == 7).all())
    for t, b in zip(ws, need):
        assert bool((t[b:] == 7).all())
