"""Inputs of the token operators on a stream that is not their own."""
import pytest
import torch

from laplace_matvec_amd import laplex as lx

pytestmark = pytest.mark.gpu

TOKENS, SLOTS, WIDTH, HEADS = 4096, 2, 128, 8


def inputs(gpu):
    """Tensors of the calls below, none of a size that any other has, so that
    a block of one that is given out again shows."""
    gen = torch.Generator(device=gpu).manual_seed(0)
    rand = lambda *s: torch.randn(*s, device=gpu, generator=gen)  # noqa: E731
    ids = torch.randint(0, 5, (TOKENS, SLOTS), device=gpu, generator=gen)
    return dict(ids=ids, x=rand(TOKENS, WIDTH), ys=rand(TOKENS * SLOTS, WIDTH), w=rand(TOKENS, SLOTS),
                g=-rand(TOKENS, HEADS).abs(), h0=rand(2, WIDTH), state=rand(TOKENS, WIDTH),
                offsets=torch.tensor([0, 1000, TOKENS], dtype=torch.int32, device=gpu),
                slots=torch.arange(TOKENS - 1, -1, -1, dtype=torch.int32, device=gpu))


CALLS = {
    "route": (("ids",), lambda t, r, s: lx.laplex_route(t["ids"], 5, stream=s)),
    "dispatch": (("x",), lambda t, r, s: lx.laplex_dispatch(r, t["x"], stream=s)),
    "combine": (("ys", "w"), lambda t, r, s: lx.laplex_combine(r, t["ys"], t["w"], stream=s)),
    "combine_backward": (("x", "ys", "w"), lambda t, r, s: lx.laplex_combine_backward(r, t["x"], t["ys"], t["w"],
                                                                                      stream=s)),
    "recur": (("x", "g", "h0", "offsets"), lambda t, r, s: lx.laplex_recur(t["x"], t["g"], t["offsets"], t["h0"],
                                                                           final=True, keep=True, stream=s)),
    "recur_backward": (("x", "g", "state", "h0", "offsets"),
                       lambda t, r, s: lx.laplex_recur_backward(t["x"], t["g"], t["state"], t["kept"], t["offsets"],
                                                                t["h0"], dfinal=t["h0"], stream=s)),
    "step": (("x", "g", "state", "slots"), lambda t, r, s: lx.laplex_recur_step(t["x"], t["g"], t["state"],
                                                                                slots=t["slots"], stream=s)),
}


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_inputs_outlive_a_call_on_another_stream(gpu, name, raw):
    """Their memory is not given out again while the stream still has the call before it."""
    used, call = CALLS[name]
    t = inputs(gpu)
    route = lx.laplex_route(t["ids"], 5)
    if name == "recur_backward":
        t["kept"] = lx.laplex_recur(t["x"], t["g"], t["offsets"], t["h0"], keep=True).states
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # some tenths of a second of work before the call
    out = call(t, route, side.cuda_stream if raw else side)
    sizes = {k: (t[k].data_ptr(), t[k].shape, t[k].dtype) for k in used}
    t.clear()  # the last references
    for k, (ptr, shape, dtype) in sizes.items():
        again = [torch.empty(shape, dtype=dtype, device=gpu) for _ in range(3)]
        assert all(a.data_ptr() != ptr for a in again), k
    busy = not side.query()
    torch.cuda.synchronize()
    assert busy, "the stream was done too early for the test to say anything"
    del out
