"""The token operators' C entry points at the ends of their ranges."""
import pytest
import torch

from laplace_matvec_amd import laplex as lx

pytestmark = pytest.mark.gpu


def at(t):
    return None if t is None else t.data_ptr()


def stream():
    return torch.cuda.current_stream().cuda_stream


def one_row(x, g, dy, width, heads, kind, gkind, ld):
    """y, final, dx, dg and dh0 of a single row whose arrays come with pitch ld."""
    lib, dev = lx.load(), x.device
    new = lambda n, like: torch.full((n,), 7.0, dtype=like.dtype, device=dev)  # noqa: E731
    y, final, dx, dg = new(width, x), torch.empty(width, device=dev), new(width, x), new(heads, g)
    dh0, ws = torch.empty(width, device=dev), torch.empty(1 << 20, dtype=torch.uint8, device=dev)
    h0 = torch.linspace(-1, 1, width, device=dev)
    sizes = (1, 1, None, width, heads, kind, gkind)
    lx._check(lib.laplex_recur(*sizes, at(x), ld, at(g), ld, at(h0), at(y), ld, at(final), None, at(ws), ws.numel(),
                               stream()), "recur")
    lx._check(lib.laplex_recur_backward(*sizes, at(x), ld, at(g), ld, at(h0), None, at(dy), ld, None, at(dx), ld,
                                        at(dg), ld, at(dh0), at(ws), ws.numel(), stream()), "recur_backward")
    return y, final, dx, dg, dh0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
# a decay per channel, shared ones, one channel per thread; 16 rows per thread with more than 256 channel tiles
@pytest.mark.parametrize("width,heads", [(64, 64), (64, 4), (66, 22), (16640, 16640), (16640, 65)])
def test_one_row_of_any_pitch(gpu, dtype, width, heads):
    gen = torch.Generator().manual_seed(width + heads)
    x, dy = (torch.randn(width, generator=gen).to(dtype).to(gpu) for _ in range(2))
    g = (-torch.rand(heads, generator=gen)).to(dtype).to(gpu)
    kind = lx._DTYPES[dtype]
    want = one_row(x, g, dy, width, heads, kind, kind, width)
    for ld in (23000000, 1 << 27, 1 << 28, 1 << 40):
        got = one_row(x, g, dy, width, heads, kind, kind, ld)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), ld
