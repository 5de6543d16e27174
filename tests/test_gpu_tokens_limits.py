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


# ---- more than 2^32 threads' worth of work, at sizes that the contract allows


def big_route(tokens, gpu):
    """One expert; the tokens' rows in reverse order."""
    place = torch.arange(tokens - 1, -1, -1, dtype=torch.int32, device=gpu).view(tokens, 1)
    return lx.Route(place.view(-1), place, torch.tensor([0, tokens], dtype=torch.int32, device=gpu))


def small_values(tokens, width, dtype, gpu):
    """Whole numbers from -100 to 100, exact in every type, another for each row and column."""
    t = torch.arange(tokens, device=gpu, dtype=torch.int32).remainder_(197).to(dtype)
    v = t[:, None].expand(tokens, width).contiguous()
    return v.sub_(torch.arange(width, device=gpu).to(dtype) + 90)


def same(a, b, rows=1 << 26):
    return all(torch.equal(p, q) for p, q in zip(a.split(rows), b.split(rows)))


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def test_combine_backward_of_2_26_short_rows(gpu):
    tokens, width = (1 << 26) + 3, 8
    route = big_route(tokens, gpu)
    dy = small_values(tokens, width, torch.bfloat16, gpu)
    ys = torch.ones_like(dy)
    w = torch.full((tokens, 1), 0.5, device=gpu)
    dys, dw = lx.laplex_combine_backward(route, dy, ys, w)
    assert same(dys, (dy * 0.5).flip(0))
    assert same(dw.view(-1), dy.float().sum(1))


def test_combine_backward_of_2_24_wide_rows(gpu):
    """The weights' gradient alone: a workgroup per token."""
    tokens, width = (1 << 24) + 1, 1032
    route = big_route(tokens, gpu)
    dy = torch.ones(tokens, width, dtype=torch.bfloat16, device=gpu)
    dw = torch.empty(tokens, device=gpu)
    lx._check(lx.load().laplex_combine_backward(tokens, 1, 1, at(route.place), at(route.offsets), 1, width, at(dy),
                                                width, at(dy), width, None, None, width, at(dw), stream()),
              "combine_backward")
    assert bool((dw == width).all())


def test_dispatch_and_combine_of_2_32_values(gpu):
    tokens, width = (1 << 32) // 7 + 5, 7  # a value per thread
    route = big_route(tokens, gpu)
    x = small_values(tokens, width, torch.bfloat16, gpu)
    xs = lx.laplex_dispatch(route, x)
    assert same(xs[:1 << 20], x[-(1 << 20):].flip(0)) and same(xs[-(1 << 20):], x[:1 << 20].flip(0))
    y = lx.laplex_combine(route, xs)
    assert same(y, x)


@pytest.mark.parametrize("backward", [False, True])
def test_states_of_2_24_sequences(gpu, backward):
    """Sequences without rows get their states, the others theirs."""
    seqs, n = (1 << 24) + 70000, 300
    offsets = torch.zeros(seqs + 1, dtype=torch.int32, device=gpu)
    offsets[5:] = 100
    offsets[-2:] = n
    h0 = torch.arange(seqs, device=gpu).remainder_(1000).float().view(seqs, 1)
    x, g = torch.ones(n, 1, device=gpu), torch.zeros(n, 1, device=gpu)
    r = lx.laplex_recur(x, g, offsets=offsets, h0=h0, final=True, keep=True)
    want = h0.clone()
    if backward:
        d = lx.laplex_recur_backward(x, g, torch.ones_like(x), r.states, offsets=offsets, h0=h0, dfinal=h0)
        got = d["dh0"]
    else:
        got = r.final
    want[4] += 100  # decays of 1
    want[seqs - 2] += 200
    assert same(got, want)


def test_one_channel_of_2_30_rows(gpu):
    """Sequences of 256 rows with decays of 1: running counts, whole numbers throughout."""
    n, length = 1 << 30, 256
    x = (torch.arange(n, device=gpu, dtype=torch.int32).bitwise_and_(0x15) == 0x11).to(torch.float16).view(-1, length, 1)
    g = torch.zeros_like(x)
    r = lx.laplex_recur(x, g, keep=True)
    one = torch.cumsum(x[:1].float(), 1)  # the pattern repeats within 256
    assert all(bool((p == one).all()) for p in r.y.split(1 << 16))
    d = lx.laplex_recur_backward(x, g, x, r.states, want=("dx", "dg"))
    back = torch.cumsum(x[:1].float().flip(1), 1).flip(1)
    assert all(bool((p == back).all()) for p in d["dx"].split(1 << 16))
    prev = torch.cat([torch.zeros_like(one[:, :1]), one[:, :-1]], 1)
    # at most 64 * 64: whole in float16 up to 2048, rounded above
    assert all(bool((p == (back * prev).half()).all()) for p in d["dg"].split(1 << 16))


def test_2_32_sums_of_shared_decays(gpu):
    """Decays of three channels that cross channel tiles: their sums have a kernel of their own."""
    width, heads, length = 66, 22, 256
    seqs = (1 << 32) // heads // length + 1
    x = torch.zeros(seqs, length, width, dtype=torch.float16, device=gpu)
    x[:, 0] = 1  # h = 1 throughout
    g = torch.zeros(seqs, length, heads, dtype=torch.float16, device=gpu)
    states = lx.laplex_recur(x, g, keep=True).states
    dy = x.flip(1)  # u = 1 throughout
    dg = lx.laplex_recur_backward(x, g, dy, states, want=("dg",))["dg"]
    assert all(bool((p[:, 1:] == 3).all()) and bool((p[:, 0] == 0).all()) for p in dg.split(1 << 14))


def test_step_of_2_32_channels(gpu):
    n, width = (1 << 32) // 3 + 7, 3
    x = small_values(n, width, torch.bfloat16, gpu)
    g = torch.zeros(n, 1, dtype=torch.bfloat16, device=gpu)
    state = torch.ones(n, width, device=gpu)
    y = lx.laplex_recur_step(x, g, state)
    assert all(torch.equal(s, p.float() + 1) for s, p in zip(state.split(1 << 26), x.split(1 << 26)))
    assert all(torch.equal(q, (p.float() + 1).bfloat16()) for q, p in zip(y.split(1 << 26), x.split(1 << 26)))
