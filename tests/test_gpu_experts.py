"""Experts' products against float64, at the sizes and layouts where they can go wrong."""
import pytest
import torch

import more_tokens_ref as ref
from laplace_matvec_amd import laplex as lx
from tokens_ref import assert_within

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def make(gpu, dtype, counts, inner, outer, transpose, before=0, past=0, seed=0):
    """x, w, dy and offsets (a list): counts rows for each expert, with rows of no expert around them."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen).to(dtype).to(gpu)  # noqa: E731
    offsets = [before]
    for c in counts:
        offsets.append(offsets[-1] + c)
    n = offsets[-1] + past
    shape = (len(counts), inner, outer) if transpose else (len(counts), outer, inner)
    return rand(n, inner), rand(*shape), rand(n, outer), offsets


def on(gpu, offsets):
    return torch.tensor(offsets, dtype=torch.int32, device=gpu)


def check(x, w, dy, offsets, transpose, gpu):
    at = on(gpu, offsets)
    y, dx, dw = ref.experts(x, w, offsets, transpose, dy)
    assert_within(lx.laplex_experts(x, w, at, transpose=transpose), *y)
    got = lx.laplex_experts_backward(x, w, dy, at, transpose=transpose)
    assert_within(got["dx"], *dx)
    assert_within(got["dw"], *dw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("counts", [[1], [0, 1, 0], [5, 0, 64, 65, 1, 0], [200, 3], [1] * 70, [0, 0, 700]])
def test_counts(gpu, dtype, transpose, counts):
    check(*make(gpu, dtype, counts, 72, 136, transpose), transpose, gpu)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("inner,outer", [(1, 1), (1, 300), (300, 1), (7, 9), (64, 64), (8, 257), (129, 250), (512, 256),
                                         (250, 520), (1000, 72)])
def test_widths(gpu, dtype, transpose, inner, outer):
    check(*make(gpu, dtype, [3, 40, 0, 90], inner, outer, transpose, seed=inner), transpose, gpu)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("rows", [16, 130, 600])
def test_rows_of_no_expert(gpu, dtype, transpose, rows):
    """Rows before the first expert's and past the last give 0 and are not used, whatever they hold."""
    x, w, dy, offsets = make(gpu, dtype, [rows, 0, 2 * rows], 96, 80, transpose, before=67, past=131)
    for t in (x, dy):
        t[:67] = float("nan")
        t[offsets[-1]:] = float("inf")
    at = on(gpu, offsets)
    clean = [t.clone() for t in (x, dy)]
    for t in clean:
        t[:67] = 0
        t[offsets[-1]:] = 0
    y, dx, dw = ref.experts(clean[0], w, offsets, transpose, clean[1])
    assert_within(lx.laplex_experts(x, w, at, transpose=transpose), *y)
    got = lx.laplex_experts_backward(x, w, dy, at, transpose=transpose)
    assert_within(got["dx"], *dx)
    assert_within(got["dw"], *dw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("counts", [[3, 2, 0, 4], [150, 70, 0, 300]])
def test_a_row_reaches_its_own_results_alone(gpu, dtype, transpose, counts):
    x, w, dy, offsets = make(gpu, dtype, counts, 128, 192, transpose)
    at = on(gpu, offsets)
    y0 = lx.laplex_experts(x, w, at, transpose=transpose)
    g0 = lx.laplex_experts_backward(x, w, dy, at, transpose=transpose)
    row = offsets[1]  # the second expert's first
    x[row, 5], dy[row, 7] = float("inf"), float("nan")
    y = lx.laplex_experts(x, w, at, transpose=transpose)
    g = lx.laplex_experts_backward(x, w, dy, at, transpose=transpose)
    others = torch.arange(x.shape[0], device=gpu) != row
    assert torch.equal(y[others], y0[others]) and not torch.isfinite(y[row]).any()
    assert torch.equal(g["dx"][others], g0["dx"][others]) and torch.isnan(g["dx"][row]).all()
    keep = [0, 2, 3]
    assert torch.equal(g["dw"][keep], g0["dw"][keep]) and not torch.isfinite(g["dw"][1]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("counts", [[2, 5], [100, 260]])
def test_strided_and_unaligned(gpu, dtype, transpose, shift, counts):
    """Rows that are parts of wider ones, from any value on; matrices with pitches of their own."""
    x, w, dy, offsets = make(gpu, dtype, counts, 136, 72, transpose)
    y0 = lx.laplex_experts(x, w, on(gpu, offsets), transpose=transpose)
    g0 = lx.laplex_experts_backward(x, w, dy, on(gpu, offsets), transpose=transpose)

    def inside(t, extra):
        wide = torch.full((*t.shape[:-1], t.shape[-1] + extra), float("nan"), dtype=t.dtype, device=gpu)
        view = wide[..., shift:shift + t.shape[-1]]
        view.copy_(t)
        return view

    x2, dy2, w2 = inside(x, 11), inside(dy, 24), inside(w, 5)
    # experts between each other's rows
    w3 = torch.empty(w.shape[1], w.shape[0], w.shape[2], dtype=dtype, device=gpu).transpose(0, 1).copy_(w)
    for m in (w2, w3):
        assert torch.equal(lx.laplex_experts(x2, m, on(gpu, offsets), transpose=transpose), y0)
        g = lx.laplex_experts_backward(x2, m, dy2, on(gpu, offsets), transpose=transpose)
        assert torch.equal(g["dx"], g0["dx"]) and torch.equal(g["dw"], g0["dw"])


@pytest.mark.parametrize("dtype", TYPES)
def test_one_matrix_for_all(gpu, dtype):
    x, w, _, offsets = make(gpu, dtype, [30, 0, 70], 64, 48, False)
    one = w[:1].expand(3, -1, -1)
    assert torch.equal(lx.laplex_experts(x, one, on(gpu, offsets)), lx.laplex_experts(x, one.contiguous(), on(gpu, offsets)))


@pytest.mark.parametrize("dtype", TYPES)
def test_no_rows(gpu, dtype):
    x, w, dy, offsets = make(gpu, dtype, [0, 0], 24, 40, False)
    assert lx.laplex_experts(x, w, on(gpu, offsets)).shape == (0, 40)
    g = lx.laplex_experts_backward(x, w, dy, on(gpu, offsets))
    assert g["dx"].shape == (0, 24) and not g["dw"].any()


@pytest.mark.parametrize("dtype", TYPES)
def test_wanted_gradients_only(gpu, dtype):
    x, w, dy, offsets = make(gpu, dtype, [30, 70], 64, 48, False)
    both = lx.laplex_experts_backward(x, w, dy, on(gpu, offsets))
    for name in ("dx", "dw"):
        one = lx.laplex_experts_backward(x, w, dy, on(gpu, offsets), want=(name,))
        assert list(one) == [name] and torch.equal(one[name], both[name])


def test_offsets_out_of_range(gpu):
    """Offsets are cut to the rows there are; nothing else is touched."""
    x, w, dy, _ = make(gpu, torch.bfloat16, [100, 100], 64, 64, False)
    wild = on(gpu, [-50, 100, 10 ** 9])
    want = lx.laplex_experts(x, w, on(gpu, [0, 100, 200]))
    assert torch.equal(lx.laplex_experts(x, w, wild), want)
    g, g0 = (lx.laplex_experts_backward(x, w, dy, o) for o in (wild, on(gpu, [0, 100, 200])))
    assert torch.equal(g["dw"], g0["dw"]) and torch.equal(g["dx"], g0["dx"])


@pytest.mark.parametrize("dtype", TYPES)
def test_gradients_against_differences(gpu, dtype):
    """<dL/dx, u> for L = <y, c> against (L(x + u) - L(x - u)) / 2: L is linear in x and in w, so the difference is the
    gradient itself, up to roundings (float64 sums of the kernels' y)."""
    x, w, c, offsets = make(gpu, dtype, [40, 0, 90], 96, 56, False)
    at = on(gpu, offsets)
    _, dx, dw = ref.experts(x, w, offsets, False, c)
    g = lx.laplex_experts_backward(x, w, c, at)
    u = torch.randn(x.shape, generator=torch.Generator().manual_seed(9)).to(dtype).to(gpu)
    m = torch.randn(w.shape, generator=torch.Generator().manual_seed(8)).to(dtype).to(gpu)
    half = torch.finfo(dtype).eps / 2

    def off(t, bound, by):  # t within its bound and one rounding, summed with `by`
        return float(((bound + half * (t.abs() + bound) + torch.finfo(dtype).tiny) * by.cpu().double().abs()).sum())

    dot = lambda a, b: float((a.cpu().double() * b.cpu().double()).sum())  # noqa: E731
    assert abs(dot(g["dx"], u) - dot(lx.laplex_experts(u, w, at), c)) <= off(*dx, u) + off(*ref.experts(u, w, offsets), c)
    assert abs(dot(g["dw"], m) - dot(lx.laplex_experts(x, m, at), c)) <= off(*dw, m) + off(*ref.experts(x, m, offsets), c)


def test_repeats_bit_for_bit_and_in_a_graph(gpu):
    x, w, dy, offsets = make(gpu, torch.bfloat16, [300, 0, 700, 25], 256, 320, False)
    at = on(gpu, offsets)

    def both():
        return lx.laplex_experts(x, w, at), lx.laplex_experts_backward(x, w, dy, at)

    y0, g0 = both()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, g = both()
    for k in range(3):
        x.mul_(-1)
        dy.mul_(2)
        graph.replay()
        torch.cuda.synchronize()
        ye, ge = both()
        assert torch.equal(y, ye) and torch.equal(g["dx"], ge["dx"]) and torch.equal(g["dw"], ge["dw"])
    assert torch.equal(ye, -y0)


def test_another_stream(gpu):
    x, w, dy, offsets = make(gpu, torch.float16, [300, 200], 128, 64, True)
    at = on(gpu, offsets)
    want, side = lx.laplex_experts(x, w, at, transpose=True), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        y = lx.laplex_experts(x, w, at, transpose=True, stream=s)
        side.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("counts,inner,outer", [
    ([1000, 0, 517, 300], 200, 5400),      # whole and broken tiles of 256, a tail of the contraction; workgroups that stay
    ([1000, 0, 517, 300], 72, 5400),       # the same where each has one tile
    ([257, 1, 700], 203, 6301),            # odd widths, by registers
    ([90, 0, 260, 41, 7, 130, 128, 150], 136, 3080),  # tiles of 128
    ([90, 0, 260, 41, 7, 130, 128, 150], 131, 3001),
])
def test_larger_tiles(gpu, dtype, transpose, counts, inner, outer):
    x, w, dy, offsets = make(gpu, dtype, counts, inner, outer, transpose, past=3)
    y, dx, _ = ref.experts(x, w, offsets, transpose, dy)
    at = on(gpu, offsets)
    assert_within(lx.laplex_experts(x, w, at, transpose=transpose), *y)
    assert_within(lx.laplex_experts_backward(x, w, dy, at, transpose=transpose, want=("dx",))["dx"], *dx)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("counts,inner,outer", [([300, 0, 517, 256], 2056, 2104), ([60, 0, 5, 33], 2056, 2104),
                                                ([300, 0, 517, 256], 2051, 2103)])
def test_larger_tiles_of_the_matrices_gradient(gpu, dtype, transpose, counts, inner, outer):
    x, w, dy, offsets = make(gpu, dtype, counts, inner, outer, transpose)
    _, _, dw = ref.experts(x, w, offsets, transpose, dy)
    assert_within(lx.laplex_experts_backward(x, w, dy, on(gpu, offsets), transpose=transpose, want=("dw",))["dw"], *dw)


def test_many_experts(gpu):
    """More experts than lanes: the largest number that routing gives, rows for some of them."""
    gen = torch.Generator().manual_seed(3)
    counts = (torch.rand(4096, generator=gen) < 0.05).int() * torch.randint(1, 40, (4096,), generator=gen)
    x, w, dy, offsets = make(gpu, torch.bfloat16, counts.tolist(), 40, 24, False)
    check(x, w, dy, offsets, False, gpu)


def test_many_experts_in_larger_tiles(gpu):
    counts = [0] * 130 + [45, 300, 0, 129] * 50
    x, w, dy, offsets = make(gpu, torch.bfloat16, counts, 40, 264, False)
    check(x, w, dy, offsets, False, gpu)


def test_offsets_past_2_31_bytes(gpu):
    """Rows, results and matrices further than 32 bits from the start of their arrays; whole numbers throughout."""
    n, width, experts = 1 << 19, 2048, 700
    x = torch.arange(n, device=gpu, dtype=torch.int32).remainder_(7).to(torch.bfloat16)[:, None].expand(n, width).contiguous()
    w = torch.zeros(experts, 8, width, dtype=torch.bfloat16, device=gpu)
    w[:, :, 0] = torch.arange(experts, device=gpu).remainder(5)[:, None].to(torch.bfloat16)
    w[:, :, width - 1] = 1
    at = torch.full((experts + 1,), n, dtype=torch.int32, device=gpu)
    at[0], at[1:experts - 1] = 0, 100  # the first expert has 100 rows, the last but one all others
    at[experts - 1] = n
    y = lx.laplex_experts(x, w, at)
    by = torch.full((n, 1), float((experts - 2) % 5 + 1), device=gpu)
    by[:100] = 1.0
    assert torch.equal(y.float(), (x[:, :1].float() * by).expand(n, 8))
    dw = lx.laplex_experts_backward(x, w, y, at, want=("dw",))["dw"]
    assert not dw[1:experts - 2].any() and not dw[experts - 1].any()
    total = (x[100:, 0].double() * y[100:, 0].double()).sum()
    assert torch.allclose(dw[experts - 2].double(), total, rtol=2.0 ** -8, atol=0)
    dx = lx.laplex_experts_backward(x, w, y, at, want=("dx",))["dx"]
    assert torch.equal(dx[:, width - 1].float(), 8 * y[:, 0].float())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("counts,inner", [([1000, 0, 517, 300], 200), ([0, 600, 2, 0, 1200], 248), ([1500, 37], 1032)])
def test_workgroups_that_take_several_tiles(gpu, dtype, transpose, counts, inner):
    """y of 9000 columns and dx of as many: 36 tiles of 256 columns by 9 row tiles of experts (with one of no expert)
    make 360, by 9 (two) 396 and by 7 (one) 288, for 256 workgroups that stay, as the contraction is at least 192.  Its
    tail is 8 of 64 (200, 1032) or 56 (248); the tile after it is loaded during the step that has it."""
    wide = 9000
    before, past = (0, 3) if counts[0] else (70, 40)
    x, w, dy, offsets = make(gpu, dtype, counts, inner, wide, transpose, before=before, past=past, seed=inner)
    at = on(gpu, offsets)
    assert_within(lx.laplex_experts(x, w, at, transpose=transpose), *ref.experts(x, w, offsets, transpose))
    # the gradient of rows of `wide` values from dy of `inner`: the same tiles by the other orientation's kernel
    w = w.transpose(1, 2).contiguous()
    _, dx, dw = ref.experts(dy, w, offsets, transpose, x)
    got = lx.laplex_experts_backward(dy, w, x, at, transpose=transpose)
    assert_within(got["dx"], *dx)
    assert_within(got["dw"], *dw)


@pytest.mark.parametrize("transpose", [False, True])
def test_bad_rows_beside_tiles_that_are_cleared(gpu, transpose):
    """The tail of a contraction is cleared in LDS while the next tile's first values arrive: rows of no expert between
    two tiles of one workgroup, and rows that hold inf and NaN, reach nothing."""
    x, w, _, offsets = make(gpu, torch.bfloat16, [1000, 0, 517, 300], 200, 9000, transpose, before=300, past=300)
    at = on(gpu, offsets)
    y0 = lx.laplex_experts(x, w, at, transpose=transpose)
    assert not y0[:300].any() and not y0[offsets[-1]:].any()
    x[:300], x[offsets[-1]:], x[700, 199] = float("nan"), float("inf"), float("inf")
    y = lx.laplex_experts(x, w, at, transpose=transpose)
    others = torch.arange(x.shape[0], device=gpu) != 700
    assert torch.equal(y[others], y0[others]) and not torch.isfinite(y[700]).any()
