"""The experts' products and the matrix memory through the C entry points, where rows, results, matrices and scratch
lie further than 32 bits from the start of their arrays."""
import pytest
import torch

from laplace_matvec_amd import laplex as lx

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def ok(status):
    torch.cuda.synchronize()
    assert status == 0, lx.load().laplex_last_error()


def test_many_rows_of_no_sequence(gpu):
    """2^25 rows before the only sequence, 512 heads of one value: 2^31 places of a workgroup's column block."""
    outside, rows, heads = 1 << 25, 64, 512
    n = outside + rows
    one = torch.ones(n, 1, dtype=torch.bfloat16, device=gpu)
    g = torch.zeros(n, heads, dtype=torch.bfloat16, device=gpu)  # 34 GB, and y
    y = torch.ones(n, heads, dtype=torch.bfloat16, device=gpu)
    at = torch.tensor([outside, n], dtype=torch.int32, device=gpu)
    p = lambda t: t.data_ptr()  # noqa: E731
    lib = lx.load()
    assert lib.laplex_attend_workspace(n, 1, heads, 1, 1, 1, 1, 1, 1, 0) == 0
    ok(lib.laplex_attend(n, 1, p(at), heads, 1, 1, 1, 1, 1, 1, 1, 1.0, p(one), 1, p(one), 1, p(one), 1, p(g), heads, None,
                         p(y), heads, None, None, None, 0, torch.cuda.current_stream().cuda_stream))
    assert not y[:outside].any()
    count = torch.arange(1, rows + 1, device=gpu).view(rows, 1).expand(rows, heads)
    assert torch.equal(y[outside:].float(), count.float())


def far(t, pitch):
    """The rows of t (its first dimension), `pitch` values apart: a view [rows, values]."""
    width = t[0].numel()
    wide = torch.empty((t.shape[0] - 1) * pitch + width, dtype=t.dtype, device=t.device)
    view = wide.as_strided((t.shape[0], width), (pitch, 1))
    view.copy_(t.reshape(t.shape[0], width))
    return view


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("dtype,kind", [(torch.float32, 0), (torch.bfloat16, 1)])
@pytest.mark.parametrize("transpose", [0, 1])
@pytest.mark.parametrize("inner,outer,wide", [
    (96, 64, 1),      # whole vectors, small tiles
    (91, 67, 0),      # odd widths and pitches
    (264, 3008, 1),   # tiles of 128
])
def test_experts_far_apart(gpu, dtype, kind, transpose, inner, outer, wide):
    """Rows of x, dy, y and dx 8 MiB apart (6 GiB and more each), matrices and their gradients 2 GiB apart, against the
    same values next to each other, bit for bit."""
    size = dtype.itemsize
    n, experts, pitch = 900, 4, (1 << 23) // size + (0 if wide else 1)
    pitch_w = (1 << 31) // size + (0 if wide else 3)
    gen = torch.Generator(device=gpu).manual_seed(0)
    rand = lambda *s: torch.randn(*s, device=gpu, generator=gen).to(dtype)  # noqa: E731
    x, dy, w = rand(n, inner), rand(n, outer), rand(experts, *((inner, outer) if transpose else (outer, inner)))
    at = torch.tensor([0, 200, 200, 500, n], dtype=torch.int32, device=gpu)
    y = lx.laplex_experts(x, w, at, transpose=bool(transpose))
    d = lx.laplex_experts_backward(x, w, dy, at, transpose=bool(transpose))
    fx, fdy, fw = far(x, pitch), far(dy, pitch), far(w, pitch_w)
    fy, fdx, fdw = far(torch.zeros_like(y), pitch), far(torch.zeros_like(x), pitch), far(torch.zeros_like(w), pitch_w)
    lib, p, ldw = lx.load(), lambda t: t.data_ptr(), w.shape[2]
    ok(lib.laplex_experts(n, experts, p(at), inner, outer, kind, transpose, p(fx), pitch, p(fw), ldw, pitch_w, p(fy), pitch,
                          stream()))
    ok(lib.laplex_experts_backward(n, experts, p(at), inner, outer, kind, transpose, p(fx), pitch, p(fw), ldw, pitch_w,
                                   p(fdy), pitch, p(fdx), pitch, p(fdw), ldw, pitch_w, stream()))
    assert torch.equal(fy, y) and torch.equal(fdx, d["dx"]) and torch.equal(fdw, d["dw"].flatten(1))


@pytest.mark.parametrize("rows_apart", [(1 << 14) + 8, 1 << 14])
def test_matrix_rows_far_apart(gpu, rows_apart):
    """One expert's matrix of 140000 rows 32 KiB apart, 4.6 GB, read and written by the larger tiles' loads to LDS and
    stores: whole numbers throughout, each its row's and column's."""
    n, inner, outer = 300, 64, 140000
    one = torch.zeros(n, inner, dtype=torch.bfloat16, device=gpu)
    one[torch.arange(n), torch.arange(n) % inner] = 1.0
    wide = torch.empty((outer - 1) * rows_apart + inner, dtype=torch.bfloat16, device=gpu)
    w = wide.as_strided((1, outer, inner), (outer * rows_apart, rows_apart, 1))
    value = (torch.arange(outer, device=gpu) % 251).view(-1, 1) + (torch.arange(inner, device=gpu) % 5).view(1, -1)
    w.copy_(value.to(torch.bfloat16)[None])
    at = torch.tensor([0, n], dtype=torch.int32, device=gpu)
    y = lx.laplex_experts(one, w, at)
    assert torch.equal(y, w[0].t()[torch.arange(n) % inner])
    # dw = dy^T x: the n-th row of x picks a column, each column is picked by rows r, r + 64, ...
    dy = torch.zeros(n, outer, dtype=torch.bfloat16, device=gpu)
    dy[:inner] = w[0].t()
    w.zero_()
    p = lambda t: t.data_ptr()  # noqa: E731
    ok(lx.load().laplex_experts_backward(n, 1, p(at), inner, outer, 1, 0, p(one), inner, None, inner, 0, p(dy), outer, None,
                                         inner, p(w), rows_apart, 0, stream()))
    assert torch.equal(w[0], value.to(torch.bfloat16))


@pytest.mark.parametrize("dtype,kind", [(torch.float32, 0), (torch.bfloat16, 1)])
@pytest.mark.parametrize("dk,dv,odd", [(64, 40, 0), (33, 70, 1), (136, 24, 0)])
def test_memory_rows_far_apart(gpu, dtype, kind, dk, dv, odd):
    """Every array of rows spread over more than 4 GiB, against the same values next to each other, bit for bit."""
    n, heads, hk, hv = 1100, 4, 2, 1
    gen = torch.Generator(device=gpu).manual_seed(1)
    rand = lambda *s: torch.randn(*s, device=gpu, generator=gen).to(dtype)  # noqa: E731
    q, k, v, dy = rand(n, hk, dk), rand(n, hk, dk), rand(n, hv, dv), rand(n, heads, dv)
    g = -torch.rand(n, heads, device=gpu, generator=gen)
    r = lx.laplex_attend(q, k, v, g, scale=0.5, final=True, keep=True)
    d = lx.laplex_attend_backward(q, k, v, g, dy, r.states, scale=0.5)
    pitch, pitch_g = (1 << 22) // dtype.itemsize + odd, (1 << 20) + odd  # 4 MiB, 1100 of them
    fq, fk, fv, fdy = (far(t, pitch) for t in (q, k, v, dy))
    fg = far(g, pitch_g)
    fy, dq, dk_, dv_ = (far(torch.zeros_like(t), pitch) for t in (r.y, q, k, v))
    dg, final, dh0 = far(torch.zeros_like(g), pitch_g), torch.zeros_like(r.final), torch.zeros_like(r.final)
    lib, p = lx.load(), lambda t: t.data_ptr()
    sizes = (heads, hk, hk, hv, dk, dv)
    ws = torch.empty(max(lib.laplex_attend_workspace(n, 1, *sizes, kind, b) for b in (0, 1)) // 4 + 1, device=gpu)
    states = torch.empty(lib.laplex_attend_states(n, 1, heads, dk, dv), device=gpu)
    rows = (p(fq), pitch, p(fk), pitch, p(fv), pitch, p(fg), pitch_g, None)
    ok(lib.laplex_attend(n, 1, None, *sizes, kind, 0, 0.5, *rows, p(fy), pitch, p(final), p(states), p(ws), ws.numel() * 4,
                         stream()))
    ok(lib.laplex_attend_backward(n, 1, None, *sizes, kind, 0, 0.5, *rows, p(states), p(fdy), pitch, None, p(dq), pitch,
                                  p(dk_), pitch, p(dv_), pitch, p(dg), pitch_g, p(dh0), p(ws), ws.numel() * 4, stream()))
    assert torch.equal(fy, r.y.flatten(1)) and torch.equal(final, r.final) and torch.equal(dg, d["dg"])
    for a, name in ((dq, "dq"), (dk_, "dk"), (dv_, "dv")):
        assert torch.equal(a, d[name].flatten(1)), name
    assert torch.equal(dh0, d["dh0"])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scratch_past_4_gib(gpu, dtype):
    """Two equal sequences whose chunks' states and gradients take 4.7 GB each, against one of them alone (half the
    scratch, the same segments): bit for bit."""
    rows, heads, dim = 150016, 16, 128  # 2344 chunks of 1 MiB
    gen = torch.Generator(device=gpu).manual_seed(2)
    rand = lambda: torch.randn(rows, heads, dim, device=gpu, generator=gen, dtype=torch.bfloat16)  # noqa: E731
    q, k, v, dy = (rand().to(dtype) for _ in range(4))
    g = -torch.rand(rows, heads, device=gpu, generator=gen)
    r = lx.laplex_attend(q, k, v, g, scale=0.125, final=True, keep=True)
    d = lx.laplex_attend_backward(q, k, v, g, dy, r.states, scale=0.125)
    q, k, v, dy, g = (torch.stack([t, t]) for t in (q, k, v, dy, g))
    kind = 0 if dtype is torch.float32 else 1
    assert lx.load().laplex_attend_workspace(2 * rows, 2, heads, heads, heads, heads, dim, dim, kind, 1) > 9 << 30
    r2 = lx.laplex_attend(q, k, v, g, scale=0.125, final=True, keep=True)
    assert all(torch.equal(r2.y[i], r.y) and torch.equal(r2.final[i], r.final[0]) for i in (0, 1))
    d2 = lx.laplex_attend_backward(q, k, v, g, dy, r2.states, scale=0.125)
    for name in d:
        for i in (0, 1):
            assert torch.equal(d2[name][i], d[name][0] if name == "dh0" else d[name]), name
