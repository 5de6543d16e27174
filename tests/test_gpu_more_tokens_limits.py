"""The experts' products and the matrix memory on arrays of more than 4 GiB,
and with more sequences and heads than usual."""
import pytest
import torch

from laplace_matvec_amd import laplex as lx

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def far_rows(t, pitch):
    """The rows of t, `pitch` values apart in one array."""
    n, width = t.shape[0], t[0].numel()
    wide = torch.empty(n * pitch, dtype=t.dtype, device=t.device)
    view = wide.as_strided((n, width), (pitch, 1))
    view.copy_(t.reshape(n, width))
    return view.unflatten(1, t.shape[1:]) if t.dim() == 3 else view


def test_rows_far_apart(gpu):
    n, heads, dk, dv, pitch = 3000, 2, 64, 40, 1 << 20  # 3000 rows of 2 MiB
    gen = torch.Generator(device=gpu).manual_seed(0)
    rand = lambda *s: torch.randn(*s, device=gpu, generator=gen).bfloat16()  # noqa: E731
    q, k, v, dy = rand(n, heads, dk), rand(n, heads, dk), rand(n, heads, dv), rand(n, heads, dv)
    g = -torch.rand(n, heads, device=gpu, generator=gen)
    r = lx.laplex_attend(q, k, v, g, keep=True)
    d = lx.laplex_attend_backward(q, k, v, g, dy, r.states)
    v2 = far_rows(v, pitch)
    r2 = lx.laplex_attend(q, k, v2, g, keep=True)
    assert torch.equal(r2.y, r.y)
    del v2
    q2 = far_rows(q, pitch)
    d2 = lx.laplex_attend_backward(q2, k, v, g, dy, r.states)
    assert all(torch.equal(d[name], d2[name]) for name in d)


def test_experts_rows_far_apart(gpu):
    n, pitch = 1500, 1 << 21  # 6 GiB of rows
    gen = torch.Generator(device=gpu).manual_seed(0)
    x = torch.randn(n, 96, device=gpu, generator=gen).bfloat16()
    w = torch.randn(3, 64, 96, device=gpu, generator=gen).bfloat16()
    dy = torch.randn(n, 64, device=gpu, generator=gen).bfloat16()
    at = torch.tensor([0, 700, 700, n], dtype=torch.int32, device=gpu)
    y, d = lx.laplex_experts(x, w, at), lx.laplex_experts_backward(x, w, dy, at)
    far = far_rows(x, pitch)
    d2 = lx.laplex_experts_backward(far, w, dy, at)
    assert torch.equal(lx.laplex_experts(far, w, at), y)
    assert torch.equal(d2["dw"], d["dw"]) and torch.equal(d2["dx"], d["dx"])


def test_a_step_far_into_the_pool(gpu):
    pool, dk, dv = 70000, 128, 128  # 4.6 GB of states
    state = torch.zeros(pool, 1, dk, dv, device=gpu)
    slots = torch.tensor([pool - 1, 3, pool, 65536], dtype=torch.int32, device=gpu)
    q, k, v = (torch.ones(4, 1, 128, dtype=torch.bfloat16, device=gpu) for _ in range(3))
    v *= torch.arange(1, 5, device=gpu).bfloat16().view(4, 1, 1)
    g = torch.zeros(4, 1, device=gpu)
    for times in (1, 2):
        y = lx.laplex_attend_step(q, k, v, g, state, slots=slots)
        want = torch.tensor([1.0, 2.0, 0.0, 4.0], device=gpu) * 128 * times
        assert torch.equal(y.float(), want.view(4, 1, 1).expand_as(y))
    assert bool((state[pool - 1] == 2).all()) and bool((state[65536] == 8).all()) and bool((state[3] == 4).all())
    assert not state[pool - 2].any() and not state[65537:pool - 1].any()


def test_many_short_sequences(gpu):
    """Sequences of 0 to 3 rows: running sums of the rows with decays of 1, whole numbers."""
    seqs = 40000
    lengths = torch.arange(seqs, device=gpu).remainder(4)
    offsets = torch.cat([lengths.new_zeros(1), lengths.cumsum(0)]).to(torch.int32)
    n = int(offsets[-1])
    one = torch.ones(n, 1, 8, dtype=torch.float16, device=gpu)
    g = torch.zeros(n, 1, device=gpu)
    r = lx.laplex_attend(one, one, one, g, offsets=offsets, scale=0.125, final=True, keep=True)
    place = torch.arange(n, device=gpu) - offsets[:-1].long().repeat_interleave(lengths) + 1
    assert torch.equal(r.y.float(), place.float().view(n, 1, 1).expand(n, 1, 8))
    assert torch.equal(r.final, lengths.float().view(seqs, 1, 1, 1).expand(seqs, 1, 8, 8))
    d = lx.laplex_attend_backward(one, one, one, g, one, r.states, offsets=offsets, scale=0.125, want=("dv", "dh0"))
    left = lengths.repeat_interleave(lengths) - place + 1
    assert torch.equal(d["dv"].float(), left.float().view(n, 1, 1).expand(n, 1, 8))
    assert torch.equal(d["dh0"], 0.125 * lengths.float().view(seqs, 1, 1, 1).expand(seqs, 1, 8, 8))


def test_many_heads_and_wide_states(gpu):
    """4096 heads of one value; one head of 1024 x 1024."""
    n = 70
    one = torch.ones(n, 4096, 1, device=gpu)
    g = torch.zeros(n, 4096, device=gpu)
    count = torch.arange(1, n + 1, device=gpu).float()
    assert torch.equal(lx.laplex_attend(one, one, one, g).y, count.view(n, 1, 1).expand(n, 4096, 1))
    wide = torch.ones(n, 1, 1024, dtype=torch.bfloat16, device=gpu)
    r = lx.laplex_attend(wide, wide, wide, g[:, :1].contiguous(), scale=2.0 ** -10, final=True)
    assert torch.equal(r.y.float(), count.view(n, 1, 1).expand(n, 1, 1024))
    assert torch.equal(r.final, torch.full((1, 1, 1024, 1024), float(n), device=gpu))
