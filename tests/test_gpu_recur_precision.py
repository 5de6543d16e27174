"""How far the recurrence's float32 results are from float64, against a plain
float32 loop over the rows."""
import pytest
import torch

from laplace_matvec_amd import laplex as lx

pytestmark = pytest.mark.gpu


def loop(x, a, dy, h0, dfinal):
    """[seqs, rows, width] in x's type, row by row: y, final, dx, dh0."""
    h, w = h0.clone(), dfinal.clone()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    for t in range(x.shape[1]):
        h = a[:, t] * h + x[:, t]
        y[:, t] = h
    for t in reversed(range(x.shape[1])):
        dx[:, t] = dy[:, t] + w
        w = a[:, t] * dx[:, t]
    return dict(y=y, final=h, dx=dx, dh0=w)


# few tiles and many, shared decays and own ones; a memory of some 2 to 1000 rows by channel
@pytest.mark.parametrize("seqs,n,width,per", [(3, 259, 520, 40), (3, 259, 520, 1), (4, 2048, 1024, 1), (4, 2048, 2048, 64),
                                              (2, 1000, 66, 3)])
def test_as_close_as_a_float32_loop(gpu, seqs, n, width, per):
    gen = torch.Generator(device=gpu).manual_seed(n + per)
    rand = lambda *s: torch.randn(*s, device=gpu, generator=gen)  # noqa: E731
    x, dy, h0, dfinal = rand(seqs, n, width), rand(seqs, n, width), rand(seqs, width), rand(seqs, width)
    heads = width // per
    rate = torch.rand(heads, device=gpu, generator=gen) * 6.2 + 0.7  # e^-0.7 to e^-6.9 a row
    g = -torch.exp(-rate + 0.5 * rand(seqs, n, heads))
    r = lx.laplex_recur(x, g, h0=h0, final=True, keep=True)
    d = lx.laplex_recur_backward(x, g, dy, r.states, h0=h0, dfinal=dfinal)
    got = dict(y=r.y, final=r.final, dx=d["dx"], dh0=d["dh0"])
    plain = loop(x, torch.exp(g).repeat_interleave(per, 2), dy, h0, dfinal)
    exact = loop(*(t.double() for t in (x, torch.exp(g.double()).repeat_interleave(per, 2), dy, h0, dfinal)))
    off = lambda t, k: float((t.double() - exact[k]).norm() / exact[k].norm())  # noqa: E731
    for k in exact:
        # Both round an exponential, a product and a sum for each row; the hardware's exponential is
        # off by an ulp where the library's is by half of one: sqrt((4 + 1 + 1) / (1 + 1 + 1)) = 1.42
        assert off(got[k], k) < 1.5 * off(plain[k], k), (k, off(got[k], k), off(plain[k], k))
