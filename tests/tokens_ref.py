"""Plain float64 forms of the token operators, with bounds on what float32
arithmetic may add to them (first-order error analysis, carried along)."""
import torch

U32 = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}


def d(t):
    return t.detach().cpu().double()


def assert_within(got, ref, err):
    """|got - ref| <= err before the store, and one rounding to got's type."""
    u, tiny = U[got.dtype], TINY[got.dtype]
    got = d(got)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert torch.isfinite(got).all()
    over = (got - ref).abs() - (err + u * (ref.abs() + err) + tiny)
    assert got.numel() == 0 or float(over.max()) <= 0, float(over.max())


def route(ids, experts):
    """order, place, offsets of a stable sort of [tokens, slots] ids."""
    flat = ids.reshape(-1).tolist()
    order = [s for e in range(experts) for s in range(len(flat)) if flat[s] == e]
    place = [-1] * len(flat)
    for r, s in enumerate(order):
        place[s] = r
    offsets = [0] + [0] * experts
    for e in range(experts):
        offsets[e + 1] = offsets[e] + flat.count(e)
    order += [-1] * (len(flat) - len(order))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return i32(order), i32(place).reshape(ids.shape), i32(offsets)


def combine(place, ys, weights):
    """(y, error bound) in float64."""
    ys, place = d(ys), place.cpu().long()
    t, k = place.shape
    w = torch.ones(t, k, dtype=torch.float64) if weights is None else d(weights)
    y = torch.zeros(t, ys.shape[1], dtype=torch.float64)
    m = torch.zeros_like(y)
    for i in range(t):
        for j in range(k):
            if place[i, j] >= 0:
                y[i] += w[i, j] * ys[place[i, j]]
                m[i] += (w[i, j] * ys[place[i, j]]).abs()
    return y, (k + 1) * U32 * m


def combine_backward(place, dy, ys, weights):
    """((dys, 0), (dw, bound)) in float64."""
    dy, ys, w, place = d(dy), d(ys), d(weights), place.cpu().long()
    dys, dw, m = torch.zeros_like(ys), torch.zeros_like(w), torch.zeros_like(w)
    for i in range(place.shape[0]):
        for j in range(place.shape[1]):
            r = place[i, j]
            if r >= 0:
                dys[r] = w[i, j] * dy[i]
                dw[i, j] = (dy[i] * ys[r]).sum()
                m[i, j] = (dy[i] * ys[r]).abs().sum()
    return (dys, U32 * dys.abs()), (dw, (dy.shape[1] + 2) * U32 * m)


class Recur:
    """The recurrence on rows x [n, width], decays' logarithms g [n, heads],
    over sequences offsets (a list), with its gradients when dy is given.

    Bounds: a float32 decay is off by (1.5 |g| + 2) u (its exponent's rounding
    and the exponential's ulp), each step adds two roundings, and composing
    maps out of order adds one per row: (6 + 2 |g|) u of the sum of absolute
    terms at each row, carried on by the decays."""

    def __init__(self, x, g, offsets, h0=None, dy=None, dfinal=None):
        x, g = d(x).reshape(-1, x.shape[-1]), d(g).reshape(-1, g.shape[-1])
        n, width = x.shape
        heads = g.shape[1]
        per = width // heads
        seqs = len(offsets) - 1
        new = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
        h0 = new(seqs, width) if h0 is None else d(h0)
        self.y, ey = new(n, width), new(n, width)
        self.final, self.efinal = h0.clone(), new(seqs, width)
        prev, mprev, eprev = new(n, width), new(n, width), new(n, width)
        spread = lambda row: row.repeat_interleave(per)  # noqa: E731
        for q in range(seqs):
            h, m, e = h0[q], h0[q].abs(), new(width)
            for t in range(offsets[q], offsets[q + 1]):
                prev[t], mprev[t], eprev[t] = h, m, e
                gt = spread(g[t])
                a = gt.exp()
                cut = a.float() == 0  # forgotten, whatever it held
                h = torch.where(cut, x[t], a * h + x[t])
                m = torch.where(cut, x[t].abs(), a * m + x[t].abs())
                k = torch.where(cut, 0.0, 6 + 2 * gt.abs().clamp(max=200))
                e = torch.where(cut, 0.0, a * e) + k * U32 * m
                self.y[t], ey[t] = h, e
                self.final[q], self.efinal[q] = h, e
        self.ey = ey
        if dy is None:
            return
        dy = d(dy).reshape(n, width)
        self.dx, self.edx = new(n, width), new(n, width)
        self.dg, self.edg = new(n, heads), new(n, heads)
        self.dh0 = new(seqs, width) if dfinal is None else d(dfinal).clone()
        self.edh0 = new(seqs, width)
        for q in range(seqs):
            w = self.dh0[q].clone()
            m, e = w.abs(), new(width)
            for t in range(offsets[q + 1] - 1, offsets[q] - 1, -1):
                u, mu = dy[t] + w, dy[t].abs() + m
                eu = e + 2 * U32 * mu
                self.dx[t], self.edx[t] = u, eu
                gt = spread(g[t])
                a = gt.exp()
                cut = a.float() == 0
                w = torch.where(cut, 0.0, a * u)
                m = torch.where(cut, 0.0, a * mu)
                e = torch.where(cut, 0.0, a * eu + (6 + 2 * gt.abs().clamp(max=200)) * U32 * m)
                p = torch.where(cut, 0.0, w * prev[t])
                mp = torch.where(cut, 0.0, m * mprev[t])
                ep = torch.where(cut, 0.0, e * mprev[t] + m * eprev[t] + 2 * U32 * mp)
                self.dg[t] = p.reshape(heads, per).sum(1)
                self.edg[t] = (ep + per * U32 * mp).reshape(heads, per).sum(1)
                self.dh0[q], self.edh0[q] = w, e
