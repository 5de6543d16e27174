"""Plain float64 forms of the experts' products and the gated matrix memory,
with bounds on what the kernels' arithmetic may add to them.

Bounds.  A float32 sum of m products is off by at most (m + 2) 2^-23 of the
sum of their absolute values (an addition inside a matrix instruction may be
cut rather than rounded: 2^-23 instead of 2^-24).  The absolute sums are the
formulas themselves with absolute values for inputs.  A decay e^G is made from
an exponent that is off by 2^-23 of itself and an exponential that is off by
2^-23, so its terms count (1 + |G|) times."""
import torch

U32 = 2.0 ** -23


def d(t):
    return None if t is None else t.detach().cpu().double()


def experts(x, w, offsets, transpose=False, dy=None):
    """(y, bound), and with dy (dx, bound), (dw, bound)."""
    x, w, dy = d(x), d(w), d(dy)
    w = w if transpose else w.transpose(1, 2)  # [experts][in][out]
    y, my = x.new_zeros(x.shape[0], w.shape[2]), x.new_zeros(x.shape[0], w.shape[2])
    dx, mx, dw, mw = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(w)
    for e in range(w.shape[0]):
        at = slice(offsets[e], offsets[e + 1])
        y[at], my[at] = x[at] @ w[e], (w.shape[1] + 2) * U32 * (x[at].abs() @ w[e].abs())
        if dy is not None:
            dx[at] = dy[at] @ w[e].t()
            mx[at] = (w.shape[2] + 2) * U32 * (dy[at].abs() @ w[e].abs().t())
            dw[e] = x[at].t() @ dy[at]
            mw[e] = (at.stop - at.start + 2) * U32 * (x[at].abs().t() @ dy[at].abs())
    if dy is None:
        return y, my
    if not transpose:
        dw, mw = dw.transpose(1, 2), mw.transpose(1, 2)
    return (y, my), (dx, mx), (dw, mw)


def _spread(t, heads):
    """[rows, some heads, ...] as [heads, rows, ...]."""
    return t.repeat_interleave(heads // t.shape[1], 1).transpose(0, 1)


def _gather(t, heads):
    """Gradients [heads, rows, width] summed over the heads that share one: [rows, some heads, width]."""
    return t.unflatten(0, (heads, -1)).sum(1).transpose(0, 1)


def _attend(q, k, v, g, offsets, h0, scale, dy, dfinal, weigh):
    """All results by the sums over earlier rows; with weigh a decay e^G counts 1 + |G| times, and dg is the sum of
    all absolute terms that its computation goes through (all pairs of the row's chunk too)."""
    n, heads = g.shape
    seqs, dk, dv = len(offsets) - 1, q.shape[-1], v.shape[-1]
    hq, hk, hv = q.shape[1], k.shape[1], v.shape[1]
    q, k, v, g = _spread(q, heads) * scale, _spread(k, heads), _spread(v, heads), g.t()
    y = torch.zeros(n, heads, dv, dtype=torch.float64)
    final = torch.zeros(seqs, heads, dk, dv, dtype=torch.float64) if h0 is None else h0.clone()
    first = final.clone()
    train = dy is not None
    dq, dkey, dval = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg = torch.zeros(n, heads, dtype=torch.float64)
    last = torch.zeros_like(final) if dfinal is None else dfinal
    dh0 = last.clone()
    if train:
        dy = dy.transpose(0, 1)
    for s in range(seqs):
        a, b = offsets[s], offsets[s + 1]
        if a == b:
            continue
        m = b - a
        qs, ks, vs, gs = q[:, a:b], k[:, a:b], v[:, a:b], g[:, a:b]
        cut = gs.float().exp() == 0
        group = cut.cumsum(-1)
        total = gs.masked_fill(cut, 0.0).cumsum(-1)

        def decay(exponent, alive):
            x = torch.where(alive, exponent, 0.0)
            return torch.where(alive, x.exp() * (1 + x.abs() if weigh else 1), 0.0)

        late = torch.ones(m, m, dtype=torch.bool).triu(1)
        w = decay(total[:, :, None] - total[:, None, :], (group[:, :, None] == group[:, None, :]) & ~late)
        into = decay(total, group == 0)
        left = decay(total[:, -1:] - total, group == group[:, -1:])
        p = w * (qs @ ks.transpose(1, 2))
        y[a:b] = (p @ vs + into[..., None] * (qs @ first[s])).transpose(0, 1)
        final[s] = (ks * left[..., None]).transpose(1, 2) @ vs + into[:, -1, None, None] * first[s]
        if not train:
            continue
        ds = dy[:, a:b]
        dp = ds @ vs.transpose(1, 2)
        pair = p * dp
        from_first = into[..., None] * (ds @ first[s].transpose(1, 2))
        to_last = left[..., None] * (vs @ last[s].transpose(1, 2))
        dq[:, a:b] = (w * dp) @ ks + from_first
        dkey[:, a:b] = (w * dp).transpose(1, 2) @ qs + to_last
        dval[:, a:b] = p.transpose(1, 2) @ ds + left[..., None] * (ks @ last[s])
        dh0[s] = (qs * into[..., None]).transpose(1, 2) @ ds + into[:, -1, None, None] * last[s]
        # pairs i >= t > j: rows from t on, then columns before t
        cross = pair.flip(1).cumsum(1).flip(1).cumsum(2)
        over = torch.zeros(heads, m, dtype=torch.float64)
        over[:, 1:] = cross.diagonal(-1, 1, 2)
        after = (qs * from_first).sum(-1).flip(-1).cumsum(-1).flip(-1)
        before = (ks * to_last).sum(-1)
        before = before.cumsum(-1) - before
        through = into[:, -1] * (first[s] * last[s]).sum((1, 2))
        grad = over + after + before + through[:, None]
        if weigh:
            for c in range(0, m, 64):
                grad[:, c:c + 64] += pair[:, c:c + 64, c:c + 64].sum((1, 2))[:, None]
        dg[a:b] = grad.masked_fill(cut, 0.0).t()
    return dict(y=y, final=final, dq=_gather(dq, hq) * scale, dk=_gather(dkey, hk), dv=_gather(dval, hv), dg=dg, dh0=dh0)


def attend(q, k, v, g, offsets, h0=None, scale=1.0, dy=None, dfinal=None):
    """{name: (value, bound)}.

    With bfloat16 rows scores (and states for y) are rounded once (2^-8), which
    reaches y, dq, dk and dv; states for gradients keep two terms, what is
    left of the second is 2^-16 of the value, rows times decays at least as
    many, and at most two such values meet in a result.  Float32 sums: over dk or dv, over 64 rows, over a row's chunks
    (three roundings each), and sums of at most 16 lanes and 8 partial
    results (planes of blocks, shared heads)."""
    kind = q.dtype
    args = [d(t) for t in (q, k, v, g)]
    h0, dy, dfinal = d(h0), d(dy), d(dfinal)
    value = _attend(*args, offsets, h0, scale, dy, dfinal, False)
    absolute = lambda t: None if t is None else t.abs()  # noqa: E731
    size = _attend(args[0].abs(), args[1].abs(), args[2].abs(), args[3], offsets, absolute(h0), abs(scale), absolute(dy),
                   absolute(dfinal), True)
    n, dk, dv = g.shape[0], q.shape[-1], v.shape[-1]
    c32 = (2 * dk + 2 * dv + 128 + 3 * (n // 64 + 1) + 32) * U32
    state = c32 + (2.0 ** -15 if kind == torch.bfloat16 else 0.0)
    score = state + (2.0 ** -8 if kind == torch.bfloat16 else 0.0)
    return {name: (x, (score if name in ("y", "dq", "dk", "dv") else state) * size[name]) for name, x in value.items()}


def attend_step(q, k, v, g, state, slots, scale):
    """(y, bound), (state, bound)."""
    n, heads = g.shape
    dk = q.shape[-1]
    q, k, v = (_spread(d(t), heads).transpose(0, 1) for t in (q, k, v))
    g, state = d(g), d(state).clone()
    y, ms = torch.zeros(n, heads, v.shape[-1], dtype=torch.float64), torch.zeros_like(state)
    my = torch.zeros_like(y)
    for i in range(n):
        s = slots[i]
        if not 0 <= s < state.shape[0]:
            continue
        a = torch.where(g[i].float().exp() == 0, 0.0, g[i].exp())[:, None, None]
        new = k[i][:, :, None] * v[i][:, None, :]
        ms[s] = (4 + 2 * g[i].abs().clamp(max=200))[:, None, None] * U32 * (torch.where(a == 0, 0.0, a * state[s].abs()) + new.abs())
        state[s] = torch.where(a == 0, 0.0, a * state[s]) + new
        y[i] = scale * (q[i][:, :, None] * state[s]).sum(1)
        my[i] = abs(scale) * (q[i].abs()[:, :, None] * (ms[s] + (dk + 4) * U32 * state[s].abs())).sum(1)
    return (y, my), (state, ms)
