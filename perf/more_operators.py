"""Cases of the experts' matrix products and of the gated matrix memory (linear attention with decays).

    experts        y_r = w[e] x_r for the rows r of each expert e (w[e]^T x_r with transpose)
    experts_train  the same with its gradients: rows and weights
    attend         S_t = exp(g_t) S_{t-1} + k_t v_t^T, y_t = scale S_t^T q_t for each head, along packed sequences
    attend_train   the same with its backward pass: gradients of q, k, v, g and the first states
    attend_step    one token for each request on a pool of states

The plain forms are elementary torch operations in 32 bits, rounded once at the end; sums of the logarithms of
decays are held in 64.
"""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


def listed():
    return [
        # one token of one request, 4 of 16 experts: latency only
        dict(name="experts token", op="experts", tokens=1, slots=4, experts=16, dropped=0.0, inner=1024, outer=512,
             transpose=False, dtype="float16"),
        # one decoding step of 64 requests, 8 of 128 experts: the weights are read once for a few rows each
        dict(name="experts decode", op="experts", tokens=64, slots=8, experts=128, dropped=0.0, inner=2048,
             outer=1536, transpose=False, dtype="bfloat16"),
        # a short prompt, 4 of 16 experts, odd sizes, the experts' second product from weights kept the other way
        dict(name="experts prompt", op="experts", tokens=391, slots=4, experts=16, dropped=0.02, inner=1000,
             outer=689, transpose=True, dtype="float16"),
        # a prefill of 16384 tokens, 2 of 8 wide experts
        dict(name="experts prefill", op="experts", tokens=16384, slots=2, experts=8, dropped=0.0, inner=4096,
             outer=4096, transpose=False, dtype="bfloat16"),
        # a training micro-batch, 4 of 64 experts, a few slots dropped
        dict(name="experts train", op="experts_train", tokens=16384, slots=4, experts=64, dropped=0.02, inner=2048,
             outer=1408, transpose=False, dtype="bfloat16"),
        # a small layer trained in full precision
        dict(name="experts train f32", op="experts_train", tokens=2048, slots=2, experts=8, dropped=0.0, inner=512,
             outer=769, transpose=False, dtype="float32"),
        # three short prompts of uneven length in one batch, narrow heads
        dict(name="attend prompts", op="attend", rows=777, seqs=3, ragged=True, heads=13, hq=13, hk=13, hv=13, dk=40,
             dv=40, dtype="float16", gates="float32", h0=True, resets=False, fused=False),
        # one long prompt of 65536 tokens
        dict(name="attend long", op="attend", rows=65536, seqs=1, ragged=False, heads=16, hq=16, hk=16, hv=16, dk=128,
             dv=128, dtype="bfloat16", gates="float32", h0=False, resets=False, fused=True),
        # packed documents of uneven length in training, queries and keys shared by groups of four heads
        dict(name="attend train packed", op="attend_train", rows=32768, seqs=24, ragged=True, heads=32, hq=8, hk=8,
             hv=32, dk=128, dv=64, dtype="bfloat16", gates="float32", h0=False, resets=True, fused=False),
        # equal sequences in full precision
        dict(name="attend train f32", op="attend_train", rows=8192, seqs=4, ragged=False, heads=8, hq=8, hk=8, hv=8,
             dk=64, dv=64, dtype="float32", gates="float32", h0=True, resets=False, fused=False),
        # one token for each of 3 requests: latency
        dict(name="step few", op="attend_step", requests=3, pool=4, heads=8, hq=8, hk=8, hv=8, dk=64, dv=64,
             dtype="bfloat16", gates="float32", idle=0.0),
        # one token for each of 256 requests out of a pool of 320 states
        dict(name="step serve", op="attend_step", requests=256, pool=320, heads=16, hq=16, hk=16, hv=16, dk=128,
             dv=128, dtype="bfloat16", gates="float32", idle=0.03),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm: a power of two or odd."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    if rng.random() < 0.35:
        return max(lo, 1 << int(math.log2(v)))
    return min(hi, int(v) | 1)


def _draw_experts(rng):
    op = rng.choice(["experts", "experts", "experts_train"])
    slots = rng.choice([1, 2, 4, 8])
    experts = max(slots, _spread(rng, 4, 256))
    inner, outer = _spread(rng, 16, 8191), _spread(rng, 16, 8191)
    if rng.random() < 0.7:  # most widths are whole vectors
        inner, outer = (inner // 8 | 1) * 8, (outer // 8 | 1) * 8
    dtype = rng.choice(["float32", "bfloat16", "bfloat16", "float16"])
    while experts * inner * outer > 1 << 28:
        experts, inner = max(slots, experts // 2), max(16, inner // 2)
    most = 2.0e11 if op == "experts_train" else 5.0e11
    tokens = _spread(rng, 1, max(1, min(16384, int(most / (2.0 * slots * inner * outer)))))
    return dict(op=op, tokens=tokens, slots=slots, experts=experts, dropped=rng.choice([0.0, 0.05]), inner=inner,
                outer=outer, transpose=rng.random() < 0.4, dtype=dtype)


def draw(rng):
    op = rng.choice(["experts", "experts", "attend", "attend", "attend_train", "attend_step"])
    if op == "experts":
        return _draw_experts(rng)
    dtype = rng.choice(["float32", "bfloat16", "bfloat16", "float16"])
    c = dict(op=op, dtype=dtype, gates=rng.choice([dtype, "float32"]))
    heads = rng.choice([1, 2, 4, 6, 8, 12, 16, 24, 32])
    shared = [h for h in (1, 2, 4, 8, heads) if heads % h == 0]
    one = rng.random() < 0.5
    c.update(heads=heads, hq=heads if one else rng.choice(shared), hk=heads if one else rng.choice(shared),
             hv=heads if one else rng.choice(shared))
    dims = [16, 24, 40, 64, 64, 80, 96, 128, 128, 192, 256]
    c.update(dk=rng.choice(dims), dv=rng.choice(dims + [7, 33]))
    size = heads * c["dk"] * c["dv"]
    if op == "attend_step":
        n = _spread(rng, 1, max(1, min(1024, (1 << 26) // size)))
        c.update(requests=n, pool=n + rng.choice([0, 1, 77]), idle=rng.choice([0.0, 0.1]))
        return c
    most = (1 << 32) if op == "attend_train" else (1 << 34)
    rows = _spread(rng, 1, min(65535, (1 << 21) // heads, max(1, most // size)))
    seqs = rng.choice([1, 1, 2, 5, 16, 63])
    ragged = rng.random() < 0.6
    if not ragged:
        rows = (rows // seqs | 1) * seqs
    c.update(rows=rows, seqs=seqs, ragged=ragged, h0=rng.random() < 0.5, resets=rng.random() < 0.3,
             fused=rng.random() < 0.3)
    return c


# ---------------------------------------------------------------- inputs

def _ends(case, gen):
    """First rows of the experts and the number of kept rows, skewed as routers are, on the host."""
    t, k, e = case["tokens"], case["slots"], case["experts"]
    u = torch.rand(t, 1, device="cuda", generator=gen)
    base = (u.pow(1.5) * e).to(torch.int64).clamp_(max=e - 1)
    ids = (base + torch.arange(k, device="cuda") * max(1, e // k)) % e
    if case["dropped"]:
        ids[torch.rand(t, k, device="cuda", generator=gen) < case["dropped"]] = e
    return [0] + torch.bincount(ids.reshape(-1), minlength=e + 1)[:e].cumsum(0).tolist()


def _offsets(case, gen):
    n, s = case["rows"], case["seqs"]
    if not case["ragged"]:
        return [i * (n // s) for i in range(s + 1)]
    cuts = sorted((torch.rand(s - 1, device="cuda", generator=gen) * n).to(torch.int64).tolist())
    if s > 4:
        cuts[2] = cuts[1]  # an empty sequence
    return [0] + cuts + [n]


def _decays(rows, heads, gen):
    """Logarithms of decays whose memory spans 2 to 1000 tokens by head, moved by each token."""
    base = torch.rand(heads, device="cuda", generator=gen) * -math.log(500.0) - math.log(2.0)
    move = torch.randn(rows, heads, device="cuda", generator=gen) * 0.5
    return -torch.exp(base + move)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    dt = DTYPES[case["dtype"]]
    normal = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
    s = {"op": op}
    if op in ("experts", "experts_train"):
        rows, e, i, o = case["tokens"] * case["slots"], case["experts"], case["inner"], case["outer"]
        ends = _ends(case, gen)
        x = normal(rows, i).to(dt)
        x[ends[-1]:] = 0  # as dispatch leaves the rows past the last kept slot
        shape = (e, i, o) if case["transpose"] else (e, o, i)
        w = torch.empty(*shape, device="cuda", dtype=dt)
        for one in w:
            one.copy_(normal(*shape[1:]) * i ** -0.5)
        s.update(x=x, w=w, ends=ends, offsets=torch.tensor(ends, dtype=torch.int32, device="cuda"),
                 transpose=case["transpose"])
        if op == "experts_train":
            s["dy"] = normal(rows, o).to(dt)
        return s
    gdt = DTYPES[case["gates"]]
    heads, dk, dv = case["heads"], case["dk"], case["dv"]
    n = case["requests"] if op == "attend_step" else case["rows"]
    parts = [case["hq"] * dk, case["hk"] * dk, case["hv"] * dv]
    if case.get("fused"):  # parts of one projection's rows
        q, k, v = normal(n, sum(parts)).to(dt).split(parts, 1)
    else:
        q, k, v = (normal(n, p).to(dt) for p in parts)
    g = _decays(n, heads, gen).to(gdt)
    s["scale"] = dk ** -0.5
    if op == "attend_step":
        slots = torch.randperm(case["pool"], device="cuda", generator=gen)[:n].to(torch.int32)
        slots[torch.rand(n, device="cuda", generator=gen) < case["idle"]] = -1  # a request without work
        return {**s, "q": q.unflatten(1, (-1, dk)), "k": k.unflatten(1, (-1, dk)), "v": v.unflatten(1, (-1, dv)),
                "g": g, "state": normal(case["pool"], heads, dk, dv), "slots": slots}
    if case["resets"]:
        g[torch.rand(n, device="cuda", generator=gen) < 0.002] = -math.inf
    seqs, ends = case["seqs"], _offsets(case, gen)
    lead = (n,) if case["ragged"] else (seqs, n // seqs)
    s.update(ends=ends, offsets=torch.tensor(ends, dtype=torch.int32, device="cuda"), ragged=case["ragged"],
             q=q.unflatten(1, (-1, dk)).unflatten(0, lead), k=k.unflatten(1, (-1, dk)).unflatten(0, lead),
             v=v.unflatten(1, (-1, dv)).unflatten(0, lead), g=g.unflatten(0, lead),
             h0=normal(seqs, heads, dk, dv) if case["h0"] else None)
    if op == "attend_train":
        s["dy"] = normal(n, heads, dv).to(dt).unflatten(0, lead)
        s["dfinal"] = normal(seqs, heads, dk, dv)
    return s


# ------------------------------------------------------------ plain forms

def _plain_experts(s):
    x, w, ends = s["x"], s["w"], s["ends"]
    o = w.shape[2] if s["transpose"] else w.shape[1]
    train = s["op"] == "experts_train"
    y = x.new_zeros(x.shape[0], o)
    dx, dw = (torch.zeros_like(x), torch.zeros_like(w)) if train else (None, None)
    for e in range(len(ends) - 1):
        at = slice(ends[e], ends[e + 1])
        if ends[e + 1] == ends[e]:
            continue
        xe, we = x[at].float(), w[e].float()
        we = we if s["transpose"] else we.t()  # [in][out]
        y[at] = (xe @ we).to(x.dtype)
        if train:
            dy = s["dy"][at].float()
            dx[at] = (dy @ we.t()).to(x.dtype)
            dw[e] = (xe.t() @ dy if s["transpose"] else dy.t() @ xe).to(w.dtype)
    return {"y": y, "dx": dx, "dw": dw} if train else y


CHUNK = 64


def _heads_of(t, heads):
    """[rows, some heads, d] in 32 bits with each head's own copy."""
    t = t.float()
    return t if t.shape[1] == heads else t.repeat_interleave(heads // t.shape[1], 1)


def _cut(t):
    """[rows, heads, ...] in pieces of CHUNK rows, zeros past the end: [pieces, heads, CHUNK, ...]."""
    n = t.shape[0]
    m = -(-n // CHUNK)
    t = torch.cat([t, t.new_zeros(m * CHUNK - n, *t.shape[1:])])
    return t.unflatten(0, (m, CHUNK)).transpose(1, 2).contiguous()


def _join(t, n):
    return t.transpose(1, 2).flatten(0, 1)[:n]


def _one_sequence(q, k, v, g, h0, dy, dfinal):
    """One sequence [rows, heads, ...] in 32 bits: pieces of CHUNK rows by masked products, states carried between."""
    n, heads, dk = q.shape
    q, k, v, g = _cut(q), _cut(k), _cut(v), _cut(g)
    cut = torch.exp(g) == 0
    at = torch.arange(CHUNK, device=q.device)
    last = torch.where(cut, at, -1).cummax(-1).values  # the last row that forgets, up to each
    total = g.double().masked_fill(cut, 0.0).cumsum(-1)
    live = (at[None, :] <= at[:, None]) & (at >= last[..., None])
    decay = torch.exp(total[..., :, None] - total[..., None, :]).masked_fill(~live, 0.0).float()
    into = torch.exp(total).masked_fill(last >= 0, 0.0).float()[..., None]
    out = torch.exp(total[..., -1:] - total).masked_fill(at < last[..., -1:], 0.0).float()[..., None]
    whole = into[..., -1:, :]
    m = q.shape[0]
    states = q.new_empty(m + 1, heads, dk, v.shape[-1])
    states[0] = 0 if h0 is None else h0
    torch.matmul((k * out).transpose(-1, -2), v, out=states[1:])
    for i in range(m):
        states[i + 1] += torch.where(whole[i] == 0, 0.0, whole[i] * states[i])
    score = q @ k.transpose(-1, -2)
    y = (score * decay) @ v + into * (q @ states[:-1])
    if dy is None:
        return _join(y, n), states[-1]
    dy = _cut(dy)
    back = torch.empty_like(states)  # gradient of the states
    back[m] = dfinal
    torch.matmul((q * into).transpose(-1, -2), dy, out=back[:-1])
    for i in reversed(range(m)):
        back[i] += torch.where(whole[i] == 0, 0.0, whole[i] * back[i + 1])
    dscore = dy @ v.transpose(-1, -2) * decay
    dq_in = into * (dy @ states[:-1].transpose(-1, -2))
    dk_out = out * (v @ back[1:].transpose(-1, -2))
    dq = dscore @ k + dq_in
    dkk = dscore.transpose(-1, -2) @ q + dk_out
    dv = (score * decay).transpose(-1, -2) @ dy + out * (k @ back[1:])
    pair = score * dscore
    here = pair.sum(-1) - pair.sum(-2) + (q * dq_in).sum(-1)
    carried = (k * dk_out).sum(-1)
    dg = here.flip(-1).cumsum(-1).flip(-1) + carried.cumsum(-1) - carried
    dg = dg + whole[..., 0] * (states[:-1] * back[1:]).sum((-1, -2))[..., None]
    dg = dg.masked_fill(cut, 0.0)
    return _join(y, n), states[-1], _join(dq, n), _join(dkk, n), _join(dv, n), _join(dg, n), back[0]


def _plain_attend(s):
    lead = s["g"].dim() - 1
    q, k, v, g = (s[name].flatten(0, lead - 1) for name in "qkvg")
    n, heads = g.shape
    train = s["op"] == "attend_train"
    seqs, dk, dv = len(s["ends"]) - 1, q.shape[-1], v.shape[-1]
    y = q.new_zeros(n, heads, dv)
    final = torch.empty(seqs, heads, dk, dv, device=q.device)
    grads = [torch.zeros(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v, g)] if train else []
    dh0 = torch.empty_like(final) if train else None
    qs, ks, vs, gs = _heads_of(q, heads), _heads_of(k, heads), _heads_of(v, heads), g.float()
    qs = qs * s["scale"]
    for i in range(seqs):
        at = slice(s["ends"][i], s["ends"][i + 1])
        h0 = None if s["h0"] is None else s["h0"][i]
        if at.start == at.stop:
            final[i] = 0 if h0 is None else h0
            if train:
                dh0[i] = s["dfinal"][i]
            continue
        args = [t[at] for t in (qs, ks, vs, gs)]
        if not train:
            r = _one_sequence(*args, h0, None, None)
            y[at], final[i] = r[0].to(y.dtype), r[1]
            continue
        r = _one_sequence(*args, h0, s["dy"].flatten(0, lead - 1)[at].float(), s["dfinal"][i])
        y[at], final[i], dh0[i] = r[0].to(y.dtype), r[1], r[6]
        for to, part, by in zip(grads, r[2:6], (s["scale"], 1.0, 1.0, 1.0)):
            to[at] = (part.unflatten(1, (to.shape[1], -1) + (() if to.dim() == 3 else (1,))).sum(2).view_as(to[at])
                      * by).to(to.dtype)
    shape = s["g"].shape[:-1]
    out = {"y": y.unflatten(0, shape), "final": final}
    if train:
        out.update({name: t.unflatten(0, shape) for name, t in zip(("dq", "dk", "dv", "dg"), grads)}, dh0=dh0)
    return out


def _plain_step(s):
    slots, state = s["slots"].long(), s["state"]
    heads = state.shape[1]
    q, k, v = _heads_of(s["q"], heads), _heads_of(s["k"], heads), _heads_of(s["v"], heads)
    a = torch.exp(s["g"].float())[..., None, None]
    h = torch.where(a == 0, 0.0, a * state[slots.clamp(min=0)]) + k[..., :, None] * v[..., None, :]
    y = (h * (q * s["scale"])[..., :, None]).sum(-2)
    # requests without work write into a row of their own past the pool
    whole = torch.cat([state, torch.zeros_like(state[:1])])
    whole[torch.where(slots >= 0, slots, state.shape[0])] = h
    state.copy_(whole[:-1])
    return torch.where((slots >= 0)[:, None, None], y, 0.0).to(s["q"].dtype), state


def run(state):
    s, op = state, state["op"]
    if not own:
        return (_plain_experts if op.startswith("experts") else _plain_step if op == "attend_step"
                else _plain_attend)(s)
    from laplace_matvec_amd import laplex as lx
    if op.startswith("experts"):
        y = lx.laplex_experts(s["x"], s["w"], s["offsets"], transpose=s["transpose"])
        if op == "experts":
            return y
        d = lx.laplex_experts_backward(s["x"], s["w"], s["dy"], s["offsets"], transpose=s["transpose"],
                                       want=("dx", "dw"))
        return {"y": y, "dx": d["dx"], "dw": d["dw"]}
    if op == "attend_step":
        return lx.laplex_attend_step(s["q"], s["k"], s["v"], s["g"], s["state"], slots=s["slots"],
                                     scale=s["scale"]), s["state"]
    offsets = s["offsets"] if s["ragged"] else None
    train = op == "attend_train"
    r = lx.laplex_attend(s["q"], s["k"], s["v"], s["g"], offsets=offsets, h0=s["h0"], scale=s["scale"], final=True,
                         keep=train)
    out = {"y": r.y, "final": r.final}
    if train:
        d = lx.laplex_attend_backward(s["q"], s["k"], s["v"], s["g"], s["dy"], r.states, offsets=offsets, h0=s["h0"],
                                      scale=s["scale"], dfinal=s["dfinal"], want=("dq", "dk", "dv", "dg", "dh0"))
        out.update({name: d[name] for name in ("dq", "dk", "dv", "dg", "dh0")})
    return out


# ------------------------------------------------------------------ work

def _size(dtype):
    return DTYPES[dtype].itemsize


def work(case):
    op, e = case["op"], _size(case["dtype"])
    if op.startswith("experts"):
        rows, i, o = case["tokens"] * case["slots"], case["inner"], case["outer"]
        weights = min(rows, case["experts"]) * i * o
        if op == "experts":
            return {"bytes": e * (rows * (i + o) + weights) + 4 * (case["experts"] + 1), "flops": 2 * rows * i * o}
        return {"bytes": e * (rows * (2 * i + 2 * o) + 2 * weights) + 4 * (case["experts"] + 1),
                "flops": 6 * rows * i * o}
    heads, dk, dv = case["heads"], case["dk"], case["dv"]
    ins = e * (case["hq"] * dk + case["hk"] * dk + case["hv"] * dv) + heads * _size(case["gates"])
    state = 4 * heads * dk * dv
    if op == "attend_step":
        n = case["requests"]
        return {"bytes": n * (ins + e * heads * dv + 2 * state + 4), "flops": 5 * n * heads * dk * dv}
    n, s = case["rows"], case["seqs"]
    if op == "attend":
        return {"bytes": n * (ins + e * heads * dv) + s * state * (1 + case["h0"]), "flops": 4 * n * heads * dk * dv}
    return {"bytes": n * (2 * ins + 2 * e * heads * dv) + s * state * (3 + case["h0"]),
            "flops": 14 * n * heads * dk * dv}


# -------------------------------------------------- definition in 64 bits

def _exact_sequence(q, k, v, g, h0, dy, dfinal):
    """One sequence [heads, rows, ...] by its sums over all earlier rows, in blocks of 256 rows."""
    heads, n, _ = q.shape
    cut = g.float().exp() == 0
    group = cut.cumsum(-1)
    total = g.masked_fill(cut, 0.0).cumsum(-1)
    y = q.new_empty(heads, n, v.shape[-1])
    first = torch.exp(total) * (group == 0)  # how much of h0 is left
    left = torch.exp(total[:, -1:] - total) * (group == group[:, -1:])  # how much of each row is left at the end
    final = (k * left[..., None]).transpose(1, 2).contiguous() @ v + first[:, -1, None, None] * h0
    train = dy is not None
    if train:
        dq, dkk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        rows, cols = torch.zeros_like(g), torch.zeros_like(g)
    for a in range(0, n, 256):
        b = min(n, a + 256)
        w = total[:, a:b, None] - total[:, None, :b]
        late = torch.arange(b, device=q.device) > torch.arange(a, b, device=q.device)[:, None]
        w = torch.exp(w.masked_fill_(late | (group[:, a:b, None] != group[:, None, :b]), -math.inf))
        p = w * (q[:, a:b] @ k[:, :b].transpose(1, 2).contiguous())
        y[:, a:b] = p @ v[:, :b] + first[:, a:b, None] * (q[:, a:b] @ h0)
        if train:
            d = dy[:, a:b]
            dp = d @ v[:, :b].transpose(1, 2).contiguous()
            dv[:, :b] += p.transpose(1, 2).contiguous() @ d
            pair = p * dp
            rows[:, a:b] += pair.sum(-1)
            cols[:, :b] += pair.sum(-2)
            dp *= w
            dq[:, a:b] = dp @ k[:, :b]
            dkk[:, :b] += dp.transpose(1, 2).contiguous() @ q[:, a:b]
    if not train:
        return y, final
    from_first = first[..., None] * (dy @ h0.transpose(1, 2).contiguous())
    to_last = left[..., None] * (v @ dfinal.transpose(1, 2).contiguous())
    dv += left[..., None] * (k @ dfinal)
    dh0 = (q * first[..., None]).transpose(1, 2).contiguous() @ dy + first[:, -1, None, None] * dfinal
    after = rows - cols + (q * from_first).sum(-1)
    before = (k * to_last).sum(-1)
    dg = after.flip(-1).cumsum(-1).flip(-1) + before.cumsum(-1) - before
    dg += (first[:, -1] * (h0 * dfinal).sum((1, 2)))[:, None]
    return y, final, dq + from_first, dkk + to_last, dv, dg.masked_fill(cut, 0.0), dh0


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op.startswith("experts"):
        w = s["w"] if s["transpose"] else s["w"].transpose(1, 2)
        y = torch.zeros(s["x"].shape[0], w.shape[2], dtype=torch.float64, device="cuda")
        train = op == "experts_train"
        if train:
            dx = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
            dw = torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
        for e, (a, b) in enumerate(zip(s["ends"], s["ends"][1:])):
            if a == b:
                continue
            x, we = s["x"][a:b].double(), w[e].double().contiguous()
            y[a:b] = x @ we
            if train:
                dy = s["dy"][a:b].double()
                dx[a:b] = dy @ we.t().contiguous()
                grad = x.t().contiguous() @ dy
                dw[e] = grad if s["transpose"] else grad.t()
        return {"y": y, "dx": dx, "dw": dw} if train else y
    heads, scale = case["heads"], s["scale"]
    spread = lambda t: t.double().repeat_interleave(heads // t.shape[1], 1)  # noqa: E731
    if op == "attend_step":
        state, slots = s["state"].double(), s["slots"].long()
        y = torch.zeros(case["requests"], heads, case["dv"], dtype=torch.float64, device="cuda")
        busy = slots >= 0
        at = slots[busy]
        decay = s["g"][busy].double().exp()[..., None, None]
        k, v = spread(s["k"])[busy], spread(s["v"])[busy]
        state[at] = decay * state[at] + k[..., None] * v[..., None, :]
        y[busy] = (state[at] * (scale * spread(s["q"])[busy])[..., None]).sum(2)
        return y, state
    lead = s["g"].dim() - 1
    q, k, v, g = (s[name].flatten(0, lead - 1) for name in "qkvg")
    n, train = case["rows"], op == "attend_train"
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")  # noqa: E731
    y, final = new(n, heads, case["dv"]), new(case["seqs"], heads, case["dk"], case["dv"])
    if train:
        grads = [new(*t.shape) for t in (q, k, v, g)]
        dh0 = s["dfinal"].double()
    for i, (a, b) in enumerate(zip(s["ends"], s["ends"][1:])):
        h0 = torch.zeros_like(final[i]) if s["h0"] is None else s["h0"][i].double()
        if a == b:
            final[i] = h0
            continue
        part = max(1, (1 << 31) // (256 * (b - a) * 8))  # heads at a time
        for c in range(0, heads, part):
            own_heads = slice(c, min(heads, c + part))
            args = [spread(t[a:b])[:, own_heads].transpose(0, 1).contiguous() for t in (q, k, v)]
            gs = g[a:b, own_heads].double().t().contiguous()
            args[0] *= scale
            dy = s["dy"].flatten(0, lead - 1)[a:b, own_heads].double().transpose(0, 1).contiguous() if train else None
            r = _exact_sequence(*args, gs, h0[own_heads].contiguous(), dy,
                                s["dfinal"][i, own_heads].double() if train else None)
            y[a:b, own_heads], final[i, own_heads] = r[0].transpose(0, 1), r[1]
            if train:
                for to, got, by in zip(grads[:3], r[2:5], (scale, 1.0, 1.0)):
                    ids = torch.arange(c, own_heads.stop, device="cuda") // (heads // to.shape[1])
                    to[a:b].index_add_(1, ids, got.transpose(0, 1) * by)
                grads[3][a:b, own_heads], dh0[i, own_heads] = r[5].t(), r[6]
    shape = s["g"].shape[:-1]
    out = {"y": y.unflatten(0, shape), "final": final}
    if train:
        out.update({name: t.unflatten(0, shape) for name, t in zip(("dq", "dk", "dv", "dg"), grads)}, dh0=dh0)
    return out
