"""Cases of the token-routing and gated-recurrence operators.

    route         stable sort of the token slots by expert: order, place, offsets
    dispatch      token rows copied to their places by expert, and the gradient (each token's copies summed)
    combine       weighted sum of each token's expert rows
    combine_grad  gradients of combine: expert rows and weights
    recur         h_t = exp(g_t) h_{t-1} + x_t along packed sequences, with initial and final states
    recur_train   the same with its backward pass: gradients of x, g and the initial states
    step          one token for each request on a pool of states

The plain forms are elementary torch operations in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


def listed():
    return [
        # one decoding step of 48 requests choosing 2 of 8 experts: latency only
        dict(name="route decode", op="route", tokens=48, slots=2, experts=8, ids="int64", dropped=0.0),
        # a training batch of 131072 tokens, 8 of 256 experts, 2 % of the slots dropped (over capacity)
        dict(name="route train", op="route", tokens=131072, slots=8, experts=256, ids="int64", dropped=0.02),
        # a short odd prompt in half precision
        dict(name="dispatch prompt", op="dispatch", tokens=391, slots=4, experts=16, dropped=0.0, width=1000,
             dtype="float16"),
        # a training micro-batch, 4 of 64 experts, a few dropped
        dict(name="dispatch train", op="dispatch", tokens=16384, slots=4, experts=64, dropped=0.02, width=2048,
             dtype="bfloat16"),
        # one decoding step of 64 requests, 8 of 128 experts
        dict(name="combine decode", op="combine", tokens=64, slots=8, experts=128, dropped=0.0, width=2048,
             dtype="bfloat16"),
        # a prefill of 16384 tokens, 2 of 8 wide experts
        dict(name="combine prefill", op="combine", tokens=16384, slots=2, experts=8, dropped=0.0, width=4096,
             dtype="bfloat16"),
        # backward of a training micro-batch
        dict(name="combine grad", op="combine_grad", tokens=16384, slots=4, experts=64, dropped=0.02, width=2048,
             dtype="bfloat16"),
        # three short prompts of uneven length in one batch, decays shared by heads of 40 channels
        dict(name="recur prompts", op="recur", rows=777, seqs=3, ragged=True, heads=13, per_head=40,
             dtype="float16", gates="float32", h0=True, resets=False, fused=False),
        # one long prompt: a single row of 65536 tokens, a decay for each channel
        dict(name="recur long", op="recur", rows=65536, seqs=1, ragged=False, heads=2048, per_head=1,
             dtype="bfloat16", gates="bfloat16", h0=True, resets=False, fused=True),
        # packed documents of uneven length in training, heads of 64 channels with one decay each
        dict(name="recur train packed", op="recur_train", rows=32768, seqs=24, ragged=True, heads=64, per_head=64,
             dtype="bfloat16", gates="float32", h0=False, resets=True, fused=False),
        # equal sequences in full precision, a decay for each channel
        dict(name="recur train f32", op="recur_train", rows=8192, seqs=4, ragged=False, heads=1024, per_head=1,
             dtype="float32", gates="float32", h0=True, resets=False, fused=False),
        # one token for each of 256 requests out of a pool of 320 states
        dict(name="step serve", op="step", requests=256, pool=320, heads=64, per_head=64, dtype="bfloat16",
             gates="float32", idle=0.03),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm: a power of two or odd."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    if rng.random() < 0.35:
        return max(lo, 1 << int(math.log2(v)))
    return min(hi, int(v) | 1)


def _moe(rng, op, most):
    slots = rng.choice([1, 2, 3, 4, 6, 8])
    experts = max(slots, _spread(rng, 4, 512))
    width = _spread(rng, 16, 8191)
    if rng.random() < 0.4:
        width = (width // 8 | 1) * 8  # rows that end on 16 bytes in every type
    dtype = rng.choice(list(DTYPES))
    tokens = _spread(rng, 1, max(1, min(16384, most // (slots * width * _size(dtype)))))
    return dict(op=op, tokens=tokens, slots=slots, experts=experts, dropped=rng.choice([0.0, 0.05]), width=width,
                dtype=dtype)


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "combine_grad", "recur", "recur", "recur_train", "recur_train",
                     "step"])
    if op == "route":
        return dict(op=op, tokens=_spread(rng, 1, 131071), slots=rng.choice([1, 2, 3, 4, 6, 8]),
                    experts=_spread(rng, 8, 4095), ids=rng.choice(["int32", "int64"]),
                    dropped=rng.choice([0.0, 0.05]))
    if op in ("dispatch", "combine", "combine_grad"):
        return _moe(rng, op, 1 << 28)
    dtype = rng.choice(list(DTYPES))
    gates = rng.choice([dtype, "float32"])
    per_head = rng.choice([1, 1, 16, 40, 64, 80, 128, 256])
    heads = _spread(rng, 1, max(1, 4096 // per_head))
    if op == "step":
        n = _spread(rng, 1, 1024)
        return dict(op=op, requests=n, pool=n + rng.choice([0, 1, 77]), heads=heads, per_head=per_head, dtype=dtype,
                    gates=gates, idle=rng.choice([0.0, 0.1]))
    width = heads * per_head
    seqs = rng.choice([1, 1, 2, 5, 16, 63])
    per_row = 4 * width * _size(dtype) + 2 * heads * _size(gates)
    rows = _spread(rng, 1, min(65535, (1 << 30) // per_row))
    ragged = rng.random() < 0.6
    if not ragged:
        rows = (rows // seqs | 1) * seqs
    return dict(op=op, rows=rows, seqs=seqs, ragged=ragged, heads=heads, per_head=per_head, dtype=dtype, gates=gates,
                h0=rng.random() < 0.5, resets=rng.random() < 0.3, fused=rng.random() < 0.3)


# ---------------------------------------------------------------- inputs

def _slots(case, gen):
    """Expert of each (token, slot): skewed, as routers are, distinct within a token; -1 where dropped."""
    t, k, e = case["tokens"], case["slots"], case["experts"]
    u = torch.rand(t, 1, device="cuda", generator=gen)
    base = (u.pow(1.5) * e).to(torch.int64).clamp_(max=e - 1)
    ids = (base + torch.arange(k, device="cuda") * max(1, e // k)) % e
    if case["dropped"]:
        ids[torch.rand(t, k, device="cuda", generator=gen) < case["dropped"]] = -1
    return ids


def _sorted(ids, experts):
    """order, place and offsets of a stable sort by expert; dropped slots come last and have no place."""
    flat = ids.reshape(-1).to(torch.int64)
    n = flat.numel()
    valid = (flat >= 0) & (flat < experts)
    keys, order = torch.sort(torch.where(valid, flat, experts), stable=True)
    offsets = torch.searchsorted(keys, torch.arange(experts + 1, device=flat.device)).to(torch.int32)
    ranks = torch.empty_like(order)
    ranks[order] = torch.arange(n, device=flat.device)
    place = torch.where(valid, ranks, -1).to(torch.int32).reshape(ids.shape)
    order = torch.where(keys < experts, order, -1).to(torch.int32)
    return order, place, offsets


def _offsets(case, gen):
    n, s = case["rows"], case["seqs"]
    if not case["ragged"]:
        return torch.arange(s + 1, device="cuda", dtype=torch.int32) * (n // s)
    cuts = torch.sort((torch.rand(s - 1, device="cuda", generator=gen) * n).to(torch.int32)).values
    if s > 4:
        cuts[2] = cuts[1]  # an empty sequence
    zero = torch.zeros(1, device="cuda", dtype=torch.int32)
    return torch.cat([zero, cuts, zero + n])


def _decays(rows, heads, gen):
    """Logarithms of decays whose memory spans 2 to 1000 tokens by channel, moved by each token."""
    base = torch.rand(heads, device="cuda", generator=gen) * -math.log(500.0) - math.log(2.0)
    move = torch.randn(rows, heads, device="cuda", generator=gen) * 0.5
    return -torch.exp(base + move)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    normal = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
    if op == "route":
        return {**s, "ids": _slots(case, gen).to(torch.int32 if case["ids"] == "int32" else torch.int64),
                "experts": case["experts"]}
    dt = DTYPES[case["dtype"]]
    if op in ("dispatch", "combine", "combine_grad"):
        t, k, d = case["tokens"], case["slots"], case["width"]
        s["order"], s["place"], s["offsets"] = _sorted(_slots(case, gen), case["experts"])
        if op == "dispatch":
            return {**s, "x": normal(t, d).to(dt), "dxs": normal(t * k, d).to(dt)}
        s["weights"] = torch.softmax(normal(t, k), -1)
        s["ys"] = normal(t * k, d).to(dt)
        if op == "combine_grad":
            s["dy"] = normal(t, d).to(dt)
        return s
    gdt = DTYPES[case["gates"]]
    heads, width = case["heads"], case["heads"] * case["per_head"]
    if op == "step":
        n, pool = case["requests"], case["pool"]
        slots = torch.randperm(pool, device="cuda", generator=gen)[:n].to(torch.int32)
        slots[torch.rand(n, device="cuda", generator=gen) < case["idle"]] = -1  # a request without work
        return {**s, "x": normal(n, width).to(dt), "g": _decays(n, heads, gen).to(gdt), "state": normal(pool, width),
                "slots": slots}
    n, seqs = case["rows"], case["seqs"]
    x, g = normal(n, width).to(dt), _decays(n, heads, gen).to(gdt)
    if case["resets"]:
        g[torch.rand(n, device="cuda", generator=gen) < 0.002] = -math.inf
    if case["fused"] and dt == gdt:  # both are parts of one projection's rows
        both = torch.cat([x, g], 1)
        x, g = both[:, :width], both[:, width:]
    s["offsets"] = _offsets(case, gen)
    if not case["ragged"]:
        x, g = x.unflatten(0, (seqs, n // seqs)), g.unflatten(0, (seqs, n // seqs))
    s.update(x=x, g=g, h0=normal(seqs, width) if case["h0"] else None, ragged=case["ragged"])
    if op == "recur_train":
        s["dy"] = normal(n, width).to(dt).view(x.shape)
        s["dfinal"] = normal(seqs, width)
    return s


# ------------------------------------------------------------ plain forms

def _scan(a, v, reverse):
    """v_t + a_t v_{t-1} + a_t a_{t-1} v_{t-2} + ... along rows (towards earlier rows if reverse), by doubling.
    A decay of zero forgets what came before, whatever it was."""
    d = 1
    while d < v.shape[0]:
        old = v
        lo, hi = slice(0, -d), slice(d, None)
        here, there = (lo, hi) if reverse else (hi, lo)
        v, b = old.clone(), a.clone()
        v[here] += torch.where(a[here] == 0, 0.0, a[here] * old[there])
        b[here] = a[here] * a[there]
        a, d = b, 2 * d
    return v


def _parts(s):
    """Rows in 32 bits: x, decays spread over channels, and the non-empty sequences with their first and last rows."""
    x = s["x"].flatten(0, -2).float()
    g = s["g"].flatten(0, -2).float()
    a = torch.exp(g).repeat_interleave(x.shape[1] // g.shape[1], 1)
    return x, a, g.shape[1], s["offsets"][:-1].long(), s["offsets"][1:].long()


def _plain_recur(s):
    x, a, heads, first, end = _parts(s)
    n = x.shape[0]
    h0 = s["h0"] if s["h0"] is not None else x.new_zeros(first.numel(), x.shape[1])
    # rows past the end take what an empty sequence would write at its start; one more row holds it
    at = torch.where(end > first, first, n)
    begin = x.new_zeros(n + 1, 1).index_fill(0, at, 1.0)[:n] > 0
    before = x.new_zeros(n + 1, x.shape[1]).index_copy(0, at, h0)[:n]
    v = x + torch.where(begin & (a != 0), a * before, 0.0)
    h = _scan(a.masked_fill(begin, 0.0), v, False)
    final = torch.where((end > first)[:, None], h[(end - 1).clamp(min=0)], h0)
    if s["op"] == "recur":
        return {"y": h.to(s["x"].dtype).view(s["x"].shape), "final": final}
    dy = s["dy"].flatten(0, -2).float()
    last = torch.where(end > first, end - 1, n)
    u = torch.cat([dy, dy.new_zeros(1, dy.shape[1])]).index_add(0, last, s["dfinal"])[:n]
    # u_t = dy_t + a_{t+1} u_{t+1} within a sequence
    step = torch.cat([a.masked_fill(begin, 0.0)[1:], a.new_zeros(1, a.shape[1])])
    u = _scan(step, u, True)
    w = torch.where(a == 0, 0.0, a * u)
    prev = torch.where(begin, before, torch.cat([h.new_zeros(1, h.shape[1]), h[:-1]]))
    dg = torch.where(w == 0, 0.0, w * prev).unflatten(1, (heads, -1)).sum(-1)
    dh0 = torch.where((end > first)[:, None], w[first.clamp(max=n - 1)], s["dfinal"])
    back = lambda t, like: t.to(like.dtype).view(like.shape)  # noqa: E731
    return {"y": back(h, s["x"]), "final": final, "dx": back(u, s["x"]), "dg": back(dg, s["g"]), "dh0": dh0}


def _rows_of(ys, place):
    """Each token's rows in 32 bits, zero where a slot has none."""
    rows = ys[place.clamp(min=0).long()].float()
    return rows.masked_fill_((place < 0)[..., None], 0.0)


def _plain(s):
    op = s["op"]
    if op == "route":
        return _sorted(s["ids"], s["experts"])
    if op == "dispatch":
        order, k = s["order"], s["place"].shape[1]
        xs = s["x"][(order.clamp(min=0) // k).long()].masked_fill_((order < 0)[:, None], 0.0)
        return xs, _rows_of(s["dxs"], s["place"]).sum(1).to(s["x"].dtype)
    if op == "combine":
        return (_rows_of(s["ys"], s["place"]) * s["weights"][..., None]).sum(1).to(s["ys"].dtype)
    if op == "combine_grad":
        dy, order = s["dy"].float(), s["order"]
        dw = (_rows_of(s["ys"], s["place"]) * dy[:, None]).sum(-1)
        slot = order.clamp(min=0).long()
        dys = dy[slot // s["place"].shape[1]] * s["weights"].reshape(-1)[slot][:, None]
        return dys.masked_fill_((order < 0)[:, None], 0.0).to(s["ys"].dtype), dw
    if op == "step":
        slots, state = s["slots"].long(), s["state"]
        x = s["x"].float()
        a = torch.exp(s["g"].float()).repeat_interleave(x.shape[1] // s["g"].shape[1], 1)
        h = torch.where(a == 0, 0.0, a * state[slots.clamp(min=0)]) + x
        busy = (slots >= 0)[:, None]
        # requests without work write into a row of their own past the pool
        whole = torch.cat([state, state.new_zeros(1, x.shape[1])])
        whole[torch.where(slots >= 0, slots, state.shape[0])] = h
        state.copy_(whole[:-1])
        return torch.where(busy, h, 0.0).to(s["x"].dtype), state
    return _plain_recur(s)


def run(state):
    if not own:
        return _plain(state)
    from laplace_matvec_amd import laplex as lx
    s, op = state, state["op"]
    if op == "route":
        return tuple(lx.laplex_route(s["ids"], s["experts"]))
    if op in ("dispatch", "combine", "combine_grad"):
        route = lx.Route(s["order"], s["place"], s["offsets"])
        if op == "dispatch":
            return lx.laplex_dispatch(route, s["x"]), lx.laplex_combine(route, s["dxs"])
        if op == "combine":
            return lx.laplex_combine(route, s["ys"], s["weights"])
        return lx.laplex_combine_backward(route, s["dy"], s["ys"], s["weights"])
    if op == "step":
        return lx.laplex_recur_step(s["x"], s["g"], s["state"], slots=s["slots"]), s["state"]
    offsets = s["offsets"] if s["ragged"] else None
    train = op == "recur_train"
    r = lx.laplex_recur(s["x"], s["g"], offsets=offsets, h0=s["h0"], final=True, keep=train)
    out = {"y": r.y, "final": r.final}
    if train:
        d = lx.laplex_recur_backward(s["x"], s["g"], s["dy"], r.states, offsets=offsets, h0=s["h0"],
                                     dfinal=s["dfinal"], want=("dx", "dg", "dh0"))
        out.update(dx=d["dx"], dg=d["dg"], dh0=d["dh0"])
    return out


# ------------------------------------------------------------------ work

def _size(dtype):
    return DTYPES[dtype].itemsize


def work(case):
    op = case["op"]
    if op == "route":
        n = case["tokens"] * case["slots"]
        return {"bytes": n * (4 if case["ids"] == "int32" else 8) + 8 * n + 4 * (case["experts"] + 1), "flops": 0}
    e = _size(case["dtype"])
    if op in ("dispatch", "combine", "combine_grad"):
        one = case["tokens"] * case["width"]
        many = one * case["slots"]
        rows = case["tokens"] * case["slots"]
        if op == "dispatch":
            return {"bytes": 2 * e * (one + many) + 4 * rows, "flops": many}
        if op == "combine":
            return {"bytes": e * (one + many) + 8 * rows, "flops": 2 * many}
        return {"bytes": e * (one + 2 * many) + 12 * rows, "flops": 3 * many}
    width, gates = case["heads"] * case["per_head"], case["heads"] * _size(case["gates"])
    if op == "step":
        n = case["requests"]
        return {"bytes": n * (width * (2 * e + 8) + gates + 4), "flops": 3 * n * width}
    n, s = case["rows"], case["seqs"]
    states = 4 * s * width * (1 + case["h0"])
    if op == "recur":
        return {"bytes": n * (2 * width * e + gates) + states, "flops": 3 * n * width}
    return {"bytes": n * (4 * width * e + 2 * gates) + states + 8 * s * width, "flops": 10 * n * width}


# -------------------------------------------------- definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "route":
        ids = s["ids"].reshape(-1).cpu().tolist()
        lists = [[] for _ in range(case["experts"])]
        for slot, e in enumerate(ids):
            if 0 <= e < case["experts"]:
                lists[e].append(slot)
        order, ends = [slot for one in lists for slot in one], [0]
        for one in lists:
            ends.append(ends[-1] + len(one))
        place = torch.full((len(ids),), -1, dtype=torch.int32)
        place[torch.tensor(order, dtype=torch.int64)] = torch.arange(len(order), dtype=torch.int32)
        order += [-1] * (len(ids) - len(order))
        return (torch.tensor(order, dtype=torch.int32), place.view(s["ids"].shape),
                torch.tensor(ends, dtype=torch.int32))
    if op in ("dispatch", "combine", "combine_grad"):
        t, k = case["tokens"], case["slots"]
        rows = t * k
        width = case["width"]
        new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")  # noqa: E731
        xs, sums, dys, dw = new(rows, width), new(t, width), new(rows, width), new(t, k)
        for j in range(k):
            p = s["place"][:, j].long()
            tok = torch.nonzero(p >= 0).reshape(-1)
            p = p[tok]
            if op == "dispatch":
                xs[p] = s["x"][tok].double()
                sums[tok] += s["dxs"][p].double()
            elif op == "combine":
                sums[tok] += s["weights"][tok, j, None].double() * s["ys"][p].double()
            else:
                dys[p] = s["weights"][tok, j, None].double() * s["dy"][tok].double()
                dw[tok, j] = (s["dy"][tok].double() * s["ys"][p].double()).sum(-1)
        return (xs, sums) if op == "dispatch" else sums if op == "combine" else (dys, dw)
    heads, per = case["heads"], case["per_head"]
    width = heads * per
    if op == "step":
        state, y = s["state"].double(), torch.zeros(case["requests"], width, dtype=torch.float64, device="cuda")
        for i, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                y[i] = s["g"][i].double().exp().repeat_interleave(per) * state[slot] + s["x"][i].double()
                state[slot] = y[i]
        return y, state
    x = s["x"].reshape(-1, width).double()
    a = s["g"].reshape(-1, heads).double().exp()
    offsets = s["offsets"].tolist()
    h0 = s["h0"].double() if s["h0"] is not None else torch.zeros(case["seqs"], width, dtype=torch.float64, device="cuda")
    y, final = torch.empty_like(x), h0.clone()
    train = op == "recur_train"
    if train:
        dy = s["dy"].reshape(-1, width).double()
        dx, dg, dh0 = torch.empty_like(x), torch.empty_like(a), s["dfinal"].double()
    for q in range(case["seqs"]):
        first, end = offsets[q], offsets[q + 1]
        h = h0[q].view(heads, per)
        for i in range(first, end):
            h = torch.addcmul(x[i].view(heads, per), a[i][:, None], h, out=y[i].view(heads, per))
        if end > first:
            final[q] = y[end - 1]
        if train:
            w = dh0[q].view(heads, per).clone()
            for i in range(end - 1, first - 1, -1):
                u = torch.add(dy[i].view(heads, per), w, out=dx[i].view(heads, per))
                w = a[i][:, None] * u
            dh0[q] = w.reshape(-1)
            if end > first:
                prev = torch.cat([h0[q][None], y[first:end - 1]])
                grad = a[first:end, :, None] * (dx[first:end] * prev).view(-1, heads, per)
                dg[first:end] = grad.sum(-1)
    shape = s["x"].shape
    out = {"y": y.view(shape), "final": final}
    if train:
        out.update(dx=dx.view(shape), dg=dg.view(s["g"].shape), dh0=dh0)
    return out
