"""Recurrences whose rows go past the caches: arrays of 256 MiB and more."""
import math

import pytest
import torch

import tokens_ref as ref
from laplace_matvec_amd import laplex as lx

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32

# rows (a ragged last tile), channels, channels per decay, types, where the channels are parted
CASES = [
    (33077, 4099, 1, BF16, BF16, 2048),
    (33077, 4099, 1, BF16, F32, 2048),
    (32333, 4160, 64, BF16, F32, 2048),
    (32333, 4160, 64, F16, F16, 2048),
    (32777, 4098, 3, BF16, F32, 1920),
    (16500, 4101, 1, F32, F32, 2048),
    (16500, 4160, 4, F32, F32, 2048),
]


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def both(x, g, dy, offsets, h0, dfinal):
    r = lx.laplex_recur(x, g, offsets=offsets, h0=h0, final=True, keep=True)
    d = lx.laplex_recur_backward(x, g, dy, r.states, offsets=offsets, h0=h0, dfinal=dfinal)
    return dict(y=r.y, final=r.final, **d)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("n,width,per,kind,gates,cut", CASES)
def test_rows_past_the_caches(gpu, n, width, per, kind, gates, cut, packed):
    assert n * width * kind.itemsize > 1 << 28 and n % 256
    gen = torch.Generator(device=gpu).manual_seed(n + per)
    x, dy = (torch.randn(n, width, device=gpu, generator=gen).to(kind) for _ in range(2))
    heads = width // per
    g = -torch.rand(n, heads, device=gpu, generator=gen)
    spans = [(0, 290), (9000, 9300), (16000, 16290), (n - 301, n)]  # start fresh, nothing comes back into them
    for lo, hi in spans:
        g[lo] = -math.inf
        if hi < n:
            g[hi] = -math.inf
    g = g.to(gates)
    ends = [0, 100, 100, 9100, 16111, n] if packed else [0, n]
    offsets = torch.tensor(ends, dtype=torch.int32, device=gpu) if packed else None
    seqs = len(ends) - 1
    h0, dfinal = (torch.randn(seqs, width, device=gpu, generator=gen) for _ in range(2))
    out = both(x, g, dy, offsets, h0, dfinal)

    again = both(x, g, dy, offsets, h0, dfinal)
    assert all(torch.equal(again[k], out[k]) for k in out)
    del again

    # parts of the channels go through the caches, with the same sums
    for c0, c1 in ((0, cut), (cut, width)):
        assert n * (c1 - c0) * kind.itemsize < 1 << 28 and c0 % per == 0
        part = both(x[:, c0:c1], g[:, c0 // per:c1 // per], dy[:, c0:c1], offsets, h0[:, c0:c1].contiguous(),
                    dfinal[:, c0:c1].contiguous())
        for k in out:
            whole = out[k][:, c0 // per:c1 // per] if k == "dg" else out[k][:, c0:c1]
            assert torch.equal(part[k], whole), (k, c0)
        del part

    cols = [per * (h % heads) for h in (0, 1, 63 // per, 64 // per, cut // per, heads - 2, heads - 1)]
    spread = [c + i for c in cols for i in range(per)]
    for lo, hi in spans:
        at = sorted({0, hi - lo} | {e - lo for e in ends if lo < e < hi})
        # the first sequence of the span begins with its reset, the last ends before one or with the rows
        first = [q for q in range(seqs) if ends[q] <= lo < ends[q + 1]][0]
        pick = list(range(first, first + len(at) - 1))
        if packed and lo == 0:
            at, pick = [0, 100, 100, 290], [0, 1, 2]
        end = dfinal[pick][:, spread].clone()
        if hi < n:
            end[-1] = 0
        want = ref.Recur(x[lo:hi][:, spread], g[lo:hi][:, [c // per for c in cols]], at, h0[pick][:, spread],
                         dy[lo:hi][:, spread], end)
        ref.assert_within(out["y"][lo:hi][:, spread], want.y, want.ey)
        ref.assert_within(out["dx"][lo:hi][:, spread], want.dx, want.edx)
        ref.assert_within(out["dg"][lo:hi][:, [c // per for c in cols]], want.dg, want.edg)
