"""Thin ctypes binding of liblaplex.so (C ABI in include/laplex.h).

Argument marshalling only: every step of the operator runs in the HIP
library.  PyTorch supplies device memory and the current stream.  If the
library is missing this module raises on import of any entry point; there
is no fallback implementation.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblaplex.so")

OK = 0
ERR_INVALID_ARGUMENT = 1
ERR_NONFINITE_ANCHOR = 2
ERR_OUT_OF_MEMORY = 3
ERR_UNSUPPORTED = 4
ERR_DEVICE = 5
ERR_NO_DEVICE = 6

OPT_GENERAL_ALGO = 1
ALGO_AUTO, ALGO_BUCKET, ALGO_EVALUATE = 0, 1, 2
PLAN_SYMMETRIC, PLAN_PHASED = 1, 2

# every entry point of include/laplex.h: name -> (restype, argtypes)
_VP, _I64, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
SIGNATURES = {
    "laplex_plan_create": (_I32, [ctypes.POINTER(_VP), _VP, _I64, _VP, _I64, _VP, _VP, _VP]),
    "laplex_plan_create_apply": (_I32, [ctypes.POINTER(_VP), _VP, _I64, _VP, _VP, _VP, _VP, _I64, _VP]),
    "laplex_apply": (_I32, [_VP, _VP, _VP, _I64, _I32, _VP]),
    "laplex_apply_noalloc": (_I32, [_VP, _VP, _VP, _I64, _I32, _VP]),
    "laplex_gram": (_I32, [_VP, _VP, _VP, _VP]),
    "laplex_plan_destroy": (_I32, [_VP]),
    "laplex_plan_perm": (_I32, [_VP, _I32, ctypes.POINTER(_VP)]),
    "laplex_plan_sorted": (_I32, [_VP, _I32, ctypes.POINTER(_VP)]),
    "laplex_plan_info": (_I32, [_VP, ctypes.POINTER(_I64), ctypes.POINTER(_I64), ctypes.POINTER(_I32)]),
    "laplex_plan_set_option": (_I32, [_VP, _I32, _I64]),
    "laplex_plan_set_temperature": (_I32, [_VP, ctypes.c_double]),
    "laplex_backward": (_I32, [_VP, _VP, _VP, _I64, _I32, _VP, _VP, _VP, _VP, _VP, _VP]),
    "laplex_route_workspace": (_I64, [_I64, _I64, _I64]),
    "laplex_route": (_I32, [_VP, _I32, _I64, _I64, _I64, _VP, _VP, _VP, _VP, _I64, _VP]),
    "laplex_dispatch": (_I32, [_I64, _I64, _I64, _VP, _VP, _I32, _I64, _VP, _I64, _VP, _I64, _VP]),
    "laplex_combine": (_I32, [_I64, _I64, _VP, _I32, _I64, _VP, _I64, _VP, _VP, _I64, _VP]),
    "laplex_combine_backward": (_I32, [_I64, _I64, _I64, _VP, _VP, _I32, _I64, _VP, _I64, _VP, _I64, _VP, _VP, _I64,
                                       _VP, _VP]),
    "laplex_recur_workspace": (_I64, [_I64, _I64, _I64, _I32]),
    "laplex_recur_states": (_I64, [_I64, _I64]),
    "laplex_recur": (_I32, [_I64, _I64, _VP, _I64, _I64, _I32, _I32, _VP, _I64, _VP, _I64, _VP, _VP, _I64, _VP, _VP,
                            _VP, _I64, _VP]),
    "laplex_recur_backward": (_I32, [_I64, _I64, _VP, _I64, _I64, _I32, _I32, _VP, _I64, _VP, _I64, _VP, _VP, _VP,
                                     _I64, _VP, _VP, _I64, _VP, _I64, _VP, _VP, _I64, _VP]),
    "laplex_recur_step": (_I32, [_I64, _I64, _VP, _I64, _I64, _I32, _I32, _VP, _I64, _VP, _I64, _VP, _VP, _I64, _VP]),
    "laplex_experts": (_I32, [_I64, _I64, _VP, _I64, _I64, _I32, _I32, _VP, _I64, _VP, _I64, _I64, _VP, _I64, _VP]),
    "laplex_experts_backward": (_I32, [_I64, _I64, _VP, _I64, _I64, _I32, _I32, _VP, _I64, _VP, _I64, _I64, _VP, _I64,
                                       _VP, _I64, _VP, _I64, _I64, _VP]),
    "laplex_attend_states": (_I64, [_I64] * 5),
    "laplex_attend_workspace": (_I64, [_I64] * 8 + [_I32, _I32]),
    "laplex_attend": (_I32, [_I64, _I64, _VP] + [_I64] * 6 + [_I32, _I32, ctypes.c_float] + [_VP, _I64] * 4
                      + [_VP, _VP, _I64, _VP, _VP, _VP, _I64, _VP]),
    "laplex_attend_backward": (_I32, [_I64, _I64, _VP] + [_I64] * 6 + [_I32, _I32, ctypes.c_float] + [_VP, _I64] * 4
                               + [_VP, _VP, _VP, _I64, _VP] + [_VP, _I64] * 4 + [_VP, _VP, _I64, _VP]),
    "laplex_attend_step": (_I32, [_I64, _I64, _VP] + [_I64] * 6 + [_I32, _I32, ctypes.c_float] + [_VP, _I64] * 4
                           + [_VP, _VP, _I64, _VP]),
    "laplex_profile_enable": (_I32, [_I32]),
    "laplex_profile_only": (_I32, [ctypes.c_char_p]),
    "laplex_profile_reset": (_I32, []),
    "laplex_profile_collect": (_I32, []),
    "laplex_profile_entry": (_I32, [_I32, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(_I64),
                                    ctypes.POINTER(ctypes.c_double)]),
    "laplex_status_str": (ctypes.c_char_p, [_I32]),
    "laplex_last_error": (ctypes.c_char_p, []),
}

_lib = None


class LaplexError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        lib = load()
        msg = lib.laplex_status_str(status).decode()
        detail = lib.laplex_last_error().decode()
        super().__init__(f"{where}: {msg}" + (f" ({detail})" if detail else ""))


def load():
    """Load liblaplex.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run laplace_matvec_amd/build.py "
                               "(or __graft_entry__.build()) first")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
    return _lib


def _check(st: int, where: str):
    if st != OK:
        raise LaplexError(st, where)


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _dev_f32(t, name):
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous float32 CUDA tensor")
    return t


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


class Plan:
    """A sorted LAPLEX operator K = LAPLEX(a, phi; b, psi) (n x k)."""

    def __init__(self, handle, n, k, symmetric, phased, device):
        self.handle = handle
        self.n, self.k = n, k
        self.symmetric, self.phased = symmetric, phased
        self.device = device

    def destroy(self):
        if self.handle:
            _check(load().laplex_plan_destroy(self.handle), "laplex_plan_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.destroy()


def laplex_plan_create(a, b=None, phi=None, psi=None, stream=None) -> Plan:
    a = _dev_f32(a, "a")
    b = _dev_f32(b, "b")
    phi = _dev_f32(phi, "phi")
    psi = _dev_f32(psi, "psi")
    h = ctypes.c_void_p()
    st = load().laplex_plan_create(ctypes.byref(h), _ptr(a), a.numel(), _ptr(b),
                                   0 if b is None else b.numel(), _ptr(phi), _ptr(psi), _stream(stream))
    _check(st, "laplex_plan_create")
    k = a.numel() if b is None else b.numel()
    return Plan(h, a.numel(), k, b is None, phi is not None, a.device)


def laplex_plan_create_apply(a, x, y=None, phi=None, psi=None, stream=None):
    """Symmetric plan and y = K x in one call; returns (plan, y)."""
    a = _dev_f32(a, "a")
    phi = _dev_f32(phi, "phi")
    psi = _dev_f32(psi, "psi")
    x = _dev_f32(x, "x")
    n = a.numel()
    one = x.dim() == 1
    batch = 1 if one else x.shape[0]
    if x.shape[-1] != n or x.dim() > 2:
        raise ValueError(f"x must have shape [batch][{n}]")
    if y is None:
        y = torch.empty_like(x)
    y = _dev_f32(y, "y")
    if y.numel() != batch * n:
        raise ValueError("y has the wrong size")
    h = ctypes.c_void_p()
    st = load().laplex_plan_create_apply(ctypes.byref(h), _ptr(a), n, _ptr(phi), _ptr(psi), _ptr(x), _ptr(y),
                                         batch, _stream(stream))
    _check(st, "laplex_plan_create_apply")
    return Plan(h, n, n, True, phi is not None, a.device), y


def laplex_apply(plan: Plan, x, y=None, transpose: bool = False, stream=None):
    """y = K x (transpose False) or K^T x; x is [batch][in] or 1-D."""
    x = _dev_f32(x, "x")
    n_in, n_out = (plan.n, plan.k) if transpose else (plan.k, plan.n)
    one = x.dim() == 1
    batch = 1 if one else x.shape[0]
    if x.shape[-1] != n_in or x.dim() > 2:
        raise ValueError(f"x must have shape [batch][{n_in}]")
    if y is None:
        y = torch.empty((n_out,) if one else (batch, n_out), dtype=torch.float32, device=x.device)
    y = _dev_f32(y, "y")
    if y.numel() != batch * n_out:
        raise ValueError("y has the wrong size")
    _check(load().laplex_apply(plan.handle, _ptr(x), _ptr(y), batch, int(bool(transpose)), _stream(stream)),
           "laplex_apply")
    return y


def laplex_apply_noalloc(plan: Plan, x, y, transpose: bool = False, stream=None):
    """laplex_apply into a caller-provided y, with the library's fixed
    scratch instead of any allocation (see include/laplex.h)."""
    x = _dev_f32(x, "x")
    y = _dev_f32(y, "y")
    n_in, n_out = (plan.n, plan.k) if transpose else (plan.k, plan.n)
    batch = 1 if x.dim() == 1 else x.shape[0]
    if x.shape[-1] != n_in or x.dim() > 2 or y.numel() != batch * n_out:
        raise ValueError(f"x must be [batch][{n_in}] and y [batch][{n_out}]")
    _check(load().laplex_apply_noalloc(plan.handle, _ptr(x), _ptr(y), batch, int(bool(transpose)),
                                       _stream(stream)), "laplex_apply_noalloc")
    return y


def laplex_gram(plan: Plan, D, M=None, stream=None):
    D = _dev_f32(D, "D")
    if D.numel() != plan.k:
        raise ValueError(f"D must have {plan.k} entries")
    if M is None:
        M = torch.empty((plan.n, plan.n), dtype=torch.float32, device=D.device)
    M = _dev_f32(M, "M")
    _check(load().laplex_gram(plan.handle, _ptr(D), _ptr(M), _stream(stream)), "laplex_gram")
    return M


def laplex_plan_set_option(plan: Plan, option: int, value: int):
    _check(load().laplex_plan_set_option(plan.handle, option, value), "laplex_plan_set_option")


def laplex_plan_set_temperature(plan: Plan, t: float):
    """Entries exp(-|a_i - b_j| / t); t = 0 routes by exact anchor equality."""
    _check(load().laplex_plan_set_temperature(plan.handle, float(t)), "laplex_plan_set_temperature")


def laplex_backward(plan: Plan, x, g, transpose: bool = False, want=("dx", "da", "db", "dphi", "dpsi"),
                    stream=None) -> dict:
    """Gradients of a step through y = K x (or K^T x): x the forward input
    (None for a plan from laplex_plan_create_apply, which kept it), g = dL/dy.  Returns the requested tensors among dx ([batch][in]), da [n],
    db [k] (general plans), dphi [n], dpsi [k] (phased plans); entries a plan
    does not have are left out."""
    g = _dev_f32(g, "g")
    n_in, n_out = (plan.n, plan.k) if transpose else (plan.k, plan.n)
    if x is None:  # the input kept by laplex_plan_create_apply
        shape = (n_in,) if g.dim() == 1 else (g.shape[0], n_in)
    else:
        x = _dev_f32(x, "x")
        shape = tuple(x.shape)
        if x.shape[-1] != n_in or x.dim() > 2:
            raise ValueError(f"x must have shape [batch][{n_in}]")
    batch = 1 if len(shape) == 1 else shape[0]
    if g.numel() != batch * n_out or g.shape[-1] != n_out:
        raise ValueError(f"g must have shape [batch][{n_out}]")
    dev = g.device
    out = {}
    if "dx" in want:
        out["dx"] = torch.empty(shape, dtype=torch.float32, device=dev)
    if "da" in want:
        out["da"] = torch.empty(plan.n, dtype=torch.float32, device=dev)
    if "db" in want and not plan.symmetric:
        out["db"] = torch.empty(plan.k, dtype=torch.float32, device=dev)
    if plan.phased:
        if "dphi" in want:
            out["dphi"] = torch.empty(plan.n, dtype=torch.float32, device=dev)
        if "dpsi" in want:
            out["dpsi"] = torch.empty(plan.k, dtype=torch.float32, device=dev)
    p = [_ptr(out.get(k)) for k in ("dx", "da", "db", "dphi", "dpsi")]
    _check(load().laplex_backward(plan.handle, _ptr(x), _ptr(g), batch, int(bool(transpose)), *p,
                                  _stream(stream)), "laplex_backward")
    return out


def _copy_device(dst: torch.Tensor, src_ptr: int, nbytes: int, stream=None):
    hip = ctypes.CDLL("libamdhip64.so")
    hip.hipMemcpyAsync.restype = ctypes.c_int
    hip.hipMemcpyAsync.argtypes = [_VP, _VP, ctypes.c_size_t, ctypes.c_int, _VP]
    rc = hip.hipMemcpyAsync(ctypes.c_void_p(dst.data_ptr()), ctypes.c_void_p(src_ptr), nbytes, 3,  # D2D
                            _stream(stream))
    if rc != 0:
        raise RuntimeError(f"hipMemcpyAsync failed ({rc})")


def laplex_plan_perm(plan: Plan, side: int = 0, stream=None) -> torch.Tensor:
    """Copy of the plan's permutation (rank -> original index) as int64."""
    p = ctypes.c_void_p()
    _check(load().laplex_plan_perm(plan.handle, side, ctypes.byref(p)), "laplex_plan_perm")
    m = plan.n if side == 0 else plan.k
    out = torch.empty(m, dtype=torch.int32, device=plan.device)
    _copy_device(out, p.value, 4 * m, stream)
    return out.to(torch.int64)  # indices are below 2^31


def laplex_plan_sorted(plan: Plan, side: int = 0, stream=None) -> torch.Tensor:
    p = ctypes.c_void_p()
    _check(load().laplex_plan_sorted(plan.handle, side, ctypes.byref(p)), "laplex_plan_sorted")
    m = plan.n if side == 0 else plan.k
    out = torch.empty(m, dtype=torch.float32, device=plan.device)
    _copy_device(out, p.value, 4 * m, stream)
    return out


def laplex_plan_info(plan: Plan):
    n, k, f = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int()
    _check(load().laplex_plan_info(plan.handle, ctypes.byref(n), ctypes.byref(k), ctypes.byref(f)),
           "laplex_plan_info")
    return n.value, k.value, f.value


def laplex_plan_destroy(plan: Plan):
    plan.destroy()


# ---- tokens: routing by expert and the gated recurrence -------------------

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class Route(NamedTuple):
    """Token slots sorted by expert (see laplex_route in include/laplex.h)."""

    order: torch.Tensor    # int32 [tokens * slots]: slot of each row, -1 past the last
    place: torch.Tensor    # int32 [tokens, slots]: row of each slot, -1 if dropped
    offsets: torch.Tensor  # int32 [experts + 1]: first row of each expert


class Recurrence(NamedTuple):
    """What laplex_recur returns."""

    y: torch.Tensor
    final: torch.Tensor | None   # float32 [seqs, width], with final=True
    states: torch.Tensor | None  # for laplex_recur_backward, with keep=True


def _rows(t, name, dtype=None, shape=None):
    """(rows, width, values between rows) of a tensor [..., width] whose
    leading dimensions step evenly through memory."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise TypeError(f"{name} must be a CUDA tensor")
    if (t.dtype not in _DTYPES) if dtype is None else (t.dtype is not dtype):
        raise TypeError(f"{name} must be {dtype or 'float32, bfloat16 or float16'}")
    sizes = t.shape
    if shape is not None and sizes != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    if len(sizes) == 0:
        raise ValueError(f"{name} must have a last dimension")
    width = sizes[-1]
    if t.is_contiguous():
        return (sizes[0] if len(sizes) == 2 else t.numel() // max(width, 1)), width, max(width, 1)
    steps = t.stride()
    ok = width == 1 or steps[-1] == 1
    ld, rows = None, 1  # pitch of the rows so far, from the innermost leading dimension
    for n, step in zip(reversed(sizes[:-1]), reversed(steps[:-1])):
        if n != 1:
            if ld is None:
                ld = step
            elif step != ld * rows:
                ok = False
        rows *= n
    ld = width if ld is None else ld
    if not ok or ld < width:
        raise ValueError(f"{name} must have unit stride along its last dimension and evenly spaced rows")
    return rows, width, ld


def _flat(t, name, dtype, shape, device):
    """A contiguous tensor of one type and shape, or None."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous {dtype} tensor on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    return t


_HERE = contextlib.nullcontext()


def _launch(stream, device, *inputs):
    """(stream handle, context in which outputs and scratch are allocated):
    with a stream other than the current one they come from its own pool, and
    the inputs' memory is not given out again before that stream is done."""
    if stream is None:
        # the handle alone: a Stream object would cost as much as the launch
        s = torch._C._cuda_getCurrentRawStream(device.index)
        return s, _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    for t in inputs:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream, torch.cuda.stream(stream)


def _at(t):
    """A tensor's address, None for no tensor."""
    return None if t is None else t.data_ptr()


def _new_like(t):
    """A contiguous tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _scratch(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes > 0 else None


def _size(value, where):
    if value < 0:
        raise ValueError(f"{where}: sizes out of range")
    return value


def _route_parts(route, device):
    place, offsets = route.place, route.offsets
    if not (isinstance(place, torch.Tensor) and place.dtype is torch.int32 and place.device == device
            and place.dim() == 2 and place.is_contiguous()):
        raise TypeError(f"route.place must be a contiguous 2-D int32 tensor on {device}")
    if not (isinstance(offsets, torch.Tensor) and offsets.dtype is torch.int32 and offsets.device == device
            and offsets.dim() == 1 and offsets.is_contiguous()):
        raise TypeError(f"route.offsets must be a contiguous 1-D int32 tensor on {device}")
    tokens, slots = place.shape
    return place, offsets, tokens, slots, offsets.shape[0] - 1


def laplex_route(experts, n_experts: int, stream=None) -> Route:
    """Stable sort of token slots by expert: experts int32 or int64
    [tokens, slots] (or [tokens]); ids outside [0, n_experts) drop the slot."""
    if not (isinstance(experts, torch.Tensor) and experts.is_cuda and experts.is_contiguous()
            and experts.dtype in (torch.int32, torch.int64) and experts.dim() in (1, 2)):
        raise TypeError("experts must be a contiguous int32 or int64 CUDA tensor [tokens, slots]")
    tokens, slots = experts.shape[0], 1 if experts.dim() == 1 else experts.shape[1]
    lib, dev = load(), experts.device
    need = _size(lib.laplex_route_workspace(tokens, slots, n_experts), "laplex_route")
    s, ctx = _launch(stream, dev, experts)
    with ctx:
        order = torch.empty(tokens * slots, dtype=torch.int32, device=dev)
        place = torch.empty((tokens, slots), dtype=torch.int32, device=dev)
        offsets = torch.empty(n_experts + 1, dtype=torch.int32, device=dev)
        ws = _scratch(need, dev)
        _check(lib.laplex_route(_at(experts), int(experts.dtype == torch.int64), tokens, slots, n_experts,
                                _at(order), _at(place), _at(offsets), _at(ws), need, s), "laplex_route")
    return Route(order, place, offsets)


def laplex_dispatch(route: Route, x, stream=None):
    """Rows of x [tokens, width] at their places by expert
    [tokens * slots, width], 0 past the last kept slot.  Its gradient is
    laplex_combine(route, dxs)."""
    rows, width, ld = _rows(x, "x")
    place, offsets, tokens, slots, experts = _route_parts(route, x.device)
    if x.dim() != 2 or rows != tokens:
        raise ValueError(f"x must have shape [{tokens}][width]")
    s, ctx = _launch(stream, x.device, place, offsets, x)
    with ctx:
        xs = x.new_empty((tokens * slots, width))
        _check(load().laplex_dispatch(tokens, slots, experts, _at(place), _at(offsets), _DTYPES[x.dtype], width,
                                      _at(x), ld, _at(xs), width, s), "laplex_dispatch")
    return xs


def laplex_combine(route: Route, ys, weights=None, stream=None):
    """Expert rows ys [tokens * slots, width] back to their tokens
    [tokens, width], summed with float32 weights [tokens, slots] (None: ones)."""
    rows, width, ld = _rows(ys, "ys")
    place, _, tokens, slots, _ = _route_parts(route, ys.device)
    if ys.dim() != 2 or rows != tokens * slots:
        raise ValueError(f"ys must have shape [{tokens * slots}][width]")
    weights = _flat(weights, "weights", torch.float32, (tokens, slots), ys.device)
    s, ctx = _launch(stream, ys.device, place, ys, weights)
    with ctx:
        y = ys.new_empty((tokens, width))
        _check(load().laplex_combine(tokens, slots, _at(place), _DTYPES[ys.dtype], width, _at(ys), ld,
                                     _at(weights), _at(y), width, s), "laplex_combine")
    return y


def laplex_combine_backward(route: Route, dy, ys, weights, stream=None):
    """Gradients (dys, dweights) of laplex_combine with weights."""
    rows, width, ld = _rows(dy, "dy")
    place, offsets, tokens, slots, experts = _route_parts(route, dy.device)
    if dy.dim() != 2 or rows != tokens:
        raise ValueError(f"dy must have shape [{tokens}][width]")
    _, _, ldys = _rows(ys, "ys", dy.dtype, (tokens * slots, width))
    if ys.device != dy.device:
        raise ValueError(f"ys must be on {dy.device}")
    if weights is None:
        raise TypeError("weights must be given")
    weights = _flat(weights, "weights", torch.float32, (tokens, slots), dy.device)
    s, ctx = _launch(stream, dy.device, place, offsets, dy, ys, weights)
    with ctx:
        dys = dy.new_empty((tokens * slots, width))
        dw = weights.new_empty((tokens, slots))
        _check(load().laplex_combine_backward(tokens, slots, experts, _at(place), _at(offsets), _DTYPES[dy.dtype],
                                              width, _at(dy), ld, _at(ys), ldys, _at(weights), _at(dys), width,
                                              _at(dw), s), "laplex_combine_backward")
    return dys, dw


def _recur_parts(x, g, offsets, h0):
    """Sizes and pitches of a recurrence's inputs, checked."""
    n, width, ldx = _rows(x, "x")
    if x.dim() not in (2, 3) or (x.dim() == 3 and offsets is not None):
        raise ValueError("x must be [rows, width], or [seqs, rows, width] without offsets")
    if not isinstance(g, torch.Tensor) or g.shape[:-1] != x.shape[:-1]:
        raise ValueError("g must have x's leading dimensions")
    if g.dtype not in (x.dtype, torch.float32):
        raise TypeError("g must have x's type or be float32")
    _, heads, ldg = _rows(g, "g")
    if width < 1 or heads < 1 or width % heads:
        raise ValueError("g's last dimension must divide x's")
    dev = x.device
    if offsets is not None:
        if not (isinstance(offsets, torch.Tensor) and offsets.dim() == 1 and offsets.numel() > 1):
            raise TypeError("offsets must be an int32 tensor [seqs + 1]")
        _flat(offsets, "offsets", torch.int32, offsets.shape, dev)
        seqs = offsets.numel() - 1
    else:
        seqs = x.shape[0] if x.dim() == 3 else 1
    if g.device != dev:
        raise ValueError(f"g must be on {dev}")
    _flat(h0, "h0", torch.float32, (seqs, width), dev)
    return n, seqs, width, heads, ldx, ldg


def laplex_recur(x, g, offsets=None, h0=None, final: bool = False, keep: bool = False, stream=None) -> Recurrence:
    """h_t = exp(g_t) h_{t-1} + x_t along each sequence; y is h.

    x [rows, width] (one sequence, or those of int32 offsets [seqs + 1]) or
    [seqs, rows, width]; g [..., heads] of x's type or float32, one decay's
    logarithm for each width / heads neighbouring channels; h0 float32
    [seqs, width] or None.  final: also return the last states; keep: also
    return what laplex_recur_backward needs."""
    n, seqs, width, heads, ldx, ldg = _recur_parts(x, g, offsets, h0)
    lib, dev = load(), x.device
    need = _size(lib.laplex_recur_workspace(n, width, heads, 0), "laplex_recur")
    s, ctx = _launch(stream, dev, x, g, offsets, h0)
    with ctx:
        y = _new_like(x)
        hf = torch.empty((seqs, width), dtype=torch.float32, device=dev) if final else None
        states = torch.empty(lib.laplex_recur_states(n, width), dtype=torch.float32, device=dev) if keep else None
        ws = _scratch(need, dev)
        _check(lib.laplex_recur(n, seqs, _at(offsets), width, heads, _DTYPES[x.dtype], _DTYPES[g.dtype], _at(x), ldx,
                                _at(g), ldg, _at(h0), _at(y), width, _at(hf), _at(states), _at(ws), need, s),
               "laplex_recur")
    return Recurrence(y, hf, states)


def laplex_recur_backward(x, g, dy, states, offsets=None, h0=None, dfinal=None, want=("dx", "dg", "dh0"),
                          stream=None) -> dict:
    """Gradients of laplex_recur from dy (y's shape and type) and dfinal
    (float32 [seqs, width] or None); x, g, offsets and h0 as in the forward
    pass, states from it (keep=True).  Returns the requested tensors among
    dx, dg and dh0 (float32 [seqs, width])."""
    n, seqs, width, heads, ldx, ldg = _recur_parts(x, g, offsets, h0)
    dev = x.device
    _, _, lddy = _rows(dy, "dy", x.dtype, x.shape)
    if dy.device != dev:
        raise ValueError(f"dy must be on {dev}")
    lib = load()
    need = _size(lib.laplex_recur_workspace(n, width, heads, 1), "laplex_recur_backward")
    if not isinstance(states, torch.Tensor):
        raise TypeError("states must be those of laplex_recur(keep=True)")
    _flat(states, "states", torch.float32, (lib.laplex_recur_states(n, width),), dev)
    _flat(dfinal, "dfinal", torch.float32, (seqs, width), dev)
    s, ctx = _launch(stream, dev, x, g, dy, states, offsets, h0, dfinal)
    out = {}
    with ctx:
        if "dx" in want:
            out["dx"] = _new_like(x)
        if "dg" in want:
            out["dg"] = _new_like(g)
        if "dh0" in want:
            out["dh0"] = torch.empty((seqs, width), dtype=torch.float32, device=dev)
        ws = _scratch(need, dev)
        _check(lib.laplex_recur_backward(n, seqs, _at(offsets), width, heads, _DTYPES[x.dtype], _DTYPES[g.dtype],
                                         _at(x), ldx, _at(g), ldg, _at(h0), _at(states), _at(dy), lddy,
                                         _at(dfinal), _at(out.get("dx")), width, _at(out.get("dg")), heads,
                                         _at(out.get("dh0")), _at(ws), need, s), "laplex_recur_backward")
    return out


def laplex_recur_step(x, g, state, slots=None, stream=None):
    """One token for each request: state[slots[i]] = exp(g_i) state[slots[i]]
    + x_i in place (float32 [pool, width]); returns y [n, width], the new
    states in x's type.  slots int32 [n] (None: request i has state i); a
    slot outside the pool has no state and gives 0."""
    n, width, ldx = _rows(x, "x")
    if x.dim() != 2:
        raise ValueError("x must have shape [n][width]")
    if not isinstance(g, torch.Tensor) or g.dim() != 2 or g.shape[0] != n or g.shape[1] < 1 or width % g.shape[1]:
        raise ValueError("g must have shape [n][heads] with heads dividing the width")
    if g.dtype not in (x.dtype, torch.float32):
        raise TypeError("g must have x's type or be float32")
    _, heads, ldg = _rows(g, "g")
    dev = x.device
    if not isinstance(state, torch.Tensor) or state.dim() != 2:
        raise TypeError("state must be a float32 tensor [pool][width]")
    _flat(state, "state", torch.float32, (state.shape[0], width), dev)
    _flat(slots, "slots", torch.int32, (n,), dev)
    if g.device != dev:
        raise ValueError(f"g must be on {dev}")
    s, ctx = _launch(stream, dev, x, g, state, slots)
    with ctx:
        y = _new_like(x)
        _check(load().laplex_recur_step(n, state.shape[0], _at(slots), width, heads, _DTYPES[x.dtype],
                                        _DTYPES[g.dtype], _at(x), ldx, _at(g), ldg, _at(state), _at(y), width, s),
               "laplex_recur_step")
    return y


# ---- experts' products and the gated matrix memory -----------------------

def _device_offsets(offsets, device):
    """int32 offsets of groups, checked; the number of groups."""
    if not (isinstance(offsets, torch.Tensor) and offsets.dim() == 1 and offsets.numel() > 1):
        raise TypeError("offsets must be an int32 tensor [groups + 1]")
    _flat(offsets, "offsets", torch.int32, offsets.shape, device)
    return offsets.numel() - 1


def _matrices(w, name, dtype, device, experts):
    """(rows, columns, values between rows, values between experts) of w [experts, rows, columns]."""
    if not (isinstance(w, torch.Tensor) and w.dtype is dtype and w.device == device):
        raise TypeError(f"{name} must be a {dtype} tensor on {device}")
    if w.dim() != 3 or w.shape[0] != experts or 0 in w.shape:
        raise ValueError(f"{name} must have shape [{experts}][rows][columns]")
    _, rows, cols = w.shape
    pitch, ld, one = w.stride()
    ld = ld if rows > 1 else cols
    if (one != 1 and cols > 1) or ld < cols:
        raise ValueError(f"{name} must have unit stride along its last dimension and rows apart")
    return rows, cols, ld, pitch if experts > 1 else rows * ld


def _experts_parts(x, w, offsets, transpose):
    n, width, ldx = _rows(x, "x")
    if x.dim() != 2 or width < 1:
        raise ValueError("x must have shape [rows][width]")
    experts = _device_offsets(offsets, x.device)
    rows, cols, ldw, pitch = _matrices(w, "w", x.dtype, x.device, experts)
    if (rows if transpose else cols) != width:
        raise ValueError("w must be [experts][out][in], or [experts][in][out] with transpose, for rows of x of `in`")
    return n, experts, width, cols if transpose else rows, ldx, ldw, pitch


def laplex_experts(x, w, offsets, transpose: bool = False, stream=None):
    """y_r = w[e] x_r for the rows r of each expert e: x [rows, in] sorted by
    expert, offsets int32 [experts + 1] (those of a Route), w [experts, out,
    in], or [experts, in, out] with transpose.  Rows of no expert give 0."""
    n, experts, width, out, ldx, ldw, pitch = _experts_parts(x, w, offsets, transpose)
    s, ctx = _launch(stream, x.device, x, w, offsets)
    with ctx:
        y = x.new_empty((n, out))
        _check(load().laplex_experts(n, experts, _at(offsets), width, out, _DTYPES[x.dtype], int(transpose), _at(x),
                                     ldx, _at(w), ldw, pitch, _at(y), out, s), "laplex_experts")
    return y


def laplex_experts_backward(x, w, dy, offsets, transpose: bool = False, want=("dx", "dw"), stream=None) -> dict:
    """Gradients of laplex_experts from dy (y's shape and type): the
    requested tensors among dx and dw (w's shape and type)."""
    n, experts, width, out, ldx, ldw, pitch = _experts_parts(x, w, offsets, transpose)
    _, _, lddy = _rows(dy, "dy", x.dtype, (n, out))
    if dy.device != x.device:
        raise ValueError(f"dy must be on {x.device}")
    s, ctx = _launch(stream, x.device, x, w, dy, offsets)
    grads = {}
    with ctx:
        if "dx" in want:
            grads["dx"] = _new_like(x)
        if "dw" in want:
            grads["dw"] = w.new_empty(w.shape)
        rows, cols = w.shape[1:]
        _check(load().laplex_experts_backward(n, experts, _at(offsets), width, out, _DTYPES[x.dtype], int(transpose),
                                              _at(x), ldx, _at(w), ldw, pitch, _at(dy), lddy, _at(grads.get("dx")),
                                              width, _at(grads.get("dw")), cols, rows * cols, s),
               "laplex_experts_backward")
    return grads


def _head_rows(t, name, dtype, lead, device):
    """(heads, width of a head, values between rows) of a tensor [..., heads,
    width] whose rows are packed and evenly spaced."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype):
        raise TypeError(f"{name} must be a {dtype} CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    sizes = t.shape
    if len(sizes) != len(lead) + 2 or sizes[:-2] != lead or sizes[-1] < 1 or sizes[-2] < 1:
        raise ValueError(f"{name} must have shape {tuple(lead)} + [heads][width]")
    heads, width = sizes[-2:]
    if t.is_contiguous():
        return heads, width, heads * width
    if (width > 1 and t.stride(-1) != 1) or (heads > 1 and t.stride(-2) != width):
        raise ValueError(f"{name}'s heads must lie next to each other, their values too")
    rows, _, ld = _rows(t.select(-2, 0), name)
    if rows > 1 and ld < heads * width:
        raise ValueError(f"{name} must have rows apart")
    return heads, width, max(ld, heads * width)


def _attend_parts(q, k, v, g, offsets, h0):
    """Sizes and pitches of a matrix memory's inputs, checked."""
    n, heads, ldg = _rows(g, "g")
    lead = g.shape[:-1]
    if len(lead) not in (1, 2) or (len(lead) == 2 and offsets is not None) or heads < 1:
        raise ValueError("g must be [rows, heads], or [seqs, rows, heads] without offsets")
    dev = g.device
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPES:
        raise TypeError("q must be a float32, bfloat16 or float16 CUDA tensor")
    if g.dtype not in (q.dtype, torch.float32):
        raise TypeError("g must have q's type or be float32")
    hq, dk, ldq = _head_rows(q, "q", q.dtype, lead, dev)
    hk, dk2, ldk = _head_rows(k, "k", q.dtype, lead, dev)
    hv, dv, ldv = _head_rows(v, "v", q.dtype, lead, dev)
    if dk2 != dk:
        raise ValueError("q's and k's heads must have one width")
    if heads % hq or heads % hk or heads % hv:
        raise ValueError("the heads of q, k and v must each divide those of g")
    seqs = _device_offsets(offsets, dev) if offsets is not None else lead[0] if len(lead) == 2 else 1
    _flat(h0, "h0", torch.float32, (seqs, heads, dk, dv), dev)
    return n, seqs, (heads, hq, hk, hv, dk, dv), (ldq, ldk, ldv, ldg)


def laplex_attend(q, k, v, g, offsets=None, h0=None, scale: float = 1.0, final: bool = False, keep: bool = False,
                  stream=None) -> Recurrence:
    """Linear attention with decays: S_t = exp(g_t) S_{t-1} + k_t v_t^T, y_t =
    scale S_t^T q_t for each head along each sequence.

    g [rows, heads] (one sequence, or those of int32 offsets [seqs + 1]) or
    [seqs, rows, heads], of q's type or float32; q, k [..., some heads, dk], v
    [..., some heads, dv], their heads dividing g's; h0 float32 [seqs, heads,
    dk, dv] or None.  y is [..., heads, dv].  final: also return the last
    states; keep: also return what laplex_attend_backward needs."""
    n, seqs, sizes, (ldq, ldk, ldv, ldg) = _attend_parts(q, k, v, g, offsets, h0)
    heads, dk, dv = sizes[0], sizes[4], sizes[5]
    lib, dev, kind = load(), q.device, _DTYPES[q.dtype]
    need = _size(lib.laplex_attend_workspace(n, seqs, *sizes, kind, 0), "laplex_attend")
    s, ctx = _launch(stream, dev, q, k, v, g, offsets, h0)
    with ctx:
        y = q.new_empty((*g.shape, dv))
        hf = torch.empty((seqs, heads, dk, dv), dtype=torch.float32, device=dev) if final else None
        states = torch.empty(lib.laplex_attend_states(n, seqs, heads, dk, dv), dtype=torch.float32, device=dev) if keep else None
        ws = _scratch(need, dev)
        _check(lib.laplex_attend(n, seqs, _at(offsets), *sizes, kind, _DTYPES[g.dtype], scale, _at(q), ldq, _at(k),
                                 ldk, _at(v), ldv, _at(g), ldg, _at(h0), _at(y), heads * dv, _at(hf), _at(states),
                                 _at(ws), need, s), "laplex_attend")
    return Recurrence(y, hf, states)


def laplex_attend_backward(q, k, v, g, dy, states, offsets=None, h0=None, scale: float = 1.0, dfinal=None,
                           want=("dq", "dk", "dv", "dg", "dh0"), stream=None) -> dict:
    """Gradients of laplex_attend from dy (y's shape and type) and dfinal
    (float32 [seqs, heads, dk, dv] or None); the other inputs as in the
    forward pass, states from it (keep=True).  Returns the requested tensors
    among dq, dk, dv, dg and dh0."""
    n, seqs, sizes, (ldq, ldk, ldv, ldg) = _attend_parts(q, k, v, g, offsets, h0)
    heads, hq, hk, hv, dk, dv = sizes
    dev, kind = q.device, _DTYPES[q.dtype]
    hy, wy, lddy = _head_rows(dy, "dy", q.dtype, g.shape[:-1], dev)
    if (hy, wy) != (heads, dv):
        raise ValueError(f"dy must have shape {(*g.shape, dv)}")
    lib = load()
    need = _size(lib.laplex_attend_workspace(n, seqs, *sizes, kind, 1), "laplex_attend_backward")
    if not isinstance(states, torch.Tensor):
        raise TypeError("states must be those of laplex_attend(keep=True)")
    _flat(states, "states", torch.float32, (lib.laplex_attend_states(n, seqs, heads, dk, dv),), dev)
    _flat(dfinal, "dfinal", torch.float32, (seqs, heads, dk, dv), dev)
    s, ctx = _launch(stream, dev, q, k, v, g, dy, states, offsets, h0, dfinal)
    out = {}
    with ctx:
        for name, like in (("dq", q), ("dk", k), ("dv", v), ("dg", g)):
            if name in want:
                out[name] = _new_like(like)
        if "dh0" in want:
            out["dh0"] = torch.empty((seqs, heads, dk, dv), dtype=torch.float32, device=dev)
        ws = _scratch(need, dev)
        _check(lib.laplex_attend_backward(n, seqs, _at(offsets), *sizes, kind, _DTYPES[g.dtype], scale, _at(q), ldq,
                                          _at(k), ldk, _at(v), ldv, _at(g), ldg, _at(h0), _at(states), _at(dy), lddy,
                                          _at(dfinal), _at(out.get("dq")), hq * dk, _at(out.get("dk")), hk * dk,
                                          _at(out.get("dv")), hv * dv, _at(out.get("dg")), heads,
                                          _at(out.get("dh0")), _at(ws), need, s), "laplex_attend_backward")
    return out


def laplex_attend_step(q, k, v, g, state, slots=None, scale: float = 1.0, stream=None):
    """One token for each request, in place on state float32 [pool, heads, dk,
    dv]: S = exp(g_i) S + k_i v_i^T for S = state[slots[i]]; returns y [n,
    heads, dv] = scale S^T q_i.  slots int32 [n] (None: request i has state i);
    a slot outside the pool has no state and gives 0.  No two requests may
    share a slot."""
    if not isinstance(g, torch.Tensor) or g.dim() != 2:
        raise TypeError("g must be a CUDA tensor [n, heads]")
    n, _, sizes, (ldq, ldk, ldv, ldg) = _attend_parts(q, k, v, g, None, None)
    heads, dk, dv = sizes[0], sizes[4], sizes[5]
    dev = q.device
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise TypeError("state must be a float32 tensor [pool][heads][dk][dv]")
    _flat(state, "state", torch.float32, (state.shape[0], heads, dk, dv), dev)
    _flat(slots, "slots", torch.int32, (n,), dev)
    s, ctx = _launch(stream, dev, q, k, v, g, state, slots)
    with ctx:
        y = q.new_empty((n, heads, dv))
        _check(load().laplex_attend_step(n, state.shape[0], _at(slots), *sizes, _DTYPES[q.dtype], _DTYPES[g.dtype],
                                         scale, _at(q), ldq, _at(k), ldk, _at(v), ldv, _at(g), ldg, _at(state),
                                         _at(y), heads * dv, s), "laplex_attend_step")
    return y


# ---- kernel timing -------------------------------------------------------

def profile_enable(on: bool = True):
    load().laplex_profile_enable(int(on))


def profile_only(label: str | None = None):
    """Bracket only launches labelled `label` (None: every launch)."""
    load().laplex_profile_only(None if label is None else label.encode())


def profile_reset():
    load().laplex_profile_reset()


def profile_read() -> dict:
    """Collect pending events; returns {kernel name: (launches, total ms)}."""
    lib = load()
    _check(lib.laplex_profile_collect(), "laplex_profile_collect")
    out = {}
    i = 0
    while True:
        name, cnt, ms = ctypes.c_char_p(), ctypes.c_int64(), ctypes.c_double()
        if lib.laplex_profile_entry(i, ctypes.byref(name), ctypes.byref(cnt), ctypes.byref(ms)) != OK:
            break
        out[name.value.decode()] = (cnt.value, ms.value)
        i += 1
    return out
