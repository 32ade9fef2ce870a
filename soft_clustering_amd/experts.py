"""ctypes binding of include/gmm_experts.h: the lists of an assignment, rows
there and back, one linear model per component.

    idx, gamma = g.assign(x, m=2)                 # gmm.Gmm, the mixture
    routes = experts.route(idx, g.k)              # the components' lists
    y = experts.linear(h, w, bias, routes)        # W_k h + b_k on every row of list k
    out = experts.combine(y, gamma, routes)       # weighted sum back at the points

    dy, dgamma = experts.combine_backward(dout, y, gamma, routes)
    dh_rows, dw, db = experts.linear_backward(dy, h, w, routes)
    dh = experts.dispatch_backward(dh_rows, routes)

    codes, scales = experts.quantize4(w)          # serving: a few points at a time
    out = experts.linear4(h, idx, gamma, codes, scales, bias=bias)

Argument marshalling only; PyTorch provides device memory and streams, and no
call takes part in autograd.  Outputs and workspaces are allocated on the
stream of the call unless outputs are passed in.  Rows by slot have n * m
rows; those behind the last list (from offsets[k] on) are neither read nor
written, so in an output that was allocated here they hold nothing.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from .gmm import GmmError, _check, _lib

MAX_TOPM, MAX_LISTS, LINEAR4_MAX_N = 16, 4096, 1024
_CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

__all__ = ["Routes", "route", "dispatch", "dispatch_backward", "combine", "combine_backward", "linear",
           "linear_backward", "quantize4", "linear4", "GmmError"]


class Routes(NamedTuple):
    """The lists: offsets int32 [k + 1], entry int32 [n * m], slot int32 [n, m]."""
    offsets: torch.Tensor
    entry: torch.Tensor
    slot: torch.Tensor


class _CRoutes(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("m", ctypes.c_int32), ("k", ctypes.c_int32),
                ("offsets", ctypes.c_void_p), ("entry", ctypes.c_void_p), ("slot", ctypes.c_void_p)]


class _CLinear(ctypes.Structure):
    _fields_ = [("d_in", ctypes.c_int64), ("d_out", ctypes.c_int64), ("ldx", ctypes.c_int64),
                ("ldy", ctypes.c_int64), ("lddx", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("sorted_rows", ctypes.c_int32)]


def _declare():
    P, S, L, I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int32   # noqa: E741
    R, D, B = ctypes.POINTER(_CRoutes), ctypes.POINTER(_CLinear), ctypes.POINTER(ctypes.c_size_t)
    for name, args in {
        "gmm_route_workspace_bytes": [L, I, I, B],
        "gmm_route": [L, I, I, P, P, S, P, P, P, P],
        "gmm_dispatch": [R, L, I, P, L, P, L, P],
        "gmm_dispatch_backward": [R, L, I, P, L, P, L, P],
        "gmm_combine": [R, L, I, P, L, P, P, L, P],
        "gmm_combine_backward": [R, L, I, P, L, P, L, P, P, L, P, P],
        "gmm_linear": [R, D, P, P, P, P, P],
        "gmm_linear_backward_workspace_bytes": [L, I, I, D, B],
        "gmm_linear_backward": [R, D, P, P, P, P, P, P, P, S, P],
        "gmm_quantize4": [L, L, I, I, P, P, P, P],
        "gmm_linear4": [L, I, I, L, L, I, I, P, L, P, P, P, P, P, P, L, P],
    }.items():
        f = getattr(_lib, name)
        f.argtypes, f.restype = args, ctypes.c_int


_declare()


_I32, _F32 = torch.int32, torch.float32
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _call(fn, index, stream, tensors, launch):
    """launch(raw stream) with device `index` current, on `stream` (default: the
    device's current one).  On another stream than the current one, memory
    allocated by launch belongs to it, and the caller's tensors are marked as
    in use there."""
    if _current_device() != index:
        with torch.cuda.device(index):
            return _call(fn, index, stream, tensors, launch)
    raw = _raw_stream(index)
    if stream is None or stream.cuda_stream == raw:
        return launch(raw)
    if stream.device.index != index:
        raise ValueError(f"{fn}: the stream belongs to another device than the tensors")
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return launch(stream.cuda_stream)


def _fail(fn, what):
    raise ValueError(f"{fn}: {what}")


def _device_of(fn, tensors):
    """Index of the one GPU that holds the tensors (None: not given)."""
    index = None
    for t in tensors:
        if t is not None:
            i = t.get_device()
            if index is None:
                if i < 0 or not t.is_cuda:
                    _fail(fn, "tensors must be on a GPU")
                index = i
            elif i != index:
                _fail(fn, "tensors must be on one device")
    return index


def _flat(fn, name, t, dtype, shape):
    """A contiguous tensor of this type and shape."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _fail(fn, f"{name} must be a contiguous {dtype} tensor of shape {shape}")


def _rows(fn, name, t, rows, width, dtype):
    """Row stride of a 2-D tensor of `rows` rows with unit column stride."""
    if t.dtype is not dtype or t.shape != (rows, width):
        _fail(fn, f"{name} must be a {dtype} tensor of shape ({rows}, {width})")
    if rows <= 1 and width <= 1:
        return width
    ld, step = t.stride()
    if width > 1 and step != 1:
        _fail(fn, f"{name} must have unit column stride")
    if rows <= 1:
        return width
    if ld < width:
        _fail(fn, f"the rows of {name} must not overlap")
    return ld


def _apart(fn, out, *inputs):
    """An output that starts where an input starts is refused (any other overlap is the caller's to avoid)."""
    if out is not None and out.data_ptr() != 0:
        for t in inputs:
            if t is not None and t.data_ptr() == out.data_ptr():
                _fail(fn, "an output must not overlap an input")


def _code(fn, t):
    code = _CODE.get(t.dtype)
    if code is None:
        _fail(fn, "rows must be fp32, bf16 or fp16")
    return code


def _lists(fn, routes):
    """(n, m, k, C struct) of checked lists."""
    offsets, entry, slot = routes
    shape, lists = slot.shape, offsets.shape
    if len(shape) != 2 or len(lists) != 1 or entry.shape != (shape[0] * shape[1],):
        _fail(fn, "routes must be offsets [k + 1], entry [n * m], slot [n, m]")
    if not (offsets.dtype is entry.dtype is slot.dtype is _I32 and offsets.is_contiguous() and entry.is_contiguous()
            and slot.is_contiguous()):
        _fail(fn, "routes must be contiguous int32 tensors")
    n, m = shape
    k = lists[0] - 1
    return n, m, k, _CRoutes(n, m, k, offsets.data_ptr(), entry.data_ptr(), slot.data_ptr())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _workspace(nbytes, device):
    """Device bytes at a 256-byte boundary: (tensor to keep, address)."""
    if nbytes == 0:
        return None, None
    t = torch.empty(nbytes + 255, dtype=torch.uint8, device=device)
    return t, (t.data_ptr() + 255) & ~255


def route(idx, k, out=None, stream=None) -> Routes:
    """The lists of an assignment idx int32 [n, m] (as Gmm.assign returns it):
    list k holds the entries point * m + column with idx == k, in order;
    entries outside [0, k) are in no list (slot -1)."""
    if idx.dtype != torch.int32 or idx.dim() != 2 or not idx.is_contiguous():
        _fail("route", "idx must be a contiguous int32 tensor [n, m]")
    n, m = idx.shape
    k = int(k)
    need = ctypes.c_size_t(0)
    _check(_lib.gmm_route_workspace_bytes(n, m, k, ctypes.byref(need)), "gmm_route_workspace_bytes")
    if out is not None:
        _flat("route", "offsets", out.offsets, _I32, (k + 1,))
        _flat("route", "entry", out.entry, _I32, (n * m,))
        _flat("route", "slot", out.slot, _I32, (n, m))
    index = _device_of("route", (idx, *(out or ())))

    def launch(raw):
        r = out
        if r is None:
            new = lambda *shape: torch.empty(shape, dtype=torch.int32, device=idx.device)   # noqa: E731
            r = Routes(new(k + 1), new(n * m), new(n, m))
        keep, ws = _workspace(need.value, idx.device)
        _check(_lib.gmm_route(n, m, k, idx.data_ptr(), ws, need.value, r.offsets.data_ptr(), r.entry.data_ptr(),
                              r.slot.data_ptr(), raw), "gmm_route")
        return r
    return _call("route", index, stream, (idx, *(out or ())), launch)


def _one_output(fn, lib_fn, routes, src, src_rows, out, out_rows, gamma, stream):
    """Rows in, rows out: dispatch, its gradient and combine."""
    if src.dim() != 2:
        _fail(fn, "rows must be a 2-D tensor")
    code, d = _code(fn, src), src.shape[1]
    n, m, k, c = _lists(fn, routes)
    ld_in = _rows(fn, "the input", src, src_rows(n, m), d, src.dtype)
    ld_out = d if out is None else _rows(fn, "out", out, out_rows(n, m), d, src.dtype)
    if gamma is not None:
        _flat(fn, "gamma", gamma, _F32, (n, m))
    _apart(fn, out, src, gamma)
    tensors = (*routes, src, out, gamma)
    index = _device_of(fn, tensors)

    def launch(raw):
        o = torch.empty((out_rows(n, m), d), dtype=src.dtype, device=src.device) if out is None else out
        weights = () if gamma is None else (gamma.data_ptr(),)
        _check(lib_fn(ctypes.byref(c), d, code, src.data_ptr(), ld_in, *weights, o.data_ptr(), ld_out, raw), fn)
        return o
    return _call(fn, index, stream, tensors, launch)


def _by_point(n, m):
    return n


def _by_slot(n, m):
    return n * m


def dispatch(x, routes, out=None, stream=None):
    """The points' rows x [n, d] as rows by slot [n * m, d]."""
    return _one_output("dispatch", _lib.gmm_dispatch, routes, x, _by_point, out, _by_slot, None, stream)


def dispatch_backward(dy, routes, out=None, stream=None):
    """Gradient of dispatch: the rows by slot dy summed at their points, [n, d]."""
    return _one_output("dispatch_backward", _lib.gmm_dispatch_backward, routes, dy, _by_slot, out, _by_point, None,
                       stream)


def combine(z, gamma, routes, out=None, stream=None):
    """The rows by slot z, weighted with gamma fp32 [n, m] and summed at their points, [n, d]."""
    if gamma is None:
        _fail("combine", "gamma must be a contiguous fp32 tensor [n, m]")
    return _one_output("combine", _lib.gmm_combine, routes, z, _by_slot, out, _by_point, gamma, stream)


def combine_backward(dout, z, gamma, routes, dz=None, dgamma=None, need=(True, True), stream=None):
    """Gradients of combine: (dz rows by slot, dgamma fp32 [n, m]); need says
    which are computed (None for the other; z may be None without dgamma)."""
    fn = "combine_backward"
    need_z, need_g = need
    if dout.dim() != 2:
        _fail(fn, "rows must be a 2-D tensor")
    code, d = _code(fn, dout), dout.shape[1]
    n, m, k, c = _lists(fn, routes)
    lddo = _rows(fn, "dout", dout, n, d, dout.dtype)
    if need_g and z is None:
        _fail(fn, "z is needed for dgamma")
    ldz = _rows(fn, "z", z, n * m, d, dout.dtype) if need_g else d
    _flat(fn, "gamma", gamma, _F32, (n, m))
    lddz = d if dz is None else _rows(fn, "dz", dz, n * m, d, dout.dtype)
    if dgamma is not None:
        _flat(fn, "dgamma", dgamma, _F32, (n, m))
    _apart(fn, dz, dout, z, gamma)
    _apart(fn, dgamma, dout, z, gamma, dz)
    tensors = (*routes, dout, z, gamma, dz, dgamma)
    index = _device_of(fn, tensors)

    def launch(raw):
        oz, og = dz if need_z else None, dgamma if need_g else None
        if need_z and oz is None:
            oz = torch.empty((n * m, d), dtype=dout.dtype, device=dout.device)
        if need_g and og is None:
            og = torch.empty((n, m), dtype=torch.float32, device=dout.device)
        _check(_lib.gmm_combine_backward(ctypes.byref(c), d, code, dout.data_ptr(), lddo, _ptr(z) if need_g else None,
                                         ldz, gamma.data_ptr(), _ptr(oz), lddz, _ptr(og), raw), fn)
        return oz, og
    return _call(fn, index, stream, tensors, launch)


def linear(x, w, bias, routes, sorted_rows=False, out=None, stream=None):
    """y = W_k x + b_k on every row of list k, as rows by slot [n * m, d_out].
    x: the points' rows [n, d_in], or with sorted_rows rows by slot; w [k,
    d_out, d_in] of x's type; bias fp32 [k, d_out] or None."""
    fn = "linear"
    if w.dim() != 3:
        _fail(fn, "w must be [k, d_out, d_in]")
    code = _code(fn, x)
    n, m, k, c = _lists(fn, routes)
    do, di = w.shape[1], w.shape[2]
    _flat(fn, "w", w, x.dtype, (k, do, di))
    ldx = _rows(fn, "x", x, n * m if sorted_rows else n, di, x.dtype)
    if bias is not None:
        _flat(fn, "bias", bias, _F32, (k, do))
    ldy = do if out is None else _rows(fn, "out", out, n * m, do, x.dtype)
    _apart(fn, out, x, w, bias)
    tensors = (*routes, x, w, bias, out)
    index = _device_of(fn, tensors)
    desc = _CLinear(di, do, ldx, ldy, di, code, 1 if sorted_rows else 0)

    def launch(raw):
        y = torch.empty((n * m, do), dtype=x.dtype, device=x.device) if out is None else out
        _check(_lib.gmm_linear(ctypes.byref(c), ctypes.byref(desc), x.data_ptr(), w.data_ptr(), _ptr(bias),
                               y.data_ptr(), raw), fn)
        return y
    return _call(fn, index, stream, tensors, launch)


def linear_backward(dy, x, w, routes, sorted_rows=False, dx=None, dw=None, db=None, need=(True, True, True),
                    stream=None):
    """Gradients of linear: (dx rows by slot [n * m, d_in], dw fp32 [k, d_out,
    d_in], db fp32 [k, d_out]); need says which are computed (None for the
    others; db needs dw; w may be given as its shape when dx is not needed, x may be None without dw)."""
    fn = "linear_backward"
    need_x, need_w, need_b = need
    if need_b and not need_w:
        _fail(fn, "db is computed with dw")
    shape = tuple(w) if isinstance(w, (tuple, list, torch.Size)) else tuple(w.shape)
    if len(shape) != 3:
        _fail(fn, "w must be [k, d_out, d_in]")
    code = _code(fn, dy)
    n, m, k, c = _lists(fn, routes)
    _, do, di = shape
    wt = w if torch.is_tensor(w) else None
    if shape[0] != k or (need_x and wt is None) or (need_w and x is None):
        _fail(fn, "w must be [k, d_out, d_in]; dx needs w, dw needs x")
    if wt is not None:
        _flat(fn, "w", wt, dy.dtype, shape)
    lddy = _rows(fn, "dy", dy, n * m, do, dy.dtype)
    ldx = _rows(fn, "x", x, n * m if sorted_rows else n, di, dy.dtype) if need_w else di
    lddx = di if dx is None else _rows(fn, "dx", dx, n * m, di, dy.dtype)
    if dw is not None:
        _flat(fn, "dw", dw, torch.float32, shape)
    if db is not None:
        _flat(fn, "db", db, _F32, (k, do))
    for o in (dx, dw, db):
        _apart(fn, o, dy, x, wt)
    tensors = (*routes, dy, x, wt, dx, dw, db)
    index = _device_of(fn, tensors)
    desc = _CLinear(di, do, ldx, lddy, lddx, code, 1 if sorted_rows else 0)
    ws_bytes = ctypes.c_size_t(0)
    if need_w:
        _check(_lib.gmm_linear_backward_workspace_bytes(n, m, k, ctypes.byref(desc), ctypes.byref(ws_bytes)),
               "gmm_linear_backward_workspace_bytes")

    def launch(raw):
        ox, ow, ob = dx if need_x else None, dw if need_w else None, db if need_b else None
        if need_x and ox is None:
            ox = torch.empty((n * m, di), dtype=dy.dtype, device=dy.device)
        if need_w and ow is None:
            ow = torch.empty(shape, dtype=torch.float32, device=dy.device)
        if need_b and ob is None:
            ob = torch.empty((k, do), dtype=torch.float32, device=dy.device)
        keep, ws = _workspace(ws_bytes.value, dy.device)
        _check(_lib.gmm_linear_backward(ctypes.byref(c), ctypes.byref(desc), dy.data_ptr(),
                                        _ptr(x) if need_w else None, _ptr(wt) if need_x else None, _ptr(ox), _ptr(ow),
                                        _ptr(ob), ws, ws_bytes.value, raw), fn)
        return ox, ow, ob
    return _call(fn, index, stream, tensors, launch)


def quantize4(w, group=128, stream=None):
    """Weights w [..., d_in] in 4 bits: (codes uint8 [..., (d_in + 1) // 2],
    scales bf16 [..., ceil(d_in / group)]), w ~ (code - 8) * scale of its group."""
    fn = "quantize4"
    code = _code(fn, w)
    if w.dim() < 1 or not w.is_contiguous():
        _fail(fn, "w must be contiguous, [..., d_in]")
    index = _device_of(fn, (w,))
    d_in = w.shape[-1]
    rows = w.numel() // d_in if d_in else 0

    def launch(raw):
        codes = torch.empty((*w.shape[:-1], (d_in + 1) // 2), dtype=torch.uint8, device=w.device)
        scales = torch.empty((*w.shape[:-1], -(-d_in // group) if group > 0 else 0), dtype=torch.bfloat16,
                             device=w.device)
        _check(_lib.gmm_quantize4(rows, d_in, int(group), code, w.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                                  raw), "gmm_quantize4")
        return codes, scales
    return _call(fn, index, stream, (w,), launch)


def linear4(x, idx, gamma, codes, scales, group=128, bias=None, out=None, stream=None):
    """The weighted sum over a point's components of W_k x + b_k, W_k in 4
    bits, straight from the assignment idx int32 [n, m], gamma fp32 [n, m]: [n,
    d_out].  For a few points (n <= 1024).  codes [k, d_out, (d_in + 1) // 2]
    and scales [k, d_out, ceil(d_in / group)] as quantize4 writes them."""
    fn = "linear4"
    if x.dim() != 2 or idx.dim() != 2 or codes.dim() != 3:
        _fail(fn, "x must be [n, d_in], idx [n, m], codes [k, d_out, (d_in + 1) // 2]")
    code = _code(fn, x)
    n, di = x.shape
    m = idx.shape[1]
    k, do = codes.shape[0], codes.shape[1]
    if group not in (32, 64, 128):
        _fail(fn, "group must be 32, 64 or 128")
    ldx = _rows(fn, "x", x, n, di, x.dtype)
    _flat(fn, "idx", idx, _I32, (n, m))
    _flat(fn, "gamma", gamma, _F32, (n, m))
    _flat(fn, "codes", codes, torch.uint8, (k, do, (di + 1) // 2))
    _flat(fn, "scales", scales, torch.bfloat16, (k, do, -(-di // group)))
    if bias is not None:
        _flat(fn, "bias", bias, _F32, (k, do))
    ldo = do if out is None else _rows(fn, "out", out, n, do, x.dtype)
    _apart(fn, out, x)
    tensors = (x, idx, gamma, codes, scales, bias, out)
    index = _device_of(fn, tensors)

    def launch(raw):
        o = torch.empty((n, do), dtype=x.dtype, device=x.device) if out is None else out
        _check(_lib.gmm_linear4(n, m, k, di, do, group, code, x.data_ptr(), ldx, idx.data_ptr(), gamma.data_ptr(),
                                codes.data_ptr(), scales.data_ptr(), _ptr(bias), o.data_ptr(), ldo, raw), fn)
        return o
    return _call(fn, index, stream, tensors, launch)
