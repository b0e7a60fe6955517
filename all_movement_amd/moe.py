"""The operators around the exchange for torch tensors (include/a2av_moe.h).

``route`` chooses each token's experts and makes the gather list and counts
that the exchange and the products take; ``gmm``, ``gmm_dx`` and ``gmm_dw`` are
the products grouped by expert and their gradients; ``combine`` returns the
rows to their tokens; ``mx4_quantize``, ``mx4_dequantize`` and ``gmm_mx4`` are
the microscaled 4-bit format and the product on it.

Every step runs in the HIP library.  Nothing is converted or copied: a tensor
that would need it is refused.  Rows may be strided, everything else is
contiguous.  Outputs that are not given are allocated; the work runs on the
tensors' device and on ``stream`` (default: torch's current stream there, which
is also the stream that outputs are allocated for).  As under
``torch.cuda.stream``, the order and the lifetime of operands across streams are
the caller's.  ``status``, an int32 tensor of one element, receives the code of a
check on device data that failed (it is never cleared); with ``check=True`` the
call waits and raises instead.

Gradients are calls of their own (``route_backward``, ``gmm_dx``, ``gmm_dw``,
``combine_backward``), for a training step or an autograd function to make; no
call records one, so that operands that require a gradient are refused unless
recording is off (``torch.no_grad()``).
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
from typing import NamedTuple

import torch

from . import a2av

MOE_EXPORTS = ["a2av_moe_route_workspace", "a2av_moe_route", "a2av_moe_route_backward",
               "a2av_moe_gmm", "a2av_moe_gmm_dx", "a2av_moe_gmm_dw", "a2av_moe_combine",
               "a2av_moe_combine_backward", "a2av_moe_mx4_quantize", "a2av_moe_mx4_dequantize",
               "a2av_moe_gmm_mx4"]

_DTYPE = {torch.float32: a2av.FP32, torch.float16: a2av.FP16, torch.bfloat16: a2av.BF16}
_lib = None


def lib() -> ctypes.CDLL:
    """liba2av.so with the signatures of include/a2av_moe.h."""
    global _lib
    if _lib is not None:
        return _lib
    L = a2av.lib()
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    sig = {
        "a2av_moe_route_workspace": [i64, i32, i32, ctypes.POINTER(i64)],
        "a2av_moe_route": [vp, i64, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, i64, vp],
        "a2av_moe_route_backward": [vp, i64, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp],
        "a2av_moe_gmm": [vp, i64, i64, vp, vp, vp, vp, i64, i64, i32, i64, i64, i32, vp, vp],
        "a2av_moe_gmm_dx": [vp, i64, vp, vp, vp, i64, i64, i32, i64, i64, i32, vp, vp],
        "a2av_moe_gmm_dw": [vp, i64, vp, i64, i64, vp, vp, vp, i64, i32, i64, i64, i32, i32, vp,
                            vp],
        "a2av_moe_combine": [vp, i64, i64, vp, vp, vp, i64, i64, i32, i64, i32, vp, vp],
        "a2av_moe_combine_backward": [vp, i64, vp, i64, i64, vp, vp, vp, i64, vp, i64, i32, i64,
                                      i32, vp, vp],
        "a2av_moe_mx4_quantize": [vp, i64, i64, i64, i32, vp, vp, vp],
        "a2av_moe_mx4_dequantize": [vp, vp, i64, i64, i32, vp, i64, vp],
        "a2av_moe_gmm_mx4": [vp, vp, i64, vp, vp, vp, vp, vp, i64, i64, i32, i64, i64, i32, vp,
                             vp],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    _lib = L
    return L


# ---------------------------------------------------------------- checks

def _matrix(t, name: str, cols: int | None = None, dtypes=None):
    """A 2-D tensor with contiguous rows: (pointer, row stride)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must have 2 dimensions, got {len(shape)}")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {tuple(dtypes)}, got {t.dtype}")
    rows, width = shape
    if cols is not None and width != cols:
        raise ValueError(f"{name} must have {cols} columns, got {width}")
    along, step = t.stride()
    if rows <= 1:
        along = width if width > 1 else 1
    if width > 1 and step != 1 or along < width:
        raise ValueError(f"{name} must have contiguous rows that do not overlap "
                         "(operands are never copied)")
    return t.data_ptr(), along


def _whole(t, name: str, shape, dtype):
    """A contiguous tensor of this shape and dtype: its pointer."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (operands are never copied)")
    return t.data_ptr()


def _device(*named):
    dev = named[0].device
    for t in named:
        if t is not None and t is not named[0] and t.device != dev:
            raise ValueError(f"operands on {dev} and {t.device}")
    if dev.type != "cuda":
        raise ValueError(f"operands must live on a GPU, not {dev}")
    return dev


def _recorded() -> None:
    """For an operand that requires a gradient."""
    if torch.is_grad_enabled():
        raise ValueError("an operand requires a gradient, which no call here records: the "
                         "gradients are calls of their own (use detach or torch.no_grad)")


def _elsewhere(dev, stream) -> bool:
    """Whether the call has to be made under another device or stream."""
    if stream is None:
        return torch._C._cuda_getDevice() != dev.index
    if stream.device != dev:
        raise ValueError(f"stream of {stream.device} for operands on {dev}")
    return True


@contextlib.contextmanager
def _there(dev, stream):
    """The tensors' device made current, and the stream on it."""
    with torch.cuda.device(dev):
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(dev)):
            yield


def _stream(dev) -> int:
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _status(status, check: bool, dev):
    """(tensor or None, pointer)."""
    if check and status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    if status is None:
        return None, None
    return status, _whole(status, "status", (1,), torch.int32)


def _done(st: int, what: str, status, check: bool) -> None:
    a2av._raise(st, what)
    if check:
        a2av._raise(int(status.item()), what + " (device-side checks)")


# ---------------------------------------------------------------- the router

class Routing(NamedTuple):
    experts: torch.Tensor  # int32 [tokens, k], -1 = empty slot
    weights: torch.Tensor  # float32 [tokens, k]
    counts: torch.Tensor   # int32 [experts]
    order: torch.Tensor    # int32 [tokens * k]: the token of each row in expert order
    place: torch.Tensor    # int32 [tokens, k]: the row of each slot, -1 = none


@functools.lru_cache(maxsize=256)
def route_workspace(tokens: int, experts: int, k: int) -> int:
    """Bytes of workspace that :func:`route` needs."""
    n = ctypes.c_int64()
    a2av._raise(lib().a2av_moe_route_workspace(tokens, experts, k, ctypes.byref(n)),
                "a2av_moe_route_workspace")
    return n.value


def route(logits, k: int, *, renormalize: bool = True, out: Routing | None = None,
          workspace=None, stream=None) -> Routing:
    """The ``k`` largest logits of each row [tokens, experts]: a :class:`Routing`."""
    p, stride = _matrix(logits, "logits", None, _DTYPE)
    T, E = logits.shape
    need = route_workspace(T, E, k)
    if logits.requires_grad:
        _recorded()
    dev = _device(logits, workspace, *(out or ()))
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return route(logits, k, renormalize=renormalize, out=out, workspace=workspace)
    n = T * k
    if out is None:
        ints = torch.empty(3, T, k, dtype=torch.int32, device=dev)
        experts, order, place = ints.unbind(0)
        weights = torch.empty(T, k, dtype=torch.float32, device=dev)
        counts = torch.empty(E, dtype=torch.int32, device=dev)
        out = Routing(experts, weights, counts, order.view(n), place)
        i = ints.data_ptr()
        ptr = (i, weights.data_ptr(), counts.data_ptr(), i + 4 * n, i + 8 * n)
    else:
        ptr = (_whole(out[0], "experts", (T, k), torch.int32),
               _whole(out[1], "weights", (T, k), torch.float32),
               _whole(out[2], "counts", (E,), torch.int32),
               _whole(out[3], "order", (n,), torch.int32),
               _whole(out[4], "place", (T, k), torch.int32))
    wp, wn = None, 0
    if need:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        wp, wn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = lib().a2av_moe_route(p, stride, T, E, k, int(renormalize), _DTYPE[logits.dtype], *ptr,
                              wp, wn, _stream(dev))
    a2av._raise(st, "a2av_moe_route")
    return out


def route_backward(logits, experts, weights, dweights, *, renormalize: bool = True, out=None,
                   stream=None):
    """dlogits of :func:`route`'s weights; ``logits``, ``experts``, ``weights`` and
    ``renormalize`` are the forward call's."""
    p, stride = _matrix(logits, "logits", None, _DTYPE)
    T, E = logits.shape
    k = experts.shape[-1]
    if (logits.requires_grad or weights.requires_grad or dweights.requires_grad or
            out is not None and out.requires_grad):
        _recorded()
    dev = _device(logits, experts, weights, dweights, out)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return route_backward(logits, experts, weights, dweights, renormalize=renormalize,
                                  out=out)
    ptr = (_whole(experts, "experts", (T, k), torch.int32),
           _whole(weights, "weights", (T, k), torch.float32),
           _whole(dweights, "dweights", (T, k), torch.float32))
    if out is None:
        out = torch.empty(T, E, dtype=logits.dtype, device=dev)
    op = _whole(out, "out", (T, E), logits.dtype)
    st = lib().a2av_moe_route_backward(p, stride, T, E, k, int(renormalize), _DTYPE[logits.dtype],
                                       *ptr, op, _stream(dev))
    a2av._raise(st, "a2av_moe_route_backward")
    return out


# ---------------------------------------------------------------- products grouped by expert

def _grouped(counts, index, E: int, rows: int):
    cp = _whole(counts, "counts", (E,), torch.int32)
    return cp, None if index is None else _whole(index, "index", (rows,), torch.int32)


def _rows_out(out, rows: int, cols: int, dtype, dev, name: str = "out"):
    """``out`` or a new [rows, cols] tensor: (tensor, pointer, row stride)."""
    if out is None:
        out = torch.empty(rows, cols, dtype=dtype, device=dev)
        return out, out.data_ptr(), max(cols, 1)
    p, stride = _matrix(out, name, cols, (dtype,))
    if out.requires_grad:
        _recorded()
    if out.shape[0] != rows:
        raise ValueError(f"{name} must have {rows} rows, got {out.shape[0]}")
    return out, p, stride


def gmm(x, w, counts, *, index=None, out=None, status=None, check: bool = False, stream=None):
    """y[r] = w[e(r)] @ x[index[r]] for the rows r in expert order: ``counts[0]``
    rows of expert 0, then ``counts[1]`` of expert 1, ...  ``x`` [x_rows, K],
    ``w`` [E, N, K]; there are as many rows as ``index`` entries (without one, as
    rows of ``x``).  Rows past the counts' sum are not written."""
    xp, xs = _matrix(x, "x", None, _DTYPE)
    if w.dim() != 3:
        raise ValueError(f"w must be [experts, N, K], got {tuple(w.shape)}")
    E, N, K = w.shape
    if x.shape[1] != K:
        raise ValueError(f"x must have {K} columns, got {x.shape[1]}")
    wp = _whole(w, "w", (E, N, K), x.dtype)
    rows = x.shape[0] if index is None else index.numel()
    cp, ip = _grouped(counts, index, E, rows)
    if x.requires_grad or w.requires_grad or out is not None and out.requires_grad:
        _recorded()
    dev = _device(x, w, counts, index, out, status)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return gmm(x, w, counts, index=index, out=out, status=status, check=check)
    out, op, os = _rows_out(out, rows, N, x.dtype, dev)
    status, sp = _status(status, check, dev)
    st = lib().a2av_moe_gmm(xp, xs, x.shape[0], wp, cp, ip, op, os, rows, E, N, K,
                            _DTYPE[x.dtype], sp, _stream(dev))
    _done(st, "a2av_moe_gmm", status, check)
    return out


def gmm_dx(dy, w, counts, *, out=None, status=None, check: bool = False, stream=None):
    """dx[r] = w[e(r)]^T @ dy[r]: the gradient of the (gathered) rows of x."""
    yp, ys = _matrix(dy, "dy", None, _DTYPE)
    if w.dim() != 3:
        raise ValueError(f"w must be [experts, N, K], got {tuple(w.shape)}")
    E, N, K = w.shape
    rows = dy.shape[0]
    if dy.shape[1] != N:
        raise ValueError(f"dy must have {N} columns, got {dy.shape[1]}")
    wp = _whole(w, "w", (E, N, K), dy.dtype)
    cp, _ = _grouped(counts, None, E, rows)
    if dy.requires_grad or w.requires_grad or out is not None and out.requires_grad:
        _recorded()
    dev = _device(dy, w, counts, out, status)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return gmm_dx(dy, w, counts, out=out, status=status, check=check)
    out, op, os = _rows_out(out, rows, K, dy.dtype, dev)
    status, sp = _status(status, check, dev)
    st = lib().a2av_moe_gmm_dx(yp, ys, wp, cp, op, os, rows, E, N, K, _DTYPE[dy.dtype], sp,
                               _stream(dev))
    _done(st, "a2av_moe_gmm_dx", status, check)
    return out


def gmm_dw(dy, x, counts, *, index=None, out=None, out_dtype=None, status=None,
           check: bool = False, stream=None):
    """dw[e] = sum over the rows r of e of dy[r] x[index[r]]^T, [E, N, K] in
    ``out_dtype`` (default: dy's; or float32).  Experts without rows get 0."""
    yp, ys = _matrix(dy, "dy", None, _DTYPE)
    xp, xs = _matrix(x, "x", None, (dy.dtype,))
    (rows, N), K, E = dy.shape, x.shape[1], counts.numel()
    cp, ip = _grouped(counts, index, E, rows)
    if out_dtype is None:
        out_dtype = dy.dtype if out is None else out.dtype
    if dy.requires_grad or x.requires_grad or out is not None and out.requires_grad:
        _recorded()
    dev = _device(dy, x, counts, index, out, status)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return gmm_dw(dy, x, counts, index=index, out=out, out_dtype=out_dtype, status=status,
                          check=check)
    if out is None:
        out = torch.empty(E, N, K, dtype=out_dtype, device=dev)
    op = _whole(out, "out", (E, N, K), out_dtype)
    status, sp = _status(status, check, dev)
    st = lib().a2av_moe_gmm_dw(yp, ys, xp, xs, x.shape[0], cp, ip, op, rows, E, N, K,
                               _DTYPE[dy.dtype], _DTYPE.get(out_dtype, -1), sp, _stream(dev))
    _done(st, "a2av_moe_gmm_dw", status, check)
    return out


# ---------------------------------------------------------------- the weighted return

def _slots(place, weights):
    if place.dim() != 2:
        raise ValueError(f"place must be [tokens, k], got {tuple(place.shape)}")
    T, k = place.shape
    pp = _whole(place, "place", (T, k), torch.int32)
    return T, k, pp, None if weights is None else _whole(weights, "weights", (T, k), torch.float32)


def combine(y, place, weights=None, *, out=None, status=None, check: bool = False, stream=None):
    """out[t] = sum over j of weights[t, j] * y[place[t, j]]; slots of -1 are left
    out, without ``weights`` each counts once."""
    yp, ys = _matrix(y, "y", None, _DTYPE)
    T, k, pp, wp = _slots(place, weights)
    if (y.requires_grad or weights is not None and weights.requires_grad or
            out is not None and out.requires_grad):
        _recorded()
    dev = _device(y, place, weights, out, status)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return combine(y, place, weights, out=out, status=status, check=check)
    rows, width = y.shape
    out, op, os = _rows_out(out, T, width, y.dtype, dev)
    status, sp = _status(status, check, dev)
    st = lib().a2av_moe_combine(yp, ys, rows, pp, wp, op, os, T, k, width, _DTYPE[y.dtype], sp,
                                _stream(dev))
    _done(st, "a2av_moe_combine", status, check)
    return out


def combine_backward(dout, y, place, weights=None, *, out=None, status=None, check: bool = False,
                     stream=None):
    """(dy, dweights) of :func:`combine`; dweights is None without ``weights``.
    Rows of dy that no slot names are not written."""
    dp, ds = _matrix(dout, "dout", None, _DTYPE)
    yp, ys = _matrix(y, "y", dout.shape[1], (dout.dtype,))
    T, k, pp, wp = _slots(place, weights)
    if dout.shape[0] != T:
        raise ValueError(f"dout must have {T} rows, got {dout.shape[0]}")
    if (dout.requires_grad or y.requires_grad or
            weights is not None and weights.requires_grad):
        _recorded()
    dev = _device(dout, y, place, weights, status, *(out or ()))
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return combine_backward(dout, y, place, weights, out=out, status=status, check=check)
    rows, width = y.shape
    dy, op, os = _rows_out(None if out is None else out[0], rows, width, y.dtype, dev, "dy")
    if out is None:
        dw = None if weights is None else torch.empty(T, k, dtype=torch.float32, device=dev)
    else:
        dw = out[1]
    gp = None if dw is None else _whole(dw, "dweights", (T, k), torch.float32)
    status, sp = _status(status, check, dev)
    st = lib().a2av_moe_combine_backward(dp, ds, yp, ys, rows, pp, wp, op, os, gp, T, k, width,
                                         _DTYPE[y.dtype], sp, _stream(dev))
    _done(st, "a2av_moe_combine_backward", status, check)
    return dy, dw


# ---------------------------------------------------------------- 4-bit rows

def mx4_quantize(x, *, out=None, stream=None):
    """(codes uint8 [rows, 16 * B], scales uint8 [rows, B]) of x [rows, cols], with
    B = ceil(cols / 32) blocks to a row."""
    p, stride = _matrix(x, "x", None, _DTYPE)
    rows, cols = x.shape
    B = (cols + 31) // 32
    if x.requires_grad:
        _recorded()
    dev = _device(x, *(out or ()))
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return mx4_quantize(x, out=out)
    if out is None:
        out = (torch.empty(rows, B * 16, dtype=torch.uint8, device=dev),
               torch.empty(rows, B, dtype=torch.uint8, device=dev))
    st = lib().a2av_moe_mx4_quantize(p, stride, rows, cols, _DTYPE[x.dtype],
                                     _whole(out[0], "codes", (rows, B * 16), torch.uint8),
                                     _whole(out[1], "scales", (rows, B), torch.uint8),
                                     _stream(dev))
    a2av._raise(st, "a2av_moe_mx4_quantize")
    return out


def mx4_dequantize(codes, scales, cols: int, dtype=torch.bfloat16, *, out=None, stream=None):
    """The values [rows, cols] of :func:`mx4_quantize`'s codes and scales."""
    rows, B = scales.shape[0], (cols + 31) // 32
    cp = _whole(codes, "codes", (rows, B * 16), torch.uint8)
    sp = _whole(scales, "scales", (rows, B), torch.uint8)
    dev = _device(codes, scales, out)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return mx4_dequantize(codes, scales, cols, dtype, out=out)
    out, op, os = _rows_out(out, rows, cols, dtype, dev)
    st = lib().a2av_moe_mx4_dequantize(cp, sp, rows, cols, _DTYPE.get(dtype, -1), op, os,
                                       _stream(dev))
    a2av._raise(st, "a2av_moe_mx4_dequantize")
    return out


def gmm_mx4(x_codes, x_scales, w_codes, w_scales, counts, *, index=None, dtype=torch.bfloat16,
            out=None, status=None, check: bool = False, stream=None):
    """:func:`gmm` on 4-bit rows and weights: ``x_codes`` [x_rows, 16 * B] and
    ``x_scales`` [x_rows, B] of :func:`mx4_quantize`, ``w_codes`` [E, N, 16 * B]
    and ``w_scales`` [E, N, B]; y in ``dtype``."""
    if w_scales.dim() != 3:
        raise ValueError(f"w_scales must be [experts, N, blocks], got {tuple(w_scales.shape)}")
    E, N, B = w_scales.shape
    x_rows = x_scales.shape[0]
    ptr = (_whole(x_codes, "x_codes", (x_rows, B * 16), torch.uint8),
           _whole(x_scales, "x_scales", (x_rows, B), torch.uint8), x_rows,
           _whole(w_codes, "w_codes", (E, N, B * 16), torch.uint8),
           _whole(w_scales, "w_scales", (E, N, B), torch.uint8))
    rows = x_rows if index is None else index.numel()
    cp, ip = _grouped(counts, index, E, rows)
    dev = _device(x_codes, x_scales, w_codes, w_scales, counts, index, out, status)
    if _elsewhere(dev, stream):
        with _there(dev, stream):
            return gmm_mx4(x_codes, x_scales, w_codes, w_scales, counts, index=index, dtype=dtype,
                           out=out, status=status, check=check)
    out, op, os = _rows_out(out, rows, N, dtype, dev)
    status, sp = _status(status, check, dev)
    st = lib().a2av_moe_gmm_mx4(*ptr, cp, ip, op, os, rows, E, N, B * 32, _DTYPE.get(dtype, -1),
                                sp, _stream(dev))
    _done(st, "a2av_moe_gmm_mx4", status, check)
    return out
