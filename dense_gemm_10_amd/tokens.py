"""Tokens sorted by group and back, and 8-bit codes of rows: the binding of
dg_dispatch, dg_spread, dg_combine, dg_combine_grad and dg_quantize
(include/densegemm.h).

Argument marshalling only, like the rest of the package: checks of shapes,
types, strides and devices, one descriptor, one call on the current stream.
Nothing is copied or cast, and nothing allocated but the results that are not
given.  With ``stream`` (a hipStream_t as int) the call runs there, and what it
allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes
import struct
import sys

from . import DG_F32, DG_SUCCESS, DgError, _DTYPE, _enum, _load
from .grouped import _code, _launch, _row_ld, _same_device, _there

_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class DgDispatchDesc(ctypes.Structure):
    """Mirror of dg_dispatch_desc."""
    _fields_ = ([("struct_size", ctypes.c_uint32)] + [(n, _i32) for n in ("x_type", "index_bits")] +
                [(n, _i64) for n in ("tokens", "top_k", "groups", "rows", "width", "ld_index", "ldx", "ldr")])


class DgCombineDesc(ctypes.Structure):
    """Mirror of dg_combine_desc."""
    _fields_ = ([("struct_size", ctypes.c_uint32)] + [(n, _i32) for n in ("z_type", "y_type", "w_type")] +
                [(n, _i64) for n in ("tokens", "top_k", "rows", "width", "ldz", "lddz", "ldy", "ldw")] +
                [("beta", _f32)])


class DgQuantizeDesc(ctypes.Structure):
    """Mirror of dg_quantize_desc."""
    _fields_ = ([("struct_size", ctypes.c_uint32), ("x_type", _i32)] +
                [(n, _i64) for n in ("tokens", "top_k", "rows", "width", "ldx", "ldq")])


_DISPATCH_SIZE, _COMBINE_SIZE = ctypes.sizeof(DgDispatchDesc), ctypes.sizeof(DgCombineDesc)
_QUANTIZE_SIZE = ctypes.sizeof(DgQuantizeDesc)
# the descriptors as bytes (native alignment; 0q pads the end as C does)
_pack_dispatch = struct.Struct("@I2i8q").pack
_pack_combine = struct.Struct("@I3i8qf0q").pack
_pack_quantize = struct.Struct("@Ii6q").pack

# pointers after the descriptor, the stream among them
_POINTERS = {"dg_dispatch": 7, "dg_spread": 4, "dg_combine": 5, "dg_combine_grad": 7, "dg_quantize": 5}
_DESCS = {"dg_dispatch": DgDispatchDesc, "dg_spread": DgDispatchDesc, "dg_combine": DgCombineDesc,
          "dg_combine_grad": DgCombineDesc, "dg_quantize": DgQuantizeDesc}
_typed, _packed = {}, {}


def _entry(name):
    """The library's function taking a descriptor structure."""
    f = _typed.get(name)
    if f is None:
        f = _load()[name]
        f.argtypes, f.restype = [ctypes.POINTER(_DESCS[name])] + [_vp] * _POINTERS[name], ctypes.c_int
        _typed[name] = f
    return f


def _fast(name):
    """The same taking the descriptor's bytes."""
    f = _packed.get(name)
    if f is None:
        f = _load()[name]
        f.argtypes, f.restype = [ctypes.c_char_p] + [_vp] * _POINTERS[name], ctypes.c_int
        _packed[name] = f
    return f


def make_dispatch_desc(tokens, top_k, groups, width=0, *, rows=None, x_type="bf16", index_bits=32,
                       ld_index=None, ldx=None, ldr=None):
    """Fill a DgDispatchDesc; leading dimensions default to the packed values,
    ``rows`` to tokens * top_k."""
    return DgDispatchDesc(
        _DISPATCH_SIZE, _enum(_DTYPE, x_type), index_bits, tokens, top_k, groups,
        tokens * top_k if rows is None else rows, width, max(1, top_k) if ld_index is None else ld_index,
        max(1, width) if ldx is None else ldx, max(1, width) if ldr is None else ldr)


def make_combine_desc(tokens, top_k, rows, width, *, z_type="bf16", y_type=None, w_type="f32", ldz=None,
                      lddz=None, ldy=None, ldw=None, beta=0.0):
    """Fill a DgCombineDesc; leading dimensions default to the packed values."""
    zt, packed = _enum(_DTYPE, z_type), max(1, width)
    return DgCombineDesc(
        _COMBINE_SIZE, zt, zt if y_type is None else _enum(_DTYPE, y_type), _enum(_DTYPE, w_type), tokens,
        top_k, rows, width, packed if ldz is None else ldz, packed if lddz is None else lddz,
        packed if ldy is None else ldy, max(1, top_k) if ldw is None else ldw, beta)


def make_quantize_desc(tokens, width, *, top_k=1, rows=None, x_type="bf16", ldx=None, ldq=None):
    """Fill a DgQuantizeDesc; leading dimensions default to the packed values."""
    return DgQuantizeDesc(
        _QUANTIZE_SIZE, _enum(_DTYPE, x_type), tokens, top_k, tokens * top_k if rows is None else rows, width,
        max(1, width) if ldx is None else ldx, max(1, width) if ldq is None else ldq)


# ---- the C ABI, one function per entry point -----------------------------------
def _call(name, check, desc, *args):
    st = _entry(name)(desc, *args)
    if check and st != DG_SUCCESS:
        raise DgError(st, name)
    return st


def dg_dispatch(desc, index, x, offsets, order, place, rows, stream=None, check=True):
    """Enqueue the sort, and the rows if x and rows are given.  Operands:
    device addresses (int) or None; stream: a hipStream_t as int.  Returns the
    status; raises DgError on failure when ``check``."""
    return _call("dg_dispatch", check, desc, index, x, offsets, order, place, rows, stream)


def dg_spread(desc, place, x, rows, stream=None, check=True):
    """Enqueue rows[place[t][j]] = x[t]; arguments as above."""
    return _call("dg_spread", check, desc, place, x, rows, stream)


def dg_combine(desc, z, place, weights, y, stream=None, check=True):
    """Enqueue the weighted sums; arguments as above."""
    return _call("dg_combine", check, desc, z, place, weights, y, stream)


def dg_combine_grad(desc, dy, z, place, weights, dz, dweights, stream=None, check=True):
    """Enqueue the gradients of dg_combine; arguments as above."""
    return _call("dg_combine_grad", check, desc, dy, z, place, weights, dz, dweights, stream)


def dg_quantize(desc, x, place, q, scales, stream=None, check=True):
    """Enqueue the codes and scales; arguments as above."""
    return _call("dg_quantize", check, desc, x, place, q, scales, stream)


# ---- torch convenience -----------------------------------------------------------
def _torch():
    return sys.modules["torch"]           # a tensor was passed: it is imported


def _ld(t, rows, cols, name):
    """Leading dimension of a row-major 2-D tensor."""
    return cols or 1 if t.is_contiguous() else _row_ld(rows, cols, *t.stride(), name)


def _matrix(t, name):
    """(rows, columns, leading dimension) of a row-major 2-D tensor."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: shape {tuple(shape)}, two dimensions are wanted")
    r, c = shape
    return r, c, _ld(t, r, c, name)


def _check_place(place):
    shape = place.shape
    if place.dtype != _torch().int32 or len(shape) != 2 or not place.is_contiguous():
        raise ValueError("place: a contiguous int32 tensor (tokens, top_k) is wanted")
    return shape


def _on_device(device, **tensors):
    """Raises unless all of them are on the GPU `device`."""
    if device < 0:
        _same_device(device)
    for t in tensors.values():
        if t is not None and t.get_device() != device:
            _same_device(device, **tensors)


def _result(t, shape, dtype, like, name):
    """t checked, or a new tensor."""
    if t is None:
        return _torch().empty(shape, dtype=dtype, device=like.device)
    if t.shape != shape or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, {dtype} {tuple(shape)} is wanted")
    return t


def _maps(index, groups):
    torch = _torch()
    shape, dtype = index.shape, index.dtype
    if len(shape) != 2 or (dtype != torch.int64 and dtype != torch.int32):
        raise ValueError("index: an int32 or int64 tensor (tokens, top_k) is wanted")
    tokens, top_k = shape
    if groups < 0:
        raise ValueError(f"groups {groups}")
    ld = _ld(index, tokens, top_k, "index")
    empty, i32, where = torch.empty, torch.int32, index.device
    return (tokens, top_k, ld, 64 if dtype == torch.int64 else 32, empty(groups + 1, dtype=i32, device=where),
            empty(tokens * top_k, dtype=i32, device=where), empty(shape, dtype=i32, device=where))


def sort_tokens(index, groups, *, stream=None):
    """The maps of dispatch_tokens alone: (offsets, order, place)."""
    if stream is not None:
        return _there(stream, index, sort_tokens, index, groups)
    tokens, top_k, ld, bits, offsets, order, place = _maps(index, groups)
    device = index.get_device()
    _same_device(device)
    desc = _pack_dispatch(_DISPATCH_SIZE, DG_F32, bits, tokens, top_k, groups, 0, 0, ld, 1, 1)
    _launch(_fast("dg_dispatch"), "dg_dispatch", device, None, desc, index.data_ptr(), None,
            offsets.data_ptr(), order.data_ptr(), place.data_ptr(), None)
    return offsets, order, place


def dispatch_tokens(x, index, groups, *, out=None, stream=None):
    """Rows of x sorted by the group that each (token, choice) slot names.

    x: (tokens, width), row-major.  index: int32 or int64 (tokens, top_k), a
    value outside [0, groups) for none.  Returns (rows, offsets, order,
    place): rows (tokens * top_k, width) with rows[place[t, j]] = x[t];
    offsets int32 (groups + 1,), as gemm_grouped takes them; order int32, the
    slot t * top_k + j of every row; place int32 (tokens, top_k), the row of
    every slot, -1 for none.  Slots of one group keep their order.  Rows from
    offsets[groups] on keep what ``out`` held (in rows allocated here: nothing
    defined) and have order -1."""
    if stream is not None:
        return _there(stream, x, dispatch_tokens, x, index, groups, out=out)
    n, width, ldx = _matrix(x, "x")
    tokens, top_k, ld, bits, offsets, order, place = _maps(index, groups)
    if n != tokens:
        raise ValueError(f"x has {n} rows, index {tokens}")
    rows = _result(out, (tokens * top_k, width), x.dtype, x, "out")
    device = x.get_device()
    _on_device(device, index=index, out=rows)
    desc = _pack_dispatch(_DISPATCH_SIZE, _code(x), bits, tokens, top_k, groups, tokens * top_k, width, ld, ldx,
                          _ld(rows, tokens * top_k, width, "out"))
    _launch(_fast("dg_dispatch"), "dg_dispatch", device, None, desc, index.data_ptr(), x.data_ptr(),
            offsets.data_ptr(), order.data_ptr(), place.data_ptr(), rows.data_ptr())
    return rows, offsets, order, place


def spread_tokens(x, place, *, out=None, stream=None):
    """rows[place[t, j]] = x[t] for every slot with a row: the rows of
    dispatch_tokens from its place, and the gradient of combine_tokens without
    weights.  ``out`` may have any number of rows; a place outside them is
    skipped.  Returns rows (tokens * top_k, width by default)."""
    if stream is not None:
        return _there(stream, x, spread_tokens, x, place, out=out)
    n, width, ldx = _matrix(x, "x")
    tokens, top_k = _check_place(place)
    if n != tokens:
        raise ValueError(f"x has {n} rows, place {tokens}")
    rows = _result(out, (tokens * top_k if out is None else out.shape[0], width), x.dtype, x, "out")
    device = x.get_device()
    _on_device(device, place=place, out=rows)
    desc = _pack_dispatch(_DISPATCH_SIZE, _code(x), 32, tokens, top_k, 0, rows.shape[0], width, max(1, top_k), ldx,
                          _ld(rows, rows.shape[0], width, "out"))
    _launch(_fast("dg_spread"), "dg_spread", device, None, desc, place.data_ptr(), x.data_ptr(),
            rows.data_ptr())
    return rows


def _weights(weights, shape):
    """(address, type, leading dimension)."""
    if weights is None:
        return None, DG_F32, max(1, shape[1])
    if weights.shape != shape:
        raise ValueError(f"weights: shape {tuple(weights.shape)}, {tuple(shape)} is wanted")
    return weights.data_ptr(), _code(weights), _ld(weights, *shape, "weights")


def combine_tokens(z, place, weights=None, y=None, *, beta=0.0, out_dtype=None, stream=None):
    """y[t] = sum_j weights[t, j] * z[place[t, j]] + beta * y[t], over the
    slots with a row of z.

    z: (rows, width), row-major.  place: int32 (tokens, top_k) of
    dispatch_tokens.  weights: (tokens, top_k) of any float type, or None for
    ones (the gradient of dispatch_tokens and spread_tokens).  y: z's type or
    fp32.  Returns y (tokens, width)."""
    if stream is not None:
        return _there(stream, z, combine_tokens, z, place, weights, y, beta=beta, out_dtype=out_dtype)
    rows, width, ldz = _matrix(z, "z")
    tokens, top_k = _check_place(place)
    if y is None and beta != 0.0:
        raise ValueError("beta != 0 needs an input y")
    y = _result(y, (tokens, width), out_dtype or (z.dtype if y is None else None), z, "y")
    device = z.get_device()
    _on_device(device, place=place, weights=weights, y=y)
    w, wt, ldw = _weights(weights, (tokens, top_k))
    desc = _pack_combine(_COMBINE_SIZE, _code(z), _code(y), wt, tokens, top_k, rows, width, ldz, ldz,
                         _ld(y, tokens, width, "y"), ldw, beta)
    _launch(_fast("dg_combine"), "dg_combine", device, None, desc, z.data_ptr(), place.data_ptr(), w,
            y.data_ptr())
    return y


def combine_tokens_grad(dy, z, place, weights, *, dz=None, stream=None):
    """Gradients of combine_tokens (beta 0): (dz, dweights) with
    dz[place[t, j]] = weights[t, j] * dy[t] and dweights[t, j] = <dy[t],
    z[place[t, j]]>, 0 for a slot without a row.  dy: (tokens, width), z's type
    or fp32; dweights has weights' type.  Rows that no slot has keep what
    ``dz`` held (in a dz allocated here: nothing defined)."""
    if stream is not None:
        return _there(stream, z, combine_tokens_grad, dy, z, place, weights, dz=dz)
    n, width, ldy = _matrix(dy, "dy")
    rows, zw, ldz = _matrix(z, "z")
    tokens, top_k = _check_place(place)
    if n != tokens or zw != width:
        raise ValueError(f"dy {tuple(dy.shape)}, z {tuple(z.shape)} and place {tuple(place.shape)} do not match")
    if weights is None:
        raise ValueError("weights are wanted (without any, the gradient is spread_tokens)")
    w, wt, ldw = _weights(weights, (tokens, top_k))
    dz = _result(dz, (rows, width), z.dtype, z, "dz")
    dw = _torch().empty((tokens, top_k), dtype=weights.dtype, device=z.device)
    device = z.get_device()
    _on_device(device, dy=dy, place=place, weights=weights, dz=dz)
    desc = _pack_combine(_COMBINE_SIZE, _code(z), _code(dy), wt, tokens, top_k, rows, width, ldz,
                         _ld(dz, rows, width, "dz"), ldy, ldw, 0.0)
    _launch(_fast("dg_combine_grad"), "dg_combine_grad", device, None, desc, dy.data_ptr(), z.data_ptr(),
            place.data_ptr(), w, dz.data_ptr(), dw.data_ptr())
    return dz, dw


def quantize_rows(x, place=None, q=None, scales=None, *, stream=None):
    """8-bit codes and scales of every row: scales[t] = max |x[t]| / 127 (fp32)
    and q[t] = x[t] / scales[t] to the nearest integer, ties to even, from the
    exact quotient.  A row of zeros has scale 0; one that holds an infinity or
    NaN has scale NaN and codes 0.

    x: (tokens, width), row-major.  With ``place`` (of dispatch_tokens) token
    t's codes and scale go to the rows place[t, j], and rows that no slot has
    keep what ``q`` and ``scales`` held (allocated here: nothing defined).
    Returns (q, scales): int8 (rows, width), each row starting on 16 bytes if
    allocated here, and fp32 (rows,)."""
    if stream is not None:
        return _there(stream, x, quantize_rows, x, place, q, scales)
    torch = _torch()
    tokens, width, ldx = _matrix(x, "x")
    top_k = 1
    if place is not None:
        n, top_k = _check_place(place)
        if n != tokens:
            raise ValueError(f"x has {tokens} rows, place {n}")
    rows = tokens * top_k if q is None or place is None else q.shape[0]
    if q is None:
        q = torch.empty((rows, max(16, (width + 15) // 16 * 16)), dtype=torch.int8, device=x.device)[:, :width]
    q = _result(q, (rows, width), torch.int8, x, "q")
    scales = _result(scales, (rows,), torch.float32, x, "scales")
    if not scales.is_contiguous():
        raise ValueError("scales: a contiguous tensor is wanted")
    device = x.get_device()
    _on_device(device, place=place, q=q, scales=scales)
    desc = _pack_quantize(_QUANTIZE_SIZE, _code(x), tokens, top_k, rows, width, ldx,
                          _ld(q, rows, width, "q"))
    _launch(_fast("dg_quantize"), "dg_quantize", device, None, desc, x.data_ptr(),
            None if place is None else place.data_ptr(), q.data_ptr(), scales.data_ptr())
    return q, scales
