"""Products over groups of rows and products with 4-bit weights: the binding
of dg_gemm_grouped and dg_gemm_qweight (include/densegemm.h).

Argument marshalling only, like the rest of the package: checks of shapes,
types, strides and devices, one descriptor, one call on the current stream.
Nothing is copied, cast or allocated, apart from C when none is given.  With
``stream`` (a hipStream_t as int) the call runs there, and such a C belongs to
that stream.
"""
from __future__ import annotations

import ctypes
import struct
import sys

from . import (DG_BF16, DG_COL_MAJOR, DG_F16, DG_F32, DG_ROW_MAJOR, DG_SUCCESS, DgError, _ACT,
               _DTYPE, _ORDER, _enum, _load)

DG_RAGGED_M, DG_RAGGED_K = 0, 1
_RAGGED = {"m": DG_RAGGED_M, "k": DG_RAGGED_K}

_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class DgGroupedDesc(ctypes.Structure):
    """Mirror of dg_grouped_desc."""
    _fields_ = ([("struct_size", ctypes.c_uint32)] +
                [(n, _i32) for n in ("ragged", "a_type", "b_type", "c_type", "bias_type", "b_order",
                                     "act")] +
                [(n, _i64) for n in ("groups", "rows", "M", "N", "K", "lda", "ldb", "ldc", "stride_b",
                                     "stride_c", "stride_bias")] +
                [("alpha", _f32), ("beta", _f32), ("bias", _vp)])


class DgQweightDesc(ctypes.Structure):
    """Mirror of dg_qweight_desc."""
    _fields_ = ([("struct_size", ctypes.c_uint32)] +
                [(n, _i32) for n in ("a_type", "c_type", "scale_type", "bias_type", "act")] +
                [(n, _i64) for n in ("groups", "M", "N", "K", "group_size", "lda", "ldc", "ldq", "lds",
                                     "stride_q", "stride_s", "stride_bias")] +
                [("alpha", _f32), ("beta", _f32), ("bias", _vp)])


_GROUPED_SIZE, _QWEIGHT_SIZE = ctypes.sizeof(DgGroupedDesc), ctypes.sizeof(DgQweightDesc)
# the same descriptors as bytes (native alignment), in a quarter of the time
_pack_grouped, _pack_qweight = struct.Struct("@I7i11q2fP").pack, struct.Struct("@I5i12q2fP").pack
_bound = _packed_entries = None


def _entry():
    """The library's functions of this module, bound once."""
    global _bound
    if _bound is None:
        lib = _load()
        G, Q = ctypes.POINTER(DgGroupedDesc), ctypes.POINTER(DgQweightDesc)
        for name, args in (("dg_gemm_grouped", [G, _vp, _vp, _vp, _vp, _vp]),
                           ("dg_gemm_qweight", [Q, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
                           ("dg_gemm_grouped_describe", [G, ctypes.c_char_p, ctypes.c_size_t]),
                           ("dg_gemm_qweight_describe", [Q, ctypes.c_char_p, ctypes.c_size_t])):
            f = getattr(lib, name)
            f.argtypes, f.restype = args, ctypes.c_int
        _bound = lib
    return _bound


def _packed():
    """dg_gemm_grouped and dg_gemm_qweight taking a packed descriptor."""
    global _packed_entries
    if _packed_entries is None:
        lib = _load()
        grouped, qweight = lib["dg_gemm_grouped"], lib["dg_gemm_qweight"]
        grouped.argtypes, qweight.argtypes = [ctypes.c_char_p] + [_vp] * 5, [ctypes.c_char_p] + [_vp] * 7
        grouped.restype = qweight.restype = ctypes.c_int
        _packed_entries = grouped, qweight
    return _packed_entries


def make_grouped_desc(ragged, groups, rows, N, *, M=0, K=0, a_type="bf16", b_type=None, c_type=None,
                      b_order="row", lda=None, ldb=None, ldc=None, stride_b=None, stride_c=None,
                      stride_bias=None, alpha=1.0, beta=0.0, bias=None, bias_type="f32", act="none"):
    """Fill a DgGroupedDesc.  ``ragged``: "m" or "k"; leading dimensions and
    strides default to the packed values; ``bias`` is a device address."""
    r, bo = _enum(_RAGGED, ragged), _enum(_ORDER, b_order)
    at = _enum(_DTYPE, a_type)
    a_len = M if r == DG_RAGGED_K else K
    b_len = N if r == DG_RAGGED_K or bo == DG_ROW_MAJOR else K
    return DgGroupedDesc(
        _GROUPED_SIZE, r, at, at if b_type is None else _enum(_DTYPE, b_type),
        at if c_type is None else _enum(_DTYPE, c_type), _enum(_DTYPE, bias_type), bo,
        _enum(_ACT, act), groups, rows, M, N, K,
        max(1, a_len) if lda is None else lda, max(1, b_len) if ldb is None else ldb,
        max(1, N) if ldc is None else ldc, K * N if stride_b is None else stride_b,
        M * N if stride_c is None else stride_c, N if stride_bias is None else stride_bias,
        alpha, beta, bias)


def make_qweight_desc(M, N, K, group_size, *, groups=1, a_type="bf16", c_type=None, scale_type=None,
                      lda=None, ldc=None, ldq=None, lds=None, stride_q=None, stride_s=None,
                      stride_bias=None, alpha=1.0, beta=0.0, bias=None, bias_type="f32", act="none"):
    """Fill a DgQweightDesc; ldq and stride_q are in bytes."""
    at = _enum(_DTYPE, a_type)
    ldq = max(1, -(-K // 2)) if ldq is None else ldq
    lds = max(1, -(-K // group_size)) if lds is None else lds
    return DgQweightDesc(
        _QWEIGHT_SIZE, at, at if c_type is None else _enum(_DTYPE, c_type),
        at if scale_type is None else _enum(_DTYPE, scale_type), _enum(_DTYPE, bias_type),
        _enum(_ACT, act), groups, M, N, K, group_size, max(1, K) if lda is None else lda,
        max(1, N) if ldc is None else ldc, ldq, lds, N * ldq if stride_q is None else stride_q,
        N * lds if stride_s is None else stride_s, N if stride_bias is None else stride_bias,
        alpha, beta, bias)


# ---- the C ABI, one function per entry point -----------------------------------
def dg_gemm_grouped(desc, A, B, C, offsets, stream=None, check=True):
    """Enqueue the grouped product.  Operands: device addresses (int) or
    None; stream: a hipStream_t as int.  Returns the status; raises DgError
    on failure when ``check``."""
    st = _entry().dg_gemm_grouped(desc, A, B, C, offsets, stream)
    if check and st != DG_SUCCESS:
        raise DgError(st, "dg_gemm_grouped")
    return st


def dg_gemm_qweight(desc, A, Q, scales, zeros, C, offsets=None, stream=None, check=True):
    """Enqueue the product with 4-bit weights; arguments as above."""
    st = _entry().dg_gemm_qweight(desc, A, Q, scales, zeros, C, offsets, stream)
    if check and st != DG_SUCCESS:
        raise DgError(st, "dg_gemm_qweight")
    return st


def _describe(name, desc):
    buf = ctypes.create_string_buffer(256)
    st = getattr(_entry(), name)(desc, buf, len(buf))
    if st != DG_SUCCESS:
        raise DgError(st, name)
    return buf.value.decode()


def dg_gemm_grouped_describe(desc):
    return _describe("dg_gemm_grouped_describe", desc)


def dg_gemm_qweight_describe(desc):
    return _describe("dg_gemm_qweight_describe", desc)


# ---- torch convenience -----------------------------------------------------------
# A call on a few rows runs for a few microseconds on the GPU, so the checks
# below read each tensor's shape, strides, type and device once.
_types = None


def _code(t):
    """dg_dtype of a tensor."""
    global _types
    if _types is None:
        torch = sys.modules["torch"]       # a tensor was passed: it is imported
        _types = {torch.float32: DG_F32, torch.bfloat16: DG_BF16, torch.float16: DG_F16}
    code = _types.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _row_ld(rows, cols, r, c, name):
    """Leading dimension of a row-major matrix with strides (r, c)."""
    if (c != 1 and cols > 1) or (r < cols and rows > 1):
        raise ValueError(f"{name}: strides ({r}, {c}) are not row-major; pass a contiguous tensor")
    return r if rows > 1 and r > 0 else cols or 1


def _same_device(device, **others):
    if device < 0:
        raise ValueError("tensors must be on a GPU")
    for name, t in others.items():
        if t is not None and t.get_device() != device:
            raise ValueError(f"{name} is on another device than A")


def _check_offsets(offsets, groups):
    if offsets.dtype != sys.modules["torch"].int32 or offsets.dim() != 1 or offsets.numel() != groups + 1 or \
            not offsets.is_contiguous():
        raise ValueError(f"offsets: a contiguous int32 tensor of {groups + 1} entries is wanted")


def _output(C, shape, dtype, A, beta):
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs an input C")
        return sys.modules["torch"].empty(shape, dtype=dtype or A.dtype, device=A.device)
    if C.shape != shape:
        raise ValueError(f"C: shape {tuple(C.shape)}, {shape} is wanted")
    if dtype is not None and C.dtype != dtype:
        raise ValueError(f"C is {C.dtype}, out_dtype {dtype}")
    return C


def _bias(bias, groups, N, grouped):
    """(address, type, stride) of a bias of N values, or one per group."""
    if bias is None:
        return 0, DG_F32, 0
    if tuple(bias.shape) not in ((N,), (groups, N)) or (bias.dim() == 2 and not grouped):
        raise ValueError(f"bias: shape {tuple(bias.shape)} for {groups} groups of {N} columns")
    if N > 1 and bias.stride(-1) != 1:
        raise ValueError("bias: the last dimension must be contiguous")
    return bias.data_ptr(), _code(bias), bias.stride(0) if bias.dim() == 2 else 0


def _launch(entry, name, device, stream, *args):
    """entry(*args, stream) with `device` current, on its current stream by
    default (the raw handle: building a torch.cuda.Stream takes longer than
    the launch's argument checks)."""
    torch = sys.modules["torch"]
    if torch.cuda.current_device() != device:
        with torch.cuda.device(device):
            return _launch(entry, name, device, stream, *args)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device)
    st = entry(*args, stream)
    if st != DG_SUCCESS:
        raise DgError(st, name)


def _stream_of(stream, like):
    """The torch stream of a hipStream_t (int) on `like`'s device."""
    torch = sys.modules["torch"]
    device = like.get_device()
    _same_device(device)
    # ExternalStream(0) is a stream of torch's pool, not the null stream
    return torch.cuda.ExternalStream(stream, like.device) if stream else torch.cuda.default_stream(device)


def _there(stream, like, call, *args, **named):
    """call(...) with `stream` current: new tensors come from its own memory,
    which no other stream's pending work can still be using."""
    with sys.modules["torch"].cuda.stream(_stream_of(stream, like)):
        return call(*args, **named)


def gemm_grouped(A, B, offsets, C=None, *, alpha=1.0, beta=0.0, bias=None, act="none",
                 out_dtype=None, stream=None):
    """C[i] = act(alpha * A[i] @ B[e] + beta * C[i] + bias[e]) for the rows i
    of every group e, offsets[e] <= i < offsets[e + 1].

    A: (rows, K), row-major.  B: (groups, K, N), each matrix row- or
    column-major (``W.transpose(1, 2)`` gives the input gradient's product).
    offsets: int32 (groups + 1,) on the GPU.  bias: (groups, N) or (N,).
    Returns C (rows, N); rows of no group keep what they held (in a C
    allocated here: nothing defined)."""
    if stream is not None and C is None:
        return _there(stream, A, gemm_grouped, A, B, offsets, alpha=alpha, beta=beta, bias=bias, act=act,
                      out_dtype=out_dtype)
    ashape, bshape = A.shape, B.shape
    if len(ashape) != 2 or len(bshape) != 3 or ashape[1] != bshape[1]:
        raise ValueError(f"A {tuple(ashape)} and B {tuple(bshape)}: (rows, K) and (groups, K, N) are wanted")
    rows, K = ashape
    groups, _, N = bshape
    _check_offsets(offsets, groups)
    C = _output(C, (rows, N), out_dtype, A, beta)
    device = A.get_device()
    _same_device(device, B=B, C=C, offsets=offsets, bias=bias)
    sb, sk, sn = B.stride()
    if (sn == 1 or N <= 1) and (sk >= N or K <= 1):
        order, ldb = DG_ROW_MAJOR, max(sk, N, 1) if K > 1 else max(N, 1)
    elif (sk == 1 or K <= 1) and (sn >= K or N <= 1):
        order, ldb = DG_COL_MAJOR, max(sn, K, 1) if N > 1 else max(K, 1)
    else:
        raise ValueError(f"B: strides {B.stride()} are neither row- nor column-major")
    bias_ptr, bias_type, stride_bias = _bias(bias, groups, N, True)
    desc = _pack_grouped(_GROUPED_SIZE, DG_RAGGED_M, _code(A), _code(B), _code(C), bias_type, order,
                         _enum(_ACT, act), groups, rows, 0, N, K, _row_ld(rows, K, *A.stride(), "A"),
                         ldb, _row_ld(rows, N, *C.stride(), "C"), sb, 0, stride_bias, alpha, beta,
                         bias_ptr)
    _launch(_packed()[0], "dg_gemm_grouped", device, stream, desc, A.data_ptr(),
            B.data_ptr(), C.data_ptr(), offsets.data_ptr())
    return C


def gemm_grouped_k(A, B, offsets, C=None, *, alpha=1.0, beta=0.0, out_dtype=None, stream=None):
    """C[e] = alpha * A[:, rows of e] @ B[rows of e] + beta * C[e]: the
    weight gradient, with A = X.t() and B = the output's gradient.

    A: (M, rows), column-major (X is (rows, M) row-major).  B: (rows, N),
    row-major.  offsets as in gemm_grouped.  Returns C (groups, M, N); an
    empty group's is beta * C[e], or zeros."""
    if stream is not None and C is None:
        return _there(stream, A, gemm_grouped_k, A, B, offsets, alpha=alpha, beta=beta, out_dtype=out_dtype)
    ashape, bshape = A.shape, B.shape
    if len(ashape) != 2 or len(bshape) != 2 or ashape[1] != bshape[0]:
        raise ValueError(f"A {tuple(ashape)} and B {tuple(bshape)}: (M, rows) and (rows, N) are wanted")
    if offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError("offsets: an int32 tensor of groups + 1 entries is wanted")
    (M, rows), N, groups = ashape, bshape[1], offsets.numel() - 1
    _check_offsets(offsets, groups)
    C = _output(C, (groups, M, N), out_dtype, A, beta)
    device = A.get_device()
    _same_device(device, B=B, C=C, offsets=offsets)
    sm, sr = A.stride()
    sc, cr, cc = C.stride()
    desc = _pack_grouped(_GROUPED_SIZE, DG_RAGGED_K, _code(A), _code(B), _code(C), DG_F32,
                         DG_ROW_MAJOR, 0, groups, rows, M, N, 0,
                         _row_ld(rows, M, sr, sm, "A transposed"), _row_ld(rows, N, *B.stride(), "B"),
                         _row_ld(M, N, cr, cc, "C"), 0, sc, 0, alpha, beta, 0)
    _launch(_packed()[0], "dg_gemm_grouped", device, stream, desc, A.data_ptr(),
            B.data_ptr(), C.data_ptr(), offsets.data_ptr())
    return C


def gemm_qweight(A, Q, scales, zeros=None, C=None, *, group_size, offsets=None, alpha=1.0, beta=0.0,
                 bias=None, act="none", out_dtype=None, stream=None):
    """C = act(alpha * A @ W.T + beta * C + bias) with the 4-bit weights
    W[n, k] = scales[n, k // group_size] * (q[n, k] - zeros[n, k // group_size]).

    A: (M, K) bf16 or fp16.  Q: uint8 (N, ceil(K / 2)), q[n, 2j] in the low
    four bits of byte j and q[n, 2j + 1] in the high ones.  scales: (N,
    ceil(K / group_size)); zeros: uint8 of the same shape and strides, or
    None for 8.  With offsets (int32, groups + 1, on the GPU), Q, scales,
    zeros and optionally bias have a leading dimension of groups, and each
    row of A uses its group's weights; rows of no group are left alone."""
    if stream is not None and C is None:
        return _there(stream, A, gemm_qweight, A, Q, scales, zeros, group_size=group_size, offsets=offsets,
                      alpha=alpha, beta=beta, bias=bias, act=act, out_dtype=out_dtype)
    uint8 = sys.modules["torch"].uint8
    ashape, qshape, sshape = A.shape, Q.shape, scales.shape
    grouped = offsets is not None
    dims = 3 if grouped else 2
    if len(ashape) != 2 or len(qshape) != dims or len(sshape) != dims or group_size < 1:
        raise ValueError("A (M, K), Q ([groups,] N, ceil(K / 2)) and scales ([groups,] N, "
                         "ceil(K / group_size)) are wanted")
    M, K = ashape
    N, per_row = qshape[-2], -(-K // group_size)
    if Q.dtype != uint8 or qshape[-1] != (K + 1) // 2:
        raise ValueError(f"Q: uint8 rows of {(K + 1) // 2} bytes are wanted")
    if sshape[-1] != per_row or sshape[:-1] != qshape[:-1]:
        raise ValueError(f"scales: shape {tuple(sshape)} for {N} rows of {per_row} groups")
    qstride, sstride = Q.stride(), scales.stride()
    if zeros is not None and (zeros.dtype != uint8 or zeros.shape != sshape or
                              zeros.stride() != sstride):
        raise ValueError("zeros: uint8 with the shape and strides of scales is wanted")
    groups = stride_q = stride_s = 0
    if grouped:
        groups, stride_q, stride_s = qshape[0], qstride[0], sstride[0]
        _check_offsets(offsets, groups)
    C = _output(C, (M, N), out_dtype, A, beta)
    device = A.get_device()
    _same_device(device, Q=Q, scales=scales, zeros=zeros, C=C, offsets=offsets, bias=bias)
    bias_ptr, bias_type, stride_bias = _bias(bias, groups, N, grouped)
    desc = _pack_qweight(_QWEIGHT_SIZE, _code(A), _code(C), _code(scales), bias_type,
                         _enum(_ACT, act), groups if grouped else 1, M, N, K, group_size,
                         _row_ld(M, K, *A.stride(), "A"), _row_ld(M, N, *C.stride(), "C"),
                         _row_ld(N, qshape[-1], *qstride[-2:], "Q"),
                         _row_ld(N, per_row, *sstride[-2:], "scales"), stride_q, stride_s,
                         stride_bias, alpha, beta, bias_ptr)
    _launch(_packed()[1], "dg_gemm_qweight", device, stream, desc, A.data_ptr(),
            Q.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr(),
            C.data_ptr(), offsets.data_ptr() if grouped else None)
    return C
