"""Products in 8-bit integers with a scale for each token and channel: the
binding of dg_gemm_scaled (include/densegemm.h).  Checks of shapes, types,
strides and devices, one descriptor, one call on the current stream; nothing
allocated but C, if none is given, and the workspace of a float A.
"""
from __future__ import annotations

import ctypes
import struct
import sys

from . import DG_F32, DG_SUCCESS, DgError, _ACT, _DTYPE, _enum, _load
from .grouped import _bias, _check_offsets, _code, _launch, _output, _row_ld, _same_device, _there

DG_I8 = 3
DG_SCALED_FEW_ROWS, DG_SCALED_FEW_ELEMENTS = 4, 8192
_A_TYPE = dict(_DTYPE, i8=DG_I8)
_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class DgScaledDesc(ctypes.Structure):
    """Mirror of dg_scaled_desc."""
    _fields_ = ([("struct_size", ctypes.c_uint32)] +
                [(n, _i32) for n in ("a_type", "c_type", "scale_type", "bias_type", "act")] +
                [(n, _i64) for n in ("groups", "M", "N", "K", "lda", "ldb", "ldc", "stride_b", "stride_s",
                                     "stride_bias")] +
                [("alpha", _f32), ("beta", _f32), ("bias", _vp)])


_SIZE = ctypes.sizeof(DgScaledDesc)
_pack = struct.Struct("@I5i10q2fP").pack
_ARGS = [_vp] * 7 + [ctypes.c_size_t, _vp]
_bound = _packed = None


def _entry():
    """The library's functions of this module, bound once."""
    global _bound
    if _bound is None:
        lib, D = _load(), ctypes.POINTER(DgScaledDesc)
        for name, args in (("dg_gemm_scaled", [D] + _ARGS),
                           ("dg_gemm_scaled_workspace_size", [D, ctypes.POINTER(ctypes.c_size_t)]),
                           ("dg_gemm_scaled_describe", [D, ctypes.c_char_p, ctypes.c_size_t])):
            f = getattr(lib, name)
            f.argtypes, f.restype = args, ctypes.c_int
        _bound = lib
    return _bound


def _fast():
    """dg_gemm_scaled taking the descriptor's bytes."""
    global _packed
    if _packed is None:
        f = _load()["dg_gemm_scaled"]
        f.argtypes, f.restype = [ctypes.c_char_p] + _ARGS, ctypes.c_int
        _packed = f
    return _packed


def make_scaled_desc(M, N, K, *, groups=1, a_type="i8", c_type="bf16", scale_type="f32", lda=None, ldb=None,
                     ldc=None, stride_b=None, stride_s=None, stride_bias=None, alpha=1.0, beta=0.0, bias=None,
                     bias_type="f32", act="none"):
    """Fill a DgScaledDesc.  ``a_type``: "i8" or a float type; leading
    dimensions and strides default to the packed values; ``bias`` is a device
    address."""
    return DgScaledDesc(
        _SIZE, _enum(_A_TYPE, a_type), _enum(_DTYPE, c_type), _enum(_DTYPE, scale_type), _enum(_DTYPE, bias_type),
        _enum(_ACT, act), groups, M, N, K, max(1, K) if lda is None else lda, max(1, K) if ldb is None else ldb,
        max(1, N) if ldc is None else ldc, N * K if stride_b is None else stride_b,
        N if stride_s is None else stride_s, N if stride_bias is None else stride_bias, alpha, beta, bias)


def dg_gemm_scaled(desc, A, scale_a, B, scale_b, C, offsets=None, workspace=None, workspace_bytes=0, stream=None,
                   check=True):
    """Enqueue the product.  Operands: device addresses (int) or None; stream:
    a hipStream_t as int.  Returns the status; raises DgError on failure when
    ``check``."""
    st = _entry().dg_gemm_scaled(desc, A, scale_a, B, scale_b, C, offsets, workspace, workspace_bytes, stream)
    if check and st != DG_SUCCESS:
        raise DgError(st, "dg_gemm_scaled")
    return st


def dg_gemm_scaled_workspace_size(desc):
    n = ctypes.c_size_t(0)
    st = _entry().dg_gemm_scaled_workspace_size(desc, ctypes.byref(n))
    if st != DG_SUCCESS:
        raise DgError(st, "dg_gemm_scaled_workspace_size")
    return int(n.value)


def dg_gemm_scaled_describe(desc):
    buf = ctypes.create_string_buffer(256)
    st = _entry().dg_gemm_scaled_describe(desc, buf, len(buf))
    if st != DG_SUCCESS:
        raise DgError(st, "dg_gemm_scaled_describe")
    return buf.value.decode()


# ---- torch convenience -----------------------------------------------------------
def gemm_scaled(A, B, scale_a=None, scale_b=None, C=None, *, offsets=None, alpha=1.0, beta=0.0, bias=None,
                act="none", out_dtype=None, stream=None):
    """C[m, n] = act(alpha * scale_a[m] * scale_b[n] * sum_k A[m, k] * B[n, k]
    + beta * C[m, n] + bias[n]), the sum exact in 32-bit integers.

    A: int8 (M, K) with scale_a fp32 (M,), as quantize_rows makes them, or a
    float (M, K) whose rows are quantized on the way (scale_a None then).  B:
    int8 (N, K); scale_b: (N,) of any float type; None: ones.  With offsets
    (int32, groups + 1, on the GPU), B, scale_b and optionally bias have a
    leading dimension of groups, and each row of A uses its group's; rows of no
    group are left alone.  out_dtype defaults to a float A's type, else bf16.
    Rows of A and B that start on 16 bytes and even K run fastest (quantize_rows
    allocates them so, of weights too).  With stream (a hipStream_t as int) the
    call runs there, and C and the workspace are allocated there."""
    if stream is not None:
        return _there(stream, A, gemm_scaled, A, B, scale_a, scale_b, C, offsets=offsets, alpha=alpha, beta=beta,
                      bias=bias, act=act, out_dtype=out_dtype)
    torch = sys.modules["torch"]
    int8 = torch.int8
    ashape, bshape = A.shape, B.shape
    grouped = offsets is not None
    if len(ashape) != 2 or len(bshape) != (3 if grouped else 2) or ashape[1] != bshape[-1]:
        raise ValueError(f"A {tuple(ashape)} and B {tuple(bshape)}: (M, K) and ([groups,] N, K) are wanted")
    if B.dtype != int8:
        raise ValueError(f"B: {B.dtype}, int8 is wanted")
    M, K = ashape
    N = bshape[-2]
    device = A.get_device()
    own, ws, ws_bytes, sa = A.dtype != int8, None, 0, None
    if own:
        if scale_a is not None:
            raise ValueError("scale_a belongs to an int8 A; a float A gets its own")
    elif scale_a is not None:
        if scale_a.dtype != torch.float32 or tuple(scale_a.shape) != (M,) or not scale_a.is_contiguous():
            raise ValueError(f"scale_a: a contiguous fp32 tensor ({M},) is wanted")
        sa = scale_a.data_ptr()
    bstride = B.stride()
    groups, stride_b, stride_s = 1, 0, 0
    if grouped:
        groups, stride_b = bshape[0], bstride[0]
        _check_offsets(offsets, groups)
    sb, sb_type = None, DG_F32
    if scale_b is not None:
        if scale_b.shape != bshape[:-1] or (N > 1 and scale_b.stride(-1) != 1):
            raise ValueError(f"scale_b: shape {tuple(scale_b.shape)}, {tuple(bshape[:-1])} is wanted, the last "
                             "dimension contiguous")
        sb, sb_type = scale_b.data_ptr(), _code(scale_b)
        stride_s = scale_b.stride(0) if grouped else 0
    C = _output(C, (M, N), out_dtype or (None if own or C is not None else torch.bfloat16), A, beta)
    _same_device(device, B=B, C=C, offsets=offsets, bias=bias, scale_a=scale_a, scale_b=scale_b)
    bias_ptr, bias_type, stride_bias = _bias(bias, groups, N, grouped)
    if own and K and M and (M > DG_SCALED_FEW_ROWS or M * K > DG_SCALED_FEW_ELEMENTS or groups > 1):
        ws_bytes = M * (((K + 15) & -16) + 4)
        ws = torch.empty(ws_bytes, dtype=int8, device=A.device)
    desc = _pack(_SIZE, _code(A) if own else DG_I8, _code(C), sb_type, bias_type, _enum(_ACT, act), groups, M, N, K,
                 _row_ld(M, K, *A.stride(), "A"), _row_ld(N, K, *bstride[-2:], "B"),
                 _row_ld(M, N, *C.stride(), "C"), stride_b, stride_s, stride_bias, alpha, beta, bias_ptr)
    _launch(_fast(), "dg_gemm_scaled", device, None, desc, A.data_ptr(), sa, B.data_ptr(), sb, C.data_ptr(),
            offsets.data_ptr() if grouped else None, None if ws is None else ws.data_ptr(), ws_bytes)
    return C
