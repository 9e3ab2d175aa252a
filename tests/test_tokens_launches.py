"""What the host side of dg_combine and dg_combine_grad hands to the kernels,
with the launchers replaced: no kernel is given work on an operand that the
call may leave out."""
import ctypes
import os
import subprocess

import pytest

import dense_gemm_10_amd as dg
from conftest import ROOT
from dense_gemm_10_amd.build import COMMON_FLAGS, CSRC, HIPCC

P1, P2, P3, P4, P5, P6 = (i << 56 for i in range(1, 7))      # never dereferenced
VP = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("no hipcc")
    out = tmp_path_factory.mktemp("launches")
    objs = []
    for src in (os.path.join(CSRC, "tokens_api.cpp"), os.path.join(ROOT, "tests", "tokens_record.hip")):
        objs.append(str(out / (os.path.basename(src) + ".o")))
        subprocess.run([HIPCC] + COMMON_FLAGS + ["-I", CSRC, "-x", "hip", "-c", src, "-o", objs[-1]], check=True,
                       capture_output=True)
    so = str(out / "librecord.so")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", so] + objs, check=True,
                   capture_output=True)
    lib = ctypes.CDLL(so)
    lib.dg_combine.argtypes = [ctypes.POINTER(dg.DgCombineDesc)] + [VP] * 5
    lib.dg_combine_grad.argtypes = [ctypes.POINTER(dg.DgCombineDesc)] + [VP] * 7
    return lib


def _last(lib):
    v = (ctypes.c_int64 * 7)()
    lib.last_combine(v)
    return dict(zip(("y", "z", "w", "tokens", "top_k", "rows", "columns"), v))


@pytest.mark.parametrize("tokens,top_k,rows,width", [(5, 2, 10, 48), (5, 2, 0, 48), (5, 2, 10, 0), (5, 2, 0, 0),
                                                     (5, 0, 10, 48), (1, 1, 1, 1)])
def test_operands_that_may_be_left_out_are_not_read(lib, tokens, top_k, rows, width):
    """Without rows of z (or columns) dy may be NULL: the gradient's kernel,
    which still has to clear dweights, then has no columns of dy to read."""
    d = dg.make_combine_desc(tokens, top_k, rows, width)
    need = top_k > 0 and rows > 0 and width > 0
    for dz, dw in ((P5, P6), (None, P6), (P5, None)):
        st = lib.dg_combine_grad(d, None, P2, P3, P4, dz, dw, None)
        if need:
            assert st == dg.DG_ERROR_INVALID_VALUE
            assert lib.dg_combine_grad(d, P1, P2, P3, P4, dz, dw, None) == dg.DG_SUCCESS
            assert _last(lib) == dict(y=P1, z=P2, w=P4, tokens=tokens, top_k=top_k, rows=rows, columns=width)
        else:
            assert st == dg.DG_SUCCESS
            if top_k:
                assert _last(lib)["columns"] == 0 and _last(lib)["top_k"] == top_k
    if width:
        st = lib.dg_combine(d, None, None, None, P4, None)
        if need:
            assert st == dg.DG_ERROR_INVALID_VALUE
        else:
            assert st == dg.DG_SUCCESS and _last(lib)["top_k"] == 0 and _last(lib)["columns"] == width


@pytest.mark.gpu
def test_gradient_without_rows_clears_the_weights():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    for tokens, top_k, width in ((7, 2, 48), (300, 9, 4000)):
        place = torch.zeros(tokens, top_k, dtype=torch.int32, device="cuda")
        w, dw = torch.ones(tokens, top_k, device="cuda"), torch.full((tokens, top_k), 5.0, device="cuda")
        d = dg.make_combine_desc(tokens, top_k, 0, width)
        dg.dg_combine_grad(d, None, None, place.data_ptr(), w.data_ptr(), None, dw.data_ptr(),
                           torch.cuda.current_stream().cuda_stream)
        assert bool((dw == 0).all())
