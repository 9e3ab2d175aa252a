"""dg_gemm_grouped and dg_gemm_qweight on the host: the Python structs mirror
the header, every invalid descriptor or pointer is refused before anything is
enqueued, shapes without work succeed, plans follow the stated rules."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

import dense_gemm_10_amd as dg
from conftest import ROOT

HEADER = os.path.join(ROOT, "include", "densegemm.h")
PA, PB, PC, PS, PZ, PO = (i << 56 for i in range(1, 7))      # never dereferenced


@pytest.mark.parametrize("cls,name", [(dg.DgGroupedDesc, "dg_grouped_desc"),
                                      (dg.DgQweightDesc, "dg_qweight_desc")])
def test_struct_layout_matches_header(cls, name):
    fields = [f for f, _ in cls._fields_]
    src = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{HEADER}"', "int main(void) {",
           f'printf("%zu\\n", sizeof({name}));']
    src += [f'printf("%zu\\n", offsetof({name}, {f}));' for f in fields] + ["return 0; }"]
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "layout.c"), os.path.join(d, "layout")
        open(c, "w").write("\n".join(src))
        subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", c, "-o", exe], check=True)
        vals = [int(v) for v in subprocess.run([exe], capture_output=True, text=True,
                                               check=True).stdout.split()]
    assert vals[0] == ctypes.sizeof(cls)
    assert [getattr(cls, f).offset for f in fields] == vals[1:]


def _grouped(ragged="m", **kw):
    base = dict(ragged=ragged, groups=4, rows=100, N=48, a_type="bf16")
    base.update(dict(M=40) if ragged == "k" else dict(K=32))
    base.update(kw)
    return dg.make_grouped_desc(**base)


def _run(d, A=PA, B=PB, C=PC, off=PO):
    return dg.dg_gemm_grouped(d, A, B, C, off, check=False)


INVALID = [
    ("m", dict(ragged=2)), ("m", dict(groups=-1)), ("m", dict(rows=-1)), ("m", dict(N=-1, ldb=1, ldc=1)),
    ("m", dict(K=-1, ldb=48)), ("k", dict(M=-1, ldb=48)), ("m", dict(a_type=5)), ("m", dict(c_type=3)),
    ("m", dict(b_order=2)), ("m", dict(act=3)), ("m", dict(lda=31)), ("m", dict(ldb=47)),
    ("m", dict(b_order="col", ldb=31)), ("m", dict(ldc=47)), ("m", dict(lda=0)), ("k", dict(lda=39)),
    ("k", dict(ldb=47)), ("k", dict(ldc=47)), ("m", dict(stride_b=-1)), ("k", dict(stride_c=-1)),
    ("k", dict(stride_c=40 * 48 - 1)), ("k", dict(stride_c=0)), ("m", dict(bias=PS, bias_type=7)),
    ("m", dict(bias=PS, stride_bias=-1)),
    ("m", dict(K=2 ** 40, lda=2 ** 40, ldb=2 ** 40, stride_b=2 ** 62)),
]


@pytest.mark.parametrize("ragged,kw", INVALID, ids=[f"{r}-{k}" for r, k in INVALID])
def test_invalid_grouped_descriptors(ragged, kw):
    d = _grouped(**{"ragged": ragged, **kw})
    assert _run(d) == dg.DG_ERROR_INVALID_VALUE
    with pytest.raises(dg.DgError) as e:
        dg.dg_gemm_grouped_describe(d)
    assert e.value.status == dg.DG_ERROR_INVALID_VALUE


@pytest.mark.parametrize("ragged,kw", [
    ("m", dict(a_type="bf16", b_type="f16")), ("m", dict(a_type="f32", c_type="bf16")),
    ("m", dict(groups=65537)), ("m", dict(rows=2 ** 31)), ("k", dict(b_order="col", ldb=100)),
    ("k", dict(bias=PS)), ("k", dict(act="gelu_erf")), ("m", dict(rows=2 ** 31 - 1, N=2 ** 20)),
])
def test_unsupported_grouped_descriptors(ragged, kw):
    assert _run(_grouped(ragged, **kw)) == dg.DG_ERROR_NOT_SUPPORTED


def test_grouped_pointers():
    d = _grouped()
    bad = dg.DG_ERROR_INVALID_VALUE
    assert _run(d, A=None) == bad and _run(d, B=None) == bad and _run(d, C=None) == bad
    assert _run(d, off=None) == bad
    assert _run(d, off=PO + 2) == bad and _run(d, A=PA + 1) == bad and _run(d, C=PC + 1) == bad
    assert _run(d, C=PA + 64) == bad and _run(d, C=PB - 8) == bad and _run(d, off=PC + 8) == bad
    assert _run(_grouped(bias=PC + 16)) == bad and _run(_grouped(bias=PS + 2)) == bad
    d.struct_size = 8
    assert _run(d) == bad


def test_shapes_without_work():
    for d in (_grouped(groups=0), _grouped(rows=0), _grouped(N=0), _grouped("k", M=0),
              _grouped("k", N=0), _grouped("k", groups=0)):
        assert _run(d, None, None, None, None) == dg.DG_SUCCESS
        assert dg.dg_gemm_grouped_describe(d) == "noop"
    for kw in (dict(M=0), dict(N=0), dict(groups=0)):
        d = _qweight(**kw)
        assert _qrun(d, None, None, None, None, None) == dg.DG_SUCCESS
        assert dg.dg_gemm_qweight_describe(d) == "noop"


def _qweight(**kw):
    base = dict(M=5, N=48, K=256, group_size=64, a_type="bf16")
    base.update(kw)
    return dg.make_qweight_desc(**base)


def _qrun(d, A=PA, Q=PB, S=PS, Z=PZ, C=PC, off=None):
    return dg.dg_gemm_qweight(d, A, Q, S, Z, C, off, check=False)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(N=-1, ldc=1), dict(K=-1), dict(groups=-1), dict(a_type=4), dict(c_type=4),
    dict(scale_type=-1), dict(act=3), dict(lda=255), dict(ldc=47), dict(ldq=127), dict(lds=3),
    dict(stride_q=-1), dict(stride_s=-1), dict(bias=PO, bias_type=3), dict(bias=PO, stride_bias=-1),
    dict(groups=2), dict(N=2 ** 40, ldq=2 ** 40),
], ids=str)
def test_invalid_qweight_descriptors(kw):
    assert _qrun(_qweight(**kw)) == dg.DG_ERROR_INVALID_VALUE      # groups = 2 lacks offsets


@pytest.mark.parametrize("kw", [dict(a_type="f32"), dict(group_size=48), dict(group_size=16),
                                dict(groups=65537), dict(M=2 ** 31)], ids=str)
def test_unsupported_qweight_descriptors(kw):
    assert _qrun(_qweight(**kw), off=PO) == dg.DG_ERROR_NOT_SUPPORTED
    with pytest.raises(dg.DgError) as e:
        dg.dg_gemm_qweight_describe(_qweight(**kw))
    assert e.value.status == dg.DG_ERROR_NOT_SUPPORTED


def test_qweight_pointers():
    d, bad = _qweight(), dg.DG_ERROR_INVALID_VALUE
    for kw in (dict(A=None), dict(Q=None), dict(S=None), dict(C=None), dict(A=PA + 1), dict(S=PS + 1),
               dict(C=PC + 1), dict(off=PO + 2), dict(C=PA), dict(C=PB), dict(C=PS), dict(C=PZ),
               dict(off=PC)):
        assert _qrun(d, **kw) == bad, kw
    assert _qrun(_qweight(bias=PC)) == bad
    d = _qweight()
    d.struct_size = 8
    assert _qrun(d) == bad


# ---- the kernel a problem gets ------------------------------------------------------
def _kernel(text):
    return dict(t.split("=") for t in text.split())["kernel"]


@pytest.mark.parametrize("kw,kernel", [
    (dict(groups=8, rows=8, K=1024, N=1024), "stream_16x32"),
    (dict(groups=64, rows=64, K=2048, N=1024), "stream_16x64"),
    (dict(groups=64, rows=1024, K=2048, N=2048), "stream_32x64"),
    (dict(groups=20, rows=1000, K=1024, N=4096), "mfma16_128x128"),
    (dict(groups=7, rows=4095, K=1000, N=4097, b_order="col"), "mfma16_256x256"),
    (dict(groups=4, rows=1000, K=4096, N=1024), "mfma16_128x128"),
    (dict(groups=16, rows=8192, K=4096, N=4096), "mfma16_256x256"),
    (dict(groups=5, rows=1000, K=512, N=260, a_type="f32"), "stream_32x64"),
    (dict(groups=16, rows=8192, K=2048, N=4096, a_type="f32"), "mfma_f32_128x128"),
    (dict(groups=4, rows=100, K=33, N=64), "generic"),              # lda off the 16-byte grid
    (dict(groups=4, rows=100, K=64, N=33), "generic"),              # ldb
    (dict(groups=4, rows=100, K=64, N=33, b_order="col"), "mfma16_128x128"),
    (dict(groups=4, rows=100, K=64, N=64, stride_b=4100), "generic"),
    (dict(groups=1, rows=100, K=64, N=64, stride_b=4100), "mfma16_128x128"),
    (dict(ragged="k", groups=16, rows=8192, M=2048, N=2048), "mfma16_128x128"),
    (dict(ragged="k", groups=8, rows=8192, M=1024, N=2048), "mfma16_128x128"),
    (dict(ragged="k", groups=8, rows=16384, M=2048, N=2048), "mfma16_256x256"),
    (dict(ragged="k", groups=1, rows=4096, M=4096, N=4096), "mfma16_256x256"),
    (dict(ragged="k", groups=8, rows=8192, M=1024, N=2048, a_type="f32"), "mfma_f32_128x128"),
    (dict(ragged="k", groups=8, rows=8192, M=1001, N=2048), "generic"),
], ids=str)
def test_kernel_of_a_grouped_problem(kw, kernel, monkeypatch):
    monkeypatch.delenv("DG_FORCE_GROUPED", raising=False)
    kw = dict({"ragged": "m"}, **kw)
    assert _kernel(dg.dg_gemm_grouped_describe(dg.make_grouped_desc(**kw))) == kernel
    # a forced kernel never replaces the generic one, whose operands no other takes
    monkeypatch.setenv("DG_FORCE_GROUPED", "mfma16_256x256")
    forced = _kernel(dg.dg_gemm_grouped_describe(dg.make_grouped_desc(**kw)))
    assert forced == ("generic" if kernel == "generic" else kernel if kw.get("a_type") == "f32"
                      else "mfma16_256x256")


@pytest.mark.parametrize("M,N,K,g,kw,kernel", [
    (1, 4096, 4096, 128, {}, "qstream_16x16"), (1, 16384, 8192, 64, {}, "qstream_16x32"),
    (16, 16384, 4096, 128, {}, "qstream_16x64"), (64, 4096, 4096, 128, {}, "qstream_32x32"),
    (128, 4096, 4096, 128, {}, "qstream_32x64"), (512, 4096, 4096, 128, {}, "qstream_32x128"),
    (2048, 4096, 4096, 128, {}, "qtile_64x512"), (1024, 4096, 4096, 128, {}, "qtile_64x256"),
    (2048, 4096, 4096, 64, {}, "qtile_64x256"), (5, 64, 4112, 128, {}, "generic"),
    (5, 64, 128, 32, dict(ldq=72), "generic"), (5, 64, 128, 32, dict(lda=132), "generic"),
    (64, 2048, 2048, 128, dict(groups=64), "qstream_16x64"),
    (64, 2048, 2048, 128, dict(groups=64, stride_q=2048 * 1024 + 8), "generic"),
    (1, 64, 2 ** 20, 32, dict(ldq=2 ** 23), "generic"),
], ids=str)
def test_kernel_of_a_4_bit_problem(M, N, K, g, kw, kernel, monkeypatch):
    monkeypatch.delenv("DG_FORCE_GROUPED", raising=False)
    assert _kernel(dg.dg_gemm_qweight_describe(dg.make_qweight_desc(M, N, K, g, **kw))) == kernel


# ---- the torch entry points refuse before any GPU call ---------------------------
def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


OFF5 = torch.zeros(5, dtype=torch.int32)


@pytest.mark.parametrize("what,call,match", [
    ("B is 2-D", lambda: dg.gemm_grouped(_t(8, 4), _t(4, 6), OFF5), "wanted"),
    ("inner sizes", lambda: dg.gemm_grouped(_t(8, 4), _t(4, 5, 6), OFF5), "wanted"),
    ("int64 offsets", lambda: dg.gemm_grouped(_t(8, 4), _t(4, 4, 6), OFF5.long()), "offsets"),
    ("too few offsets", lambda: dg.gemm_grouped(_t(8, 4), _t(4, 4, 6), OFF5[:4]), "offsets"),
    ("strided offsets", lambda: dg.gemm_grouped(_t(8, 4), _t(4, 4, 6),
                                                torch.zeros(10, dtype=torch.int32)[::2]), "offsets"),
    ("beta without C", lambda: dg.gemm_grouped(_t(8, 4), _t(4, 4, 6), OFF5, beta=1.0), "beta"),
    ("C's shape", lambda: dg.gemm_grouped(_t(8, 4), _t(4, 4, 6), OFF5, _t(7, 6)), "C"),
    ("C's type", lambda: dg.gemm_grouped(_t(8, 4), _t(4, 4, 6), OFF5, _t(8, 6),
                                         out_dtype=torch.float32), "out_dtype"),
    ("on the CPU", lambda: dg.gemm_grouped(_t(8, 4), _t(4, 4, 6), OFF5), "GPU"),
    ("A of K rows", lambda: dg.gemm_grouped_k(_t(4, 8), _t(7, 6), OFF5), "wanted"),
    ("K: beta without C", lambda: dg.gemm_grouped_k(_t(4, 8), _t(8, 6), OFF5, beta=2.0), "beta"),
    ("K: 2-D offsets", lambda: dg.gemm_grouped_k(_t(4, 8), _t(8, 6), OFF5[None]), "offsets"),
    ("Q's type", lambda: dg.gemm_qweight(_t(2, 64), _t(6, 32), _t(6, 2), group_size=32), "uint8"),
    ("Q's width", lambda: dg.gemm_qweight(_t(2, 64), _t(6, 64, dtype=torch.uint8), _t(6, 2),
                                          group_size=32), "uint8"),
    ("scales' shape", lambda: dg.gemm_qweight(_t(2, 64), _t(6, 32, dtype=torch.uint8), _t(6, 1),
                                              group_size=32), "scales"),
    ("zeros' type", lambda: dg.gemm_qweight(_t(2, 64), _t(6, 32, dtype=torch.uint8), _t(6, 2), _t(6, 2),
                                            group_size=32), "zeros"),
    ("zeros' strides", lambda: dg.gemm_qweight(
        _t(2, 64), _t(6, 32, dtype=torch.uint8), _t(6, 2), _t(2, 6, dtype=torch.uint8).t(),
        group_size=32), "zeros"),
    ("experts without offsets", lambda: dg.gemm_qweight(
        _t(2, 64), _t(4, 6, 32, dtype=torch.uint8), _t(4, 6, 2), group_size=32), "wanted"),
], ids=lambda v: v if isinstance(v, str) else "")
def test_torch_entry_points_refuse(what, call, match):
    with pytest.raises(ValueError, match=match):
        call()


def test_packed_descriptors_match_the_structures():
    """The torch entry points pack the descriptors' bytes directly."""
    from dense_gemm_10_amd import grouped as G
    ints = list(range(1, 19))
    for cls, pack, size in ((G.DgGroupedDesc, G._pack_grouped, G._GROUPED_SIZE),
                            (G.DgQweightDesc, G._pack_qweight, G._QWEIGHT_SIZE)):
        n = len(cls._fields_) - 4
        values = [size, *ints[:n], 1.5, -0.25, 0x1234567890]
        assert pack(*values) == bytes(cls(*values))
