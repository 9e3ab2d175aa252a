"""dg_dispatch, dg_spread, dg_combine, dg_combine_grad and dg_quantize on the
host: the structs mirror the header, every invalid descriptor or pointer is
refused before anything is enqueued, shapes without work succeed, the torch
entry points refuse before any GPU call."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

import dense_gemm_10_amd as dg
from conftest import ROOT
from dense_gemm_10_amd import tokens as T

HEADER = os.path.join(ROOT, "include", "densegemm.h")
P1, P2, P3, P4, P5, P6 = (i << 56 for i in range(1, 7))      # never dereferenced
BAD, NO, OK = dg.DG_ERROR_INVALID_VALUE, dg.DG_ERROR_NOT_SUPPORTED, dg.DG_SUCCESS


@pytest.mark.parametrize("cls,name", [(dg.DgDispatchDesc, "dg_dispatch_desc"),
                                      (dg.DgCombineDesc, "dg_combine_desc"),
                                      (dg.DgQuantizeDesc, "dg_quantize_desc")])
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


def test_packed_descriptors_match_the_structures():
    for cls, pack, size, tail in ((T.DgDispatchDesc, T._pack_dispatch, T._DISPATCH_SIZE, ()),
                                  (T.DgCombineDesc, T._pack_combine, T._COMBINE_SIZE, (1.5,)),
                                  (T.DgQuantizeDesc, T._pack_quantize, T._QUANTIZE_SIZE, ())):
        values = [size, *range(1, len(cls._fields_) - len(tail)), *tail]
        assert pack(*values) == bytes(cls(*values))


def _dispatch(d, index=P1, x=P2, offsets=P3, order=P4, place=P5, rows=P6):
    return dg.dg_dispatch(d, index, x, offsets, order, place, rows, check=False)


def _dd(**kw):
    return dg.make_dispatch_desc(**dict(dict(tokens=5, top_k=2, groups=4, width=48), **kw))


def _spread(d, place=P1, x=P2, rows=P3):
    return dg.dg_spread(d, place, x, rows, check=False)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), BAD), (dict(top_k=-1), BAD), (dict(groups=-1), BAD), (dict(width=-1), BAD),
    (dict(x_type=3), BAD), (dict(index_bits=16), BAD), (dict(ld_index=1), BAD), (dict(ldx=47), BAD),
    (dict(ldr=47), BAD), (dict(ld_index=0, top_k=0), BAD), (dict(groups=8193), NO),
    (dict(tokens=2 ** 30, top_k=2), NO), (dict(tokens=2 ** 62, top_k=4), NO),
    (dict(tokens=0, top_k=2 ** 31), NO), (dict(width=2 ** 60, ldx=2 ** 60, ldr=2 ** 60), BAD),
], ids=str)
def test_invalid_dispatch_descriptors(kw, want):
    assert _dispatch(_dd(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), BAD), (dict(rows=-1), BAD), (dict(width=-1), BAD), (dict(x_type=-1), BAD),
    (dict(ldx=47), BAD), (dict(ldr=47), BAD), (dict(rows=2 ** 31), NO), (dict(tokens=2 ** 30, rows=4), NO),
], ids=str)
def test_invalid_spread_descriptors(kw, want):
    assert _spread(_dd(**kw)) == want


def test_dispatch_pointers():
    d = _dd()
    for kw in (dict(index=None), dict(offsets=None), dict(order=None), dict(place=None), dict(x=None),
               dict(rows=None), dict(index=P1 + 2), dict(x=P2 + 1), dict(rows=P6 + 1), dict(offsets=P3 + 2),
               dict(order=P4 + 1), dict(place=P5 + 3), dict(order=P5), dict(offsets=P1 + 8), dict(rows=P2),
               dict(rows=P5 - 16), dict(place=P1 - 4)):
        assert _dispatch(d, **kw) == BAD, kw
    assert _dispatch(_dd(index_bits=64), index=P1 + 4) == BAD
    d.struct_size = 8
    assert _dispatch(d) == BAD and _spread(d) == BAD
    d = _dd()
    for kw in (dict(place=None), dict(x=None), dict(rows=None), dict(place=P1 + 2), dict(x=P2 + 1),
               dict(rows=P2 + 32), dict(rows=P1)):
        assert _spread(d, **kw) == BAD, kw
    for kw in (dict(tokens=0), dict(top_k=0), dict(rows=0), dict(width=0)):
        assert _spread(_dd(**kw), None, None, None) == OK


def _cd(**kw):
    return dg.make_combine_desc(**dict(dict(tokens=5, top_k=2, rows=10, width=48), **kw))


def _combine(d, z=P1, place=P2, w=P3, y=P4):
    return dg.dg_combine(d, z, place, w, y, check=False)


def _grad(d, dy=P1, z=P2, place=P3, w=P4, dz=P5, dw=P6):
    return dg.dg_combine_grad(d, dy, z, place, w, dz, dw, check=False)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), BAD), (dict(top_k=-1), BAD), (dict(rows=-1), BAD), (dict(width=-1), BAD),
    (dict(z_type=3), BAD), (dict(y_type=-1), BAD), (dict(w_type=5), BAD), (dict(ldz=47), BAD),
    (dict(ldy=47), BAD), (dict(ldw=1), BAD), (dict(y_type="f16"), NO), (dict(z_type="f32", y_type="bf16"), NO),
    (dict(rows=2 ** 31), NO), (dict(tokens=2 ** 30), NO), (dict(width=2 ** 60, ldz=2 ** 60), BAD),
], ids=str)
def test_invalid_combine_descriptors(kw, want):
    assert _combine(_cd(**kw)) == want
    assert _grad(_cd(**kw)) == want


def test_combine_pointers():
    d = _cd()
    for kw in (dict(z=None), dict(place=None), dict(y=None), dict(z=P1 + 1), dict(place=P2 + 2),
               dict(w=P3 + 2), dict(y=P4 + 1), dict(y=P1 + 64), dict(y=P2), dict(y=P3 + 4)):
        assert _combine(d, **kw) == BAD, kw
    for kw in (dict(dy=None), dict(z=None), dict(place=None), dict(dy=P1 + 1), dict(z=P2 + 1),
               dict(place=P3 + 1), dict(w=P4 + 2), dict(dz=P5 + 1), dict(dw=P6 + 2), dict(dz=P1), dict(dz=P2),
               dict(dw=P3), dict(dw=P4), dict(dw=P5)):
        assert _grad(d, **kw) == BAD, kw
    assert _grad(_cd(lddz=47)) == BAD
    d.struct_size = 8
    assert _combine(d) == BAD and _grad(d) == BAD
    for kw in (dict(tokens=0), dict(width=0)):
        assert _combine(_cd(**kw), None, None, None, None) == OK
    assert _grad(_cd(tokens=0), None, None, None, None) == OK
    assert _grad(_cd(), dz=None, dw=None) == OK


def _quantize(d, x=P1, place=P2, q=P3, scales=P4):
    return dg.dg_quantize(d, x, place, q, scales, check=False)


def _qd(**kw):
    return dg.make_quantize_desc(**dict(dict(tokens=5, width=48), **kw))


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), BAD), (dict(width=-1), BAD), (dict(x_type=3), BAD), (dict(ldx=47), BAD), (dict(ldq=47), BAD),
    (dict(top_k=-1), BAD), (dict(rows=-1), BAD), (dict(rows=2 ** 31), NO), (dict(tokens=2 ** 30, top_k=2, rows=5), NO),
    (dict(width=2 ** 61, ldx=2 ** 62), BAD),
], ids=str)
def test_invalid_quantize_descriptors(kw, want):
    assert _quantize(_qd(**kw)) == want


def test_quantize_pointers():
    d = _qd()
    for kw in (dict(x=None), dict(q=None), dict(scales=None), dict(x=P1 + 1), dict(place=P2 + 2),
               dict(scales=P4 + 2), dict(q=P1 + 9), dict(scales=P1), dict(scales=P3), dict(q=P2)):
        assert _quantize(d, **kw) == BAD, kw
    d.struct_size = 8
    assert _quantize(d) == BAD
    for kw in (dict(tokens=0), dict(rows=0)):
        assert _quantize(_qd(**kw), None, P2, None, None) == OK
    assert _quantize(_qd(tokens=0), None, None, None, None) == OK


# ---- the torch entry points ------------------------------------------------------
def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


IDX, PLACE = _t(4, 2, dtype=torch.int64), _t(4, 2, dtype=torch.int32)


@pytest.mark.parametrize("what,call,match", [
    ("index of floats", lambda: dg.sort_tokens(_t(4, 2), 3), "index"),
    ("1-D index", lambda: dg.sort_tokens(IDX[:, 0], 3), "index"),
    ("index by columns", lambda: dg.sort_tokens(_t(2, 4, dtype=torch.int64).t(), 3), "row-major"),
    ("negative groups", lambda: dg.sort_tokens(IDX, -1), "groups"),
    ("on the CPU", lambda: dg.sort_tokens(IDX, 3), "GPU"),
    ("x and index", lambda: dg.dispatch_tokens(_t(5, 8), IDX, 3), "rows"),
    ("x by columns", lambda: dg.dispatch_tokens(_t(8, 4).t(), IDX, 3), "row-major"),
    ("out's shape", lambda: dg.dispatch_tokens(_t(4, 8), IDX, 3, out=_t(7, 8)), "out"),
    ("out's type", lambda: dg.dispatch_tokens(_t(4, 8), IDX, 3, out=_t(8, 8, dtype=torch.float32)), "out"),
    ("dispatch on the CPU", lambda: dg.dispatch_tokens(_t(4, 8), IDX, 3), "GPU"),
    ("place of int64", lambda: dg.spread_tokens(_t(4, 8), IDX), "place"),
    ("place strided", lambda: dg.spread_tokens(_t(4, 8), _t(4, 4, dtype=torch.int32)[:, :2]), "place"),
    ("x and place", lambda: dg.spread_tokens(_t(3, 8), PLACE), "rows"),
    ("spread width", lambda: dg.spread_tokens(_t(4, 8), PLACE, out=_t(8, 7)), "out"),
    ("1-D z", lambda: dg.combine_tokens(_t(8), PLACE), "dimensions"),
    ("weights' shape", lambda: dg.combine_tokens(_t(8, 4), PLACE, _t(4, 3)), None),
    ("y's shape", lambda: dg.combine_tokens(_t(8, 4), PLACE, None, _t(4, 5)), "y"),
    ("beta without y", lambda: dg.combine_tokens(_t(8, 4), PLACE, beta=1.0), "beta"),
    ("y and out_dtype", lambda: dg.combine_tokens(_t(8, 4), PLACE, None, _t(4, 4), out_dtype=torch.float32), "y"),
    ("combine on the CPU", lambda: dg.combine_tokens(_t(8, 4), PLACE), "GPU"),
    ("dy's rows", lambda: dg.combine_tokens_grad(_t(5, 4), _t(8, 4), PLACE, _t(4, 2)), "match"),
    ("z's width", lambda: dg.combine_tokens_grad(_t(4, 4), _t(8, 5), PLACE, _t(4, 2)), "match"),
    ("no weights", lambda: dg.combine_tokens_grad(_t(4, 4), _t(8, 4), PLACE, None), "weights"),
    ("weights' width", lambda: dg.combine_tokens_grad(_t(4, 4), _t(8, 4), PLACE, _t(4, 3)), "weights"),
    ("dz's type", lambda: dg.combine_tokens_grad(_t(4, 4), _t(8, 4), PLACE, _t(4, 2),
                                                 dz=_t(8, 4, dtype=torch.float16)), "dz"),
    ("q's type", lambda: dg.quantize_rows(_t(4, 4), None, _t(4, 4)), "q"),
    ("q's rows", lambda: dg.quantize_rows(_t(4, 4), None, _t(5, 4, dtype=torch.int8)), "q"),
    ("scales' type", lambda: dg.quantize_rows(_t(4, 4), None, None, _t(4)), "scales"),
    ("scales strided", lambda: dg.quantize_rows(_t(4, 4), None, None, _t(8, dtype=torch.float32)[::2]), "scales"),
    ("quantize place", lambda: dg.quantize_rows(_t(5, 4), PLACE), "rows"),
    ("quantize on the CPU", lambda: dg.quantize_rows(_t(4, 4)), "GPU"),
], ids=lambda v: v if isinstance(v, str) else "")
def test_torch_entry_points_refuse(what, call, match):
    with pytest.raises(ValueError, match=match):
        call()


def test_types_that_are_refused():
    for call in (lambda: dg.combine_tokens(_t(8, 4, dtype=torch.float64), PLACE),
                 lambda: dg.dispatch_tokens(_t(4, 8, dtype=torch.int32), IDX, 3)):
        with pytest.raises((TypeError, ValueError)):
            call()
