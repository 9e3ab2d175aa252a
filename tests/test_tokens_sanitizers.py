"""AddressSanitizer and UndefinedBehaviorSanitizer over the host code of the
routed tokens and the 8-bit products (built host-only): validation, kernel
choice and description on valid, extreme and invalid descriptors.  Any report
aborts the child, and its answers must equal those of the normal build."""
import os
import subprocess
import tempfile

import pytest

from conftest import ROOT
from test_sanitizers import (CLANGXX, CSRC, HIPCC, INCLUDE, SAN_ENV, _clang_asan_runtime, _run_battery)

# a null pointer among the operands keeps every call from a launch
BATTERY = r'''
import itertools, json, sys
sys.path.insert(0, ROOT)
import dense_gemm_10_amd as dg
out = []
A, B, C, S, Z, O = (i << 56 for i in range(1, 7))
BIG = 2 ** 62
sizes = (-1, 0, 1, 7, 300, 2 ** 31 - 1, 2 ** 40, BIG)
for tokens, k, groups, width in itertools.product(sizes, (-1, 0, 1, 8, 2 ** 31), (0, 1, 8192, 2 ** 40), (0, 1, 4097, BIG)):
    d = dg.make_dispatch_desc(tokens, k, groups, width, rows=min(max(tokens, 0), 2 ** 31 - 1), index_bits=64)
    out.append(dg.dg_dispatch(d, A, B, None, S, Z, O, check=False))
    if tokens > 0 and k > 0 and width > 0:
        out.append(dg.dg_spread(d, None, B, C, check=False))
for tokens, k, rows, width in itertools.product(sizes, (-1, 0, 1, 2 ** 31), sizes, (0, 1, 4097, BIG)):
    d = dg.make_combine_desc(tokens, k, rows, width)
    out.append(dg.dg_combine(d, A, B, C, None, check=False))
    if rows > 0 and width > 0:
        out.append(dg.dg_combine_grad(d, None, B, C, S, Z, O, check=False))
    q = dg.make_quantize_desc(tokens, width, top_k=k, rows=rows)
    out.append(dg.dg_quantize(q, A, B, C, None, check=False))
def rec(f, d):
    try:
        out.append(f(d))
    except dg.DgError as e:
        out.append(e.status)
for groups, M, N, K in itertools.product((0, 1, 2, 65536, 2 ** 40), sizes, (0, 1, 4097, BIG), (0, 1, 4096, 131071, BIG)):
    for dt in ("i8", "bf16", "f32"):
        d = dg.make_scaled_desc(M, N, K, groups=groups, a_type=dt, stride_b=min(N * K, BIG), stride_s=min(N, BIG))
        rec(dg.dg_gemm_scaled_describe, d)
        rec(dg.dg_gemm_scaled_workspace_size, d)
        out.append(dg.dg_gemm_scaled(d, A, None, B, S, None, O, Z, 2 ** 60, check=False))
print(json.dumps(out))
'''


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANGXX) and _clang_asan_runtime()),
                    reason="no hipcc / clang ASan runtime")
def test_tokens_and_8_bit_host_code_under_asan_and_ubsan():
    tests = os.path.join(ROOT, "tests")
    sources = [os.path.join(CSRC, f) for f in ("tokens_api.cpp", "scaled_api.cpp", "api.cpp", "kernel_generic.hip",
                                               "kernel_valu_f32.hip", "kernel_mfma16.hip", "kernel_sliver.hip",
                                               "tiles_f32.cpp")]
    sources += [os.path.join(tests, f) for f in ("sanitizer_stubs.hip", "tokens_stubs.hip")]
    with tempfile.TemporaryDirectory() as d:
        objs, procs = [], []
        for src in sources:
            obj = os.path.join(d, os.path.basename(src) + ".o")
            cmd = [HIPCC, "-x", "hip", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
                   "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                   "-Xarch_host", "-fno-sanitize-recover=all", "-I", INCLUDE, "-I", CSRC, "-c", src,
                   "-o", obj]
            procs.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE))
            objs.append(obj)
        for pr in procs:
            _, err = pr.communicate(timeout=600)
            assert pr.returncode == 0, err.decode()[-3000:]
        lib = os.path.join(d, "libdensegemm_san.so")
        subprocess.run([CLANGXX, "-shared", "-fPIC", "-shared-libasan", "-fsanitize=address,undefined",
                        "-o", lib] + objs + ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"],
                       check=True, capture_output=True)
        san = _run_battery(BATTERY, dict(SAN_ENV, DG_LIBRARY=lib, LD_PRELOAD=_clang_asan_runtime()))
    plain = _run_battery(BATTERY, {"DG_LIBRARY": os.path.join(ROOT, "dense_gemm_10_amd",
                                                               "libdensegemm.so")})
    assert san == plain
