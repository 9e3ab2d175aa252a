"""AddressSanitizer and UndefinedBehaviorSanitizer over the host code of the
grouped and 4-bit-weight products (built host-only): validation, kernel
choice and description on valid, extreme and invalid descriptors.  Any report
aborts the child, and its answers must equal those of the normal build."""
import os
import subprocess
import tempfile

import pytest

from conftest import ROOT
from test_sanitizers import (CLANGXX, CSRC, HIPCC, INCLUDE, SAN_ENV, _clang_asan_runtime, _run_battery)

BATTERY = r'''
import itertools, json, sys
sys.path.insert(0, ROOT)
import dense_gemm_10_amd as dg
out = []
A, B, C, S, Z, O = (i << 56 for i in range(1, 7))
BIG = 2 ** 62
def rec(f, d):
    try:
        out.append(f(d))
    except dg.DgError as e:
        out.append(e.status)
sizes = (0, 1, 7, 300, 2 ** 31 - 1, 2 ** 40, BIG)
for ragged in "mk":
    for groups, rows, N, K in itertools.product((0, 1, 65536, 2 ** 40), sizes, (0, 1, 264, BIG), (0, 1, 4096, BIG)):
        for dt in ("bf16", "f32"):
            kw = dict(M=K) if ragged == "k" else dict(K=K)
            kw.update(stride_b=min(N * K, BIG), stride_c=min(N * K, BIG))
            d = dg.make_grouped_desc(ragged, groups, rows, N, a_type=dt, **kw)
            rec(dg.dg_gemm_grouped_describe, d)
            out.append(dg.dg_gemm_grouped(d, A, B, None, O, check=False))
for groups, M, N, K in itertools.product((0, 1, 65536, 2 ** 40), sizes, (0, 1, 4097, BIG), (0, 1, 4096, BIG)):
    for g in (-1, 0, 31, 32, 128, BIG):
        lds = max(1, -(-K // g)) if g > 0 else 1
        ldq = max(1, -(-K // 2))
        d = dg.make_qweight_desc(M, N, K, g, groups=groups, lds=lds, stride_q=min(N * ldq, BIG),
                                 stride_s=min(N * lds, BIG))
        rec(dg.dg_gemm_qweight_describe, d)
        out.append(dg.dg_gemm_qweight(d, A, B, S, Z, None, O, check=False))
print(json.dumps(out))
'''


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANGXX) and _clang_asan_runtime()),
                    reason="no hipcc / clang ASan runtime")
def test_grouped_host_code_under_asan_and_ubsan():
    tests = os.path.join(ROOT, "tests")
    sources = [os.path.join(CSRC, f) for f in ("grouped_api.cpp", "api.cpp", "kernel_generic.hip",
                                               "kernel_valu_f32.hip", "kernel_mfma16.hip",
                                               "kernel_sliver.hip", "tiles_f32.cpp")]
    sources += [os.path.join(tests, f) for f in ("sanitizer_stubs.hip", "grouped_stubs.hip")]
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
