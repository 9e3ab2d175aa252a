"""Plans of the grouped and 4-bit-weight products at the ends of their range
(on the host): a launch that the chosen tile would make too large takes the
next larger tile."""
import pytest

import dense_gemm_10_amd as dg

LIMIT = 2 ** 32 - 1                  # threads of a launch


def _plan(text):
    p = dict(t.split("=") for t in text.split())
    return p["kernel"], int(p["programs"])


def _grouped(ragged="m", **kw):
    return _plan(dg.dg_gemm_grouped_describe(dg.make_grouped_desc(ragged, **kw)))


@pytest.fixture(autouse=True)
def _no_forced_kernel(monkeypatch):
    monkeypatch.delenv("DG_FORCE_GROUPED", raising=False)


# threads of a workgroup, as launched
THREADS = {"stream_16x32": 512, "stream_16x64": 512, "stream_32x64": 512, "mfma16_128x128": 256,
           "mfma16_256x256": 256, "mfma_f32_128x128": 256, "generic": 256}


@pytest.mark.parametrize("kw,kernel", [
    (dict(groups=16384, rows=131072, N=16384, K=512), "stream_16x64"),
    (dict(groups=65536, rows=524288, N=4096, K=512), "stream_16x64"),
    (dict(groups=64, rows=512, N=2 ** 22, K=32, b_order="col", stride_b=0), "stream_16x64"),
    (dict(groups=64, rows=512, N=2 ** 23, K=32, b_order="col", stride_b=0), "mfma16_128x128"),
    (dict(groups=62, rows=62, N=2 ** 23, K=32, b_order="col", stride_b=0), "stream_32x64"),
    (dict(groups=64, rows=512, N=2 ** 25, K=32, b_order="col", stride_b=0), "mfma16_256x256"),
    (dict(groups=16384, rows=131072, N=32768, K=512), "mfma16_128x128"),
    (dict(groups=16384, rows=131072, N=32768, K=512, a_type="f32"), "mfma_f32_128x128"),
    (dict(groups=1, rows=2 ** 31 - 1, N=256, K=512), "mfma16_256x256"),
    (dict(groups=1, rows=2 ** 31 - 1, N=128, K=512), "mfma16_256x256"),
    (dict(ragged="k", groups=65536, rows=10 ** 6, M=2048, N=2048), "mfma16_256x256"),
    (dict(ragged="k", groups=65536, rows=10 ** 6, M=1024, N=2048), "mfma16_128x128"),
], ids=str)
def test_grouped_plan_takes_a_larger_tile(kw, kernel):
    name, programs = _grouped(**kw)
    assert name == kernel
    assert 0 < programs * THREADS[name] <= LIMIT


@pytest.mark.parametrize("kw", [
    dict(groups=64, rows=2 ** 20, N=2 ** 21, K=32, b_order="col", stride_b=0),
    dict(groups=1, rows=2 ** 31 - 1, N=256, K=33),                  # the kernel for any alignment has one tile
    dict(ragged="k", groups=65536, rows=100, M=4096, N=8192),
    dict(ragged="k", groups=65536, rows=100, M=2048, N=2048, a_type="f32"),
], ids=str)
def test_grouped_launches_past_the_limit_are_refused(kw):
    with pytest.raises(dg.DgError) as e:
        _grouped(**kw)
    assert e.value.status == dg.DG_ERROR_NOT_SUPPORTED


def _qweight(M, N, K, g, **kw):
    return _plan(dg.dg_gemm_qweight_describe(dg.make_qweight_desc(M, N, K, g, **kw)))


@pytest.mark.parametrize("M,N,g,groups,kernel", [
    (16, 2 ** 28, 128, 1, "qstream_16x64"), (16, 2 ** 29 - 2 ** 14, 128, 1, "qstream_16x64"),
    (16, 2 ** 29, 128, 1, "qstream_32x128"), (16, 2 ** 30, 64, 1, "qtile_64x256"),
    (16, 2 ** 31, 128, 1, "qtile_64x512"), (64, 2 ** 32 - 2 ** 17, 128, 1, "qtile_64x512"),
    (524288, 4096, 128, 65536, "qstream_16x64"), (524288, 16384, 128, 65536, "qtile_64x256"),
    (524288, 32768, 128, 65536, "qtile_64x512"), (2 ** 21, 2 ** 15, 64, 1, "qtile_64x256"),
], ids=str)
def test_4_bit_plan_takes_a_larger_tile(M, N, g, groups, kernel):
    name, programs = _qweight(M, N, 32, g, groups=groups, ldq=16)
    assert name == kernel
    assert 0 < programs * 512 <= LIMIT


@pytest.mark.parametrize("M,N,g,groups", [(64, 2 ** 31, 64, 1), (524288, 32768, 64, 65536),
                                          (2 ** 31 - 1, 4096, 128, 1)], ids=str)
def test_4_bit_launches_past_the_limit_are_refused(M, N, g, groups):
    with pytest.raises(dg.DgError) as e:
        _qweight(M, N, 32, g, groups=groups, ldq=16)
    assert e.value.status == dg.DG_ERROR_NOT_SUPPORTED
