"""Streaming kernels of the 8-bit products on long K: many steps in a wavefront's
ring, workgroups that begin at different steps, a last part of a step; against
the definition, with sums that no other order of k would repeat by chance."""
import pytest
import torch

import dense_gemm_10_amd as dg
from grouped_util import DT, check, finish, groups_of
from tokens_util import codes64

pytestmark = pytest.mark.gpu

KERNELS = ["i8_stream_16x16", "i8_stream_16x32", "i8_stream_16x32_short", "i8_stream_16x64", "i8_stream_32x32"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _i8(gen, *shape, pad=0):
    t = torch.randint(-128, 128, shape[:-1] + (shape[-1] + pad,), device="cuda", generator=gen, dtype=torch.int8)
    return t[..., :shape[-1]]


# 16 steps of 128 (a loop only with four wavefronts), 17, 32 and a part, 35 and
# a part, 64 and two bytes (rows at odd addresses), 127 and a part
@pytest.mark.parametrize("K,pad", [(2048, 0), (2176, 16), (4112, 0), (4496, 0), (8194, 1), (16383, 0)])
@pytest.mark.parametrize("kernel", KERNELS)
def test_long_sums_are_exact(kernel, K, pad, monkeypatch):
    """Rounded once, from the exact sum to fp32."""
    monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    gen = torch.Generator(device="cuda").manual_seed(K)
    for M, N in ((1, 1000), (13, 330), (40, 203)):
        assert f"kernel={kernel} " in dg.dg_gemm_scaled_describe(dg.make_scaled_desc(M, N, K))
        A, B = _i8(gen, M, K, pad=pad), _i8(gen, N, K, pad=pad)
        want = (A.double() @ B.double().t()).float()
        assert torch.equal(dg.gemm_scaled(A, B, out_dtype=torch.float32), want), (M, N)
    M, N, groups = 50, 203, 5
    A, B = _i8(gen, M, K, pad=pad), _i8(gen, groups, N, K, pad=pad)
    off = [3, 20, 20, 21, 44, 48]
    C = torch.full((M, N), 7.0, device="cuda")
    dg.gemm_scaled(A, B, None, None, C, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
    want = torch.full((M, N), 7.0, device="cuda")
    for e, (lo, hi) in enumerate(groups_of(off, M)):
        want[lo:hi] = (A[lo:hi].double() @ B[e].double().t()).float()
    assert torch.equal(C, want)


@pytest.mark.parametrize("kernel", ["i8_stream_16x16", "i8_stream_16x32", "i8_stream_16x64"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_few_float_rows_against_the_definition(dtype, kernel, monkeypatch):
    """Codes made inside the product.  Tolerance: codes and scales are the
    definition's; conversion and two scales are three roundings of fp32,
    3.01 * 2^-24 of the value; the rest as in grouped_util."""
    monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    gen = torch.Generator(device="cuda").manual_seed(2)
    for M, K, pad in ((1, 8192, 0), (1, 8100, 1), (2, 4096, 0), (3, 2600, 3), (4, 2048, 0)):
        N = 330
        x = torch.randn(M, K + pad, device="cuda", generator=gen).to(DT[dtype])[:, :K]
        B, sb = _i8(gen, N, K, pad=pad), torch.rand(N, device="cuda", generator=gen) / 1000
        desc = dg.make_scaled_desc(M, N, K, a_type=dtype)
        assert dg.dg_gemm_scaled_workspace_size(desc) == 0 and f"kernel={kernel} " in dg.dg_gemm_scaled_describe(desc)
        codes, scales = codes64(x.cpu())
        y = codes.double() @ B.cpu().double().t() * scales[:, None].double() * sb.cpu().double()
        for out in ("f32", dtype):
            ref, tol = finish(y, None, 3.01 * 2.0 ** -24 * y.abs(), DT[out])
            check(dg.gemm_scaled(x, B, None, sb, out_dtype=DT[out]).cpu(), ref, tol, f"{M} {K} {out}")
