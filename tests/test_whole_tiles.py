"""Products on 256 x 256 tiles that stay whole.  The tiles of a last, partly
filled pass over the chip's 256 compute units are cut into halves, so only
products of more than 128 tiles have whole ones at all; here are whole tiles
alone, whole and cut ones, and both next to a short last one, exactly, and with
every epilogue into rows of any alignment."""
import pytest
import torch

import dense_gemm_10_amd as dg
from grouped_util import DT, check, finish, groups_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _deal(lens, N):
    """(whole, cut, short) tiles of groups of these lengths."""
    columns = -(-N // 256)
    short = sum(1 for n in lens if 0 < n % 256 <= 128)
    whole = (sum(-(-n // 256) for n in lens) - short) * columns
    cut = whole % 256
    if 2 * cut + short * columns > 256:
        cut = 0
    return whole - cut, cut, short * columns


# rows of each group (one: also a matrix without offsets), N, K
SIZES = [([4096], 4096, 128), ([4196], 4396, 130), ([5170], 3328, 64), ([4096], 4096, 2050), ([2048], 4096, 256),
         ([1500, 0, 2700, 77, 900, 256], 4200, 192), ([700] * 9 + [129, 128, 1], 4096, 66)]


def test_the_sizes_have_whole_cut_and_short_tiles():
    deals = [_deal(lens, N) for lens, N, _ in SIZES]
    assert deals[0] == (256, 0, 0) and deals[1] == (256, 32, 18) and deals[2] == (256, 4, 13)
    assert deals[4] == (0, 128, 0) and all(d[0] >= 256 for i, d in enumerate(deals) if i != 4)


def _i8(gen, *shape, pad=0):
    t = torch.randint(-128, 128, shape[:-1] + (shape[-1] + pad,), device="cuda", generator=gen, dtype=torch.int8)
    return t[..., :shape[-1]]


def _offsets(lens, lead=0):
    off = [lead]
    for n in lens:
        off.append(off[-1] + n)
    return off


@pytest.mark.parametrize("size", SIZES, ids=lambda s: f"{sum(s[0])}in{len(s[0])}x{s[1]}x{s[2]}")
def test_8_bit_sums_are_exact(size, monkeypatch):
    """Below 2^24 up to K 1024, so equal; above, rounded once to fp32."""
    lens, N, K = size
    monkeypatch.setenv("DG_FORCE_GROUPED", "i8_tile_256x256")
    pad, gen = -K % 16, torch.Generator(device="cuda").manual_seed(K)
    A, B = _i8(gen, sum(lens) + 9, K, pad=pad), _i8(gen, len(lens), N, K, pad=pad)
    desc = dg.make_scaled_desc(A.shape[0], N, K, groups=len(lens), lda=K + pad, ldb=K + pad, stride_b=N * (K + pad))
    assert "kernel=i8_tile_256x256 " in dg.dg_gemm_scaled_describe(desc)
    off = _offsets(lens, 4)
    C = torch.full((A.shape[0], N), 7.0, device="cuda")
    dg.gemm_scaled(A, B, None, None, C, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
    want = torch.full(C.shape, 7.0, device="cuda")
    for e, (lo, hi) in enumerate(groups_of(off, A.shape[0])):
        want[lo:hi] = (A[lo:hi].double() @ B[e].double().t()).float()
    assert torch.equal(C, want)
    if len(lens) == 1:                                      # the deal of one matrix
        got = dg.gemm_scaled(A[:lens[0]], B[0], out_dtype=torch.float32)
        assert torch.equal(got, (A[:lens[0]].double() @ B[0].double().t()).float())


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", ["none", "gelu_erf", "gelu_tanh"])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_8_bit_epilogue(shift, act, out, monkeypatch):
    """Bias, scales, beta and activation into rows that start on any element.
    Tolerance: three roundings of fp32 for conversion and scales, 3.01 * 2^-24
    of the value, the rest as in grouped_util."""
    monkeypatch.setenv("DG_FORCE_GROUPED", "i8_tile_256x256")
    lens, N, K = SIZES[2]
    M, gen = lens[0], torch.Generator(device="cuda").manual_seed(shift)
    A, B = _i8(gen, M, K), _i8(gen, N, K)
    sa = torch.rand(M, device="cuda", generator=gen) / 80
    sb = (0.5 + torch.rand(N, device="cuda", generator=gen)) / (80 * K ** 0.5)
    bias = torch.randn(N, device="cuda", generator=gen).to(DT[out])
    wide = torch.randn(M, N + (shift and 5), device="cuda", generator=gen).to(DT[out])
    before, C = wide.clone(), wide[:, shift:shift + N]
    y = A.double() @ B.double().t() * sa[:, None].double() * sb.double()
    ref, tol = finish(y, None, 3.01 * 2.0 ** -24 * y.abs(), DT[out], alpha=0.75, beta=-0.5, C=C.clone(), bias=bias,
                      act=act)
    dg.gemm_scaled(A, B, sa, sb, C, alpha=0.75, beta=-0.5, bias=bias, act=act)
    check(C, ref, tol)
    outside = torch.ones(wide.shape, dtype=torch.bool, device="cuda")
    outside[:, shift:shift + N] = False
    assert torch.equal(wide[outside], before[outside])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("order", ["row", "col"])
@pytest.mark.parametrize("size", [SIZES[1], SIZES[2], SIZES[5], SIZES[6]],
                         ids=lambda s: f"{sum(s[0])}in{len(s[0])}x{s[1]}x{s[2]}")
def test_16_bit_grouped_sums_are_exact(size, order, dtype, monkeypatch):
    """Integers in [-2, 2]: every product and partial sum is exact."""
    lens, N, K = size
    monkeypatch.setenv("DG_FORCE_GROUPED", "mfma16_256x256")
    gen = torch.Generator(device="cuda").manual_seed(K)
    small = lambda *s: torch.randint(-2, 3, s, device="cuda", generator=gen).to(DT[dtype])
    K8, N8 = (K + 7) // 8 * 8, (N + 7) // 8 * 8             # rows on 16 bytes
    A = small(sum(lens), K8)[:, :K]
    B = (small(len(lens), K, N8)[..., :N] if order == "row" else small(len(lens), N, K8)[..., :K].transpose(1, 2))
    off = _offsets(lens)
    desc = dg.make_grouped_desc("m", len(lens), A.shape[0], N, K=K, a_type=dtype, c_type="f32", b_order=order,
                                lda=K8, ldb=N8 if order == "row" else K8, stride_b=B.stride(0))
    assert "kernel=mfma16_256x256 " in dg.dg_gemm_grouped_describe(desc)
    got = dg.gemm_grouped(A, B, torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
    for e, (lo, hi) in enumerate(groups_of(off, A.shape[0])):
        assert torch.equal(got[lo:hi], A[lo:hi].float() @ B[e].float().contiguous())
