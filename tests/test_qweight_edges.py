"""4-bit weights on every kernel where A holds NaN, infinities or subnormals."""
import pytest
import torch

import dense_gemm_10_amd as dg
from grouped_util import ints

pytestmark = pytest.mark.gpu

KERNELS = ["qstream_16x16", "qstream_16x32", "qstream_16x64", "qstream_32x32", "qstream_32x64",
           "qstream_32x128", "qtile_64x256", "qtile_64x512"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _pack(q):
    return q[..., 0::2] | (q[..., 1::2] << 4)


def _weights(q, scales, zeros, g):
    at = torch.arange(q.shape[-1]) // g
    zero = 8.0 if zeros is None else zeros.double()[..., at]
    return (q.double() - zero) * scales.double()[..., at]


def _case(gen, lead, N, K, g, with_zeros, scale_dtype=torch.float32, low=-2):
    """Codes, scales that are powers of two from 2^low, zeros."""
    q = torch.randint(0, 16, (*lead, N, K), generator=gen, dtype=torch.uint8)
    scales = 2.0 ** torch.randint(low, low + 4, (*lead, N, K // g), generator=gen)
    zeros = torch.randint(0, 16, (*lead, N, K // g), generator=gen, dtype=torch.uint8) if with_zeros else None
    return q, scales.to(scale_dtype), zeros


def _dev(t):
    return None if t is None else t.cuda()


def _forced(kernel, monkeypatch, M, N, K, g):
    monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    got = dg.dg_gemm_qweight_describe(dg.make_qweight_desc(M, N, K, g))
    assert f"kernel={kernel} " in got


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("g", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_nan_stays_in_its_row_and_column(kernel, g, dtype, monkeypatch):
    """A last row tile that is cut, NaN in its last row and in two others; a
    column with an infinite and one with a NaN scale."""
    if kernel == "qtile_64x512" and g % 128:
        pytest.skip("taken for group sizes that are multiples of 128")
    M, N, K = 70, 530, 1184
    K -= K % g
    _forced(kernel, monkeypatch, M, N, K, g)
    gen = torch.Generator().manual_seed(g)
    q, scales, zeros = _case(gen, (), N, K, g, dtype == torch.float16)
    A = ints(gen, M, K, dtype=dtype)
    ref = A.double() @ _weights(q, scales, zeros, g).t()
    rows, cols = [1, 65, 69], [7, 529]
    A[1, 5], A[65, K - 1], A[69, 0] = (float("nan"),) * 3
    scales[7, 1], scales[529, 0] = float("inf"), float("nan")
    got = dg.gemm_qweight(A.cuda(), _pack(q).cuda(), scales.cuda(), _dev(zeros), group_size=g,
                          out_dtype=torch.float32).cpu().double()
    keep = torch.ones(M, N, dtype=torch.bool)
    keep[rows], keep[:, cols] = False, False
    assert torch.equal(got[keep], ref[keep])
    assert bool(got[rows].isnan().all()) and not bool(got[:, cols].isfinite().any())


@pytest.mark.parametrize("kernel", KERNELS + ["generic"])
@pytest.mark.parametrize("g", [32, 64, 128])
@pytest.mark.parametrize("dtype,with_zeros", [(torch.float16, False), (torch.float16, True), (torch.bfloat16, True)])
def test_subnormals(kernel, g, dtype, with_zeros, monkeypatch):
    """Multiples of the type's smallest subnormal, scales that bring them
    back: the products' absolute values add to less than 2^24 units, so every
    product and sum is exact."""
    if kernel == "qtile_64x512" and g % 128:
        pytest.skip("taken for group sizes that are multiples of 128")
    M, N, K = 67, 520, 768
    if kernel == "generic":
        K += 16                                # no whole step
    else:
        _forced(kernel, monkeypatch, M, N, K, g)
    unit, normal, low = (2.0 ** -24, 2.0 ** -14, 20) if dtype == torch.float16 else (2.0 ** -133, 2.0 ** -126, 118)
    gen = torch.Generator().manual_seed(g)
    q = torch.randint(0, 16, (N, K), generator=gen, dtype=torch.uint8)
    S = -(-K // g)
    scales = (2.0 ** torch.randint(low, low + 2, (N, S), generator=gen).double()).float()
    zeros = torch.randint(0, 16, (N, S), generator=gen, dtype=torch.uint8) if with_zeros else None
    A = (torch.randint(-60, 61, (M, K), generator=gen).double() * unit).to(dtype)
    A[5] = unit                                # one sign: the sums of A are large
    A[6, ::2] = normal                         # the smallest normal beside subnormals
    got = dg.gemm_qweight(A.cuda(), _pack(q).cuda(), scales.cuda(), _dev(zeros), group_size=g,
                          out_dtype=torch.float32)
    assert torch.equal(got.cpu().double(), A.double() @ _weights(q, scales, zeros, g).t())


@pytest.mark.parametrize("kernel", KERNELS + ["generic"])
@pytest.mark.parametrize("g", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("experts", [False, True])
def test_infinities_and_large_values_follow_the_formula(kernel, g, dtype, experts, monkeypatch):
    """Infinities in A and in the scales, and (bf16) rows whose products with
    16 + q pass the largest fp32: the formula's infinity, NaN or value, the
    same from every kernel."""
    if kernel == "qtile_64x512" and g % 128:
        pytest.skip("taken for group sizes that are multiples of 128")
    M, N, K = 70, 530, 512
    if kernel == "generic":
        K += 16
    else:
        _forced(kernel, monkeypatch, M, N, K, g)
    gen = torch.Generator().manual_seed(g)
    lead, S = (3,) if experts else (), -(-K // g)
    q = torch.randint(0, 16, (*lead, N, K), generator=gen, dtype=torch.uint8)
    scales = 2.0 ** torch.randint(-9, -7, (*lead, N, S), generator=gen).float()
    scales[..., 7, 1], scales[..., 300, 0], scales[..., 11, 0] = float("inf"), -float("inf"), 0.0
    zeros = torch.randint(0, 16, (*lead, N, S), generator=gen, dtype=torch.uint8) if g == 64 else None
    A = ints(gen, M, K, dtype=dtype)
    inf = float("inf")
    A[1, 5], A[65, K - 1], A[69, 0], A[69, 9], A[40, 3], A[40, 4] = inf, -inf, inf, -inf, -inf, float("nan")
    if dtype == torch.bfloat16:                # (16 + q) A passes 2^128; the sums of W A are exact, below 2^126
        A[30] = 2.0 ** 124 * (1 - 2 * (torch.arange(K) % 2))
        A[68] = A[30]
    off = [0, 31, 60, M] if experts else None
    C = dg.gemm_qweight(A.cuda(), _pack(q).cuda(), scales.cuda(), _dev(zeros), group_size=g,
                        offsets=None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda"),
                        out_dtype=torch.float32).cpu().double()
    W = _weights(q, scales, zeros, g)
    ref = A.double() @ W.t() if off is None else torch.cat(
        [A[lo:hi].double() @ W[e].t() for e, (lo, hi) in enumerate(zip(off[:-1], off[1:]))])
    assert bool(ref[30, 12:299].isfinite().all()) and bool(ref[1].isinf().any()) and bool(ref[1].isnan().any())
    torch.testing.assert_close(C, ref, rtol=0, atol=0, equal_nan=True)


def test_launch_past_the_first_choice():
    """16 rows of so many columns that the 16 x 64 shape would make more
    threads than a launch can have."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    M, N, K, g = 16, 2 ** 29, 32, 128
    assert "kernel=qstream_32x128 " in dg.dg_gemm_qweight_describe(dg.make_qweight_desc(M, N, K, g))
    A = torch.randint(-2, 3, (M, K), generator=gen, device="cuda").bfloat16()
    Q = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.ones(N, 1, dtype=torch.bfloat16, device="cuda")
    C = torch.full((M, N), float("nan"), dtype=torch.float16, device="cuda")
    dg.gemm_qweight(A, Q, scales, None, C, group_size=g)
    step = 2 ** 24
    for lo in range(0, N, step):                                # whole numbers of at most 512: exact in fp16
        q = Q[lo:lo + step]
        w = torch.stack([q & 15, q >> 4], -1).flatten(-2).half() - 8
        assert torch.equal(C[:, lo:lo + step].float(), A.float() @ w.float().t())


@pytest.mark.parametrize("M,N", [(1, 8320), (16, 9000), (32, 4100), (64, 4096), (300, 16600)])
@pytest.mark.parametrize("stride", [0, 8])
def test_one_group_with_offsets_runs_what_one_without_them_runs(M, N, stride):
    """With one group the offsets change nothing in the kernel's choice, and
    the distance of a second group, which is not there, neither: the same
    sums, bit for bit, whatever the rows of the group."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    K, g = 1056, 32
    A = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    Q = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.rand(N, K // g, generator=gen, device="cuda")
    one = Q.as_strided((1, N, K // 2), (N * K // 2 + stride, K // 2, 1))
    ref = dg.gemm_qweight(A, Q, scales, group_size=g, out_dtype=torch.float32)
    for lo, hi in ((0, M), (M // 3, M), (0, M - M // 4)):
        C = torch.full((M, N), 3.0, device="cuda")
        dg.gemm_qweight(A, one, scales[None], None, C, group_size=g,
                        offsets=torch.tensor([lo, hi], dtype=torch.int32, device="cuda"))
        assert bool((C[:lo] == 3.0).all()) and bool((C[hi:] == 3.0).all())
        assert torch.equal(C[lo:hi], ref[lo:hi])


@pytest.mark.parametrize("kernel", ["", "qstream_16x16", "qstream_32x128"])
def test_the_most_groups(kernel, monkeypatch):
    if kernel:
        monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    gen = torch.Generator(device="cuda").manual_seed(9)
    groups, rows, N, K, g = 65536, 70000, 24, 32, 32
    count = torch.bincount(torch.randint(0, groups, (rows - 50,), generator=gen, device="cuda"), minlength=groups)
    count[-1] += 43                                             # seven rows behind the last group
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), count.cumsum(0)]).int()
    of_row = torch.repeat_interleave(torch.arange(groups, device="cuda"), count)
    A = torch.randint(-2, 3, (rows, K), generator=gen, device="cuda").bfloat16()
    Q = torch.randint(0, 256, (groups, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = 2.0 ** torch.randint(-1, 2, (groups, N, 1), generator=gen, device="cuda").float()
    C = torch.full((rows, N), 9.0, device="cuda")
    dg.gemm_qweight(A, Q, scales, None, C, group_size=g, offsets=off)
    n = of_row.numel()
    assert n == rows - 7 and bool((C[n:] == 9.0).all())
    w = (torch.stack([Q & 15, Q >> 4], -1).flatten(-2).float() - 8) * scales
    assert torch.equal(C[:n], torch.bmm(w[of_row], A[:n, :, None].float())[:, :, 0])
