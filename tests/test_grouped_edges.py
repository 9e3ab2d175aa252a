"""Grouped products on the matrix-core kernels where a row ends inside a
16-byte piece, and the large tiles as long problems use them.

The kernels take any operand whose leading dimension is a whole number of 16
bytes, so a row length that is not reaches them as a part of padded rows.  The
padding holds NaN and each allocation ends with the last valid element: a
value read from beside the operand shows in the result."""
import pytest
import torch

import dense_gemm_10_amd as dg
from grouped_util import DT, check, finish, groups_of, ints, offsets_like, sum_error

pytestmark = pytest.mark.gpu

TILES16 = ["mfma16_256x256", "mfma16_128x128"]
STREAMS = ["stream_16x32", "stream_16x64", "stream_32x64"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _offsets(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _padded(t):
    """t on the GPU in rows of a whole number of 16 bytes and at least one
    element of padding, which is NaN; nothing behind the last element."""
    step = 16 // t.element_size()
    ld = (t.shape[-1] // step + 1) * step
    rows = t.numel() // t.shape[-1]
    flat = torch.full(((rows - 1) * ld + t.shape[-1],), float("nan"), dtype=t.dtype, device="cuda")
    part = flat.as_strided((rows, t.shape[-1]), (ld, 1))
    part.copy_(t.reshape(rows, -1))
    strides = (t.shape[-2] * ld, ld, 1) if t.dim() == 3 else (ld, 1)
    return flat.as_strided(t.shape, strides)


def _weights(B, order):
    """B (groups, K, N) padded along N ("kn") or along K ("nk")."""
    return _padded(B) if order == "kn" else _padded(B.transpose(1, 2).contiguous()).transpose(1, 2)


def _runs_on(kernel, dtype, A, W, off, order):
    rows, K = A.shape
    d = dg.make_grouped_desc("m", W.shape[0], rows, W.shape[2], K=K, a_type=dtype, c_type="f32",
                             b_order="row" if order == "kn" else "col", lda=A.stride(0),
                             ldb=max(W.stride(1), W.stride(2)), stride_b=W.stride(0))
    assert f"kernel={kernel} " in dg.dg_gemm_grouped_describe(d)


def _reference(A, B, off, **kw):
    """(reference, tolerance, covered rows) on the GPU, in fp64."""
    A, B = A.cuda().double(), B.cuda().double()
    rows, N, out, C, bias = A.shape[0], B.shape[2], kw["out"], kw.get("C"), kw.get("bias")
    ref, tol = torch.zeros(rows, N, dtype=torch.float64, device="cuda"), None
    tol, inside = torch.zeros_like(ref), torch.zeros(rows, dtype=torch.bool, device="cuda")
    for e, (lo, hi) in enumerate(groups_of(off, rows)):
        if lo < hi:
            y, mag = A[lo:hi] @ B[e], A[lo:hi].abs() @ B[e].abs()
            ref[lo:hi], tol[lo:hi] = finish(
                y, mag, sum_error(A.shape[1], mag), out, alpha=kw.get("alpha", 1.0), beta=kw.get("beta", 0.0),
                C=None if C is None else C[lo:hi], bias=None if bias is None else bias[e], act=kw.get("act", "none"))
            inside[lo:hi] = True
    return ref, tol, inside


# K, N one to seven short of a piece; K below and above a K tile, N past one tile
SHORT = [(7, 9), (33, 65), (66, 130), (75, 131), (132, 260), (141, 29), (70, 143), (191, 263), (129, 7)]


@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("kernel,dtype", [(k, t) for k in TILES16 + STREAMS for t in ("bf16", "f16")] +
                         [(k, "f32") for k in ["mfma_f32_128x128"] + STREAMS])
def test_rows_that_end_inside_a_piece(kernel, dtype, order, monkeypatch):
    monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    gen = torch.Generator().manual_seed(len(kernel))
    for groups, rows in ((3, 45), (4, 301)):
        for K, N in SHORT:
            A, B = ints(gen, rows, K, dtype=DT[dtype]), ints(gen, groups, K, N, dtype=DT[dtype])
            Ad, W, off = _padded(A), _weights(B, order), offsets_like("random", groups, rows, gen)
            _runs_on(kernel, dtype, Ad, W, off, order)
            C = dg.gemm_grouped(Ad, W, _offsets(off), out_dtype=torch.float32)
            assert torch.equal(C.double(), _reference(A, B, off, out=torch.float32)[0]), (K, N, off)


# M, N and group lengths that end inside pieces and K tiles
@pytest.mark.parametrize("kernel,dtype", [(k, t) for k in TILES16 for t in ("bf16", "f16")] +
                         [("mfma_f32_128x128", "f32")])
@pytest.mark.parametrize("M,N", [(9, 130), (131, 7), (70, 261), (263, 69), (124, 140)])
def test_weight_gradient_with_cut_columns(kernel, dtype, M, N, monkeypatch):
    monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    gen = torch.Generator().manual_seed(M)
    rows, off = 400, [0, 1, 1, 64, 128, 203, 267, 400]
    X, G = ints(gen, rows, M, dtype=DT[dtype]), ints(gen, rows, N, dtype=DT[dtype])
    got = dg.gemm_grouped_k(_padded(X).t(), _padded(G), _offsets(off), out_dtype=torch.float32).cpu()
    for e, (lo, hi) in enumerate(groups_of(off, rows)):
        assert torch.equal(got[e], X[lo:hi].float().t() @ G[lo:hi].float()), e


LENGTHS = [
    [300, 0, 128, 129, 256, 1, 640, 512, 127, 1000, 255, 257, 300, 295],   # every kind of last tile
    [1500, 100, 1400],
    [2300, 2300],                                # 4100 columns: a whole wave, and 50 tiles to cut
]


@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "bf16")])
@pytest.mark.parametrize("lengths", LENGTHS, ids=["last tiles", "all cut", "one wave and cut"])
def test_large_tile_with_long_sums_and_epilogues(lengths, dtype, out, order, monkeypatch):
    """The 256 x 256 tile and its halves over five K tiles and a cut one,
    with each group's own bias, activations, alpha and beta, into C of odd
    row starts."""
    monkeypatch.setenv("DG_FORCE_GROUPED", "mfma16_256x256")
    gen = torch.Generator().manual_seed(len(lengths))
    off = [4]
    for n in lengths:
        off.append(off[-1] + n)
    rows, groups = off[-1] + 3, len(lengths)
    N = 4100 if len(lengths) == 2 else 1101
    for K, (alpha, beta, with_bias, act), pad in (
            (320, (1.0, 0.0, True, "gelu_erf"), 0), (360, (0.5, -1.5, True, "gelu_tanh"), 2),
            (363, (1.0, 1.0, False, "none"), 7), (320, (2.0, 0.0, False, "none"), 3)):
        A = torch.randn(rows, K, generator=gen).to(DT[dtype])
        B = (torch.randn(groups, K, N, generator=gen) / K ** 0.5).to(DT[dtype])
        bias = torch.randn(groups, N, generator=gen).to(DT[dtype]).cuda() if with_bias else None
        Ad, W = _padded(A), _weights(B, order)
        _runs_on("mfma16_256x256", dtype, Ad, W, off, order)
        wide = torch.randn(rows, N + pad, generator=gen).to(DT[out]).cuda()
        before, C = wide.clone(), wide[:, pad // 2:pad // 2 + N]
        ref, tol, inside = _reference(A, B, off, out=DT[out], C=C.clone(), alpha=alpha, beta=beta, bias=bias, act=act)
        dg.gemm_grouped(Ad, W, _offsets(off), C, alpha=alpha, beta=beta, bias=bias, act=act)
        check(C[inside], ref[inside], tol[inside], f"{K} {alpha} {beta} {act}")
        wide[:, pad // 2:pad // 2 + N][inside] = 0
        before[:, pad // 2:pad // 2 + N][inside] = 0
        assert torch.equal(wide, before)                        # the other rows and the padding


@pytest.mark.parametrize("kernel", TILES16)
@pytest.mark.parametrize("dtype,out", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16")])
def test_weight_gradient_of_long_groups(kernel, dtype, out, monkeypatch):
    """Groups of several K tiles, accumulated onto C."""
    monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    gen = torch.Generator().manual_seed(77)
    rows, M, N, off = 2100, 333, 518, [3, 703, 703, 1023, 1346, 1347, 2090]
    X, G = (torch.randn(rows, w, generator=gen).to(DT[dtype]) for w in (M, N))
    C0 = torch.randn(len(off) - 1, M, N, generator=gen).to(DT[out])
    for alpha, beta in ((1.0, 0.0), (0.5, 1.0), (1.0, -2.0)):
        C = C0.cuda()
        dg.gemm_grouped_k(_padded(X).t(), _padded(G), _offsets(off), C, alpha=alpha, beta=beta)
        for e, (lo, hi) in enumerate(groups_of(off, rows)):
            x, g = X[lo:hi].double().t(), G[lo:hi].double()
            y, mag = x @ g, x.abs() @ g.abs()
            ref, tol = finish(y, mag, sum_error(hi - lo, mag), DT[out], alpha=alpha, beta=beta, C=C0[e])
            check(C[e], ref, tol, f"{e} {alpha} {beta}")


@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("kernel", ["mfma_f32_128x128"] + STREAMS)
def test_fp32_kernels_with_epilogues(kernel, order, monkeypatch):
    monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    gen = torch.Generator().manual_seed(5)
    groups, rows, K, N = 4, 423, 205, 301
    A, B = torch.randn(rows, K, generator=gen), torch.randn(groups, K, N, generator=gen) / K ** 0.5
    bias, off = torch.randn(groups, N, generator=gen).cuda(), [1, 200, 200, 330, 420]
    Ad, W = _padded(A), _weights(B, order)
    _runs_on(kernel, "f32", Ad, W, off, order)
    for alpha, beta, b, act in ((1.0, 0.0, bias, "gelu_erf"), (0.5, -1.5, bias, "gelu_tanh"), (2.0, 1.0, None, "none")):
        wide = torch.randn(rows, N + 3, generator=gen).cuda()
        C = wide[:, 1:1 + N]
        C0 = C.clone()
        ref, tol, inside = _reference(A, B, off, out=torch.float32, C=C0, alpha=alpha, beta=beta, bias=b, act=act)
        dg.gemm_grouped(Ad, W, _offsets(off), C, alpha=alpha, beta=beta, bias=b, act=act)
        check(C[inside], ref[inside], tol[inside], f"{alpha} {beta} {act}")
        assert torch.equal(C[~inside], C0[~inside])


@pytest.mark.parametrize("N,kernel", [(2 ** 22, "stream_16x64"), (2 ** 23, "mfma16_128x128")])
def test_grids_of_millions_of_workgroups(N, kernel):
    """6.3 million workgroups, and a problem whose first choice would make
    more threads than a launch can have."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    groups, rows, K = 64, 512, 32
    A = torch.randint(-2, 3, (rows, K), generator=gen, device="cuda").bfloat16()
    W = torch.randint(-2, 3, (N, K), generator=gen, device="cuda").bfloat16()
    B = W.t().expand(groups, K, N)
    off = sorted(torch.randint(0, rows + 1, (groups - 1,), generator=gen, device="cuda").tolist())
    d = dg.make_grouped_desc("m", groups, rows, N, K=K, b_order="col", stride_b=0)
    assert f"kernel={kernel} " in dg.dg_gemm_grouped_describe(d)
    C = torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.gemm_grouped(A, B, _offsets([0] + off + [rows]), C)
    for lo in range(0, N, 2 ** 21):                             # whole numbers below 2^8: exact in bf16
        assert torch.equal(C[:, lo:lo + 2 ** 21].float(), A.float() @ W[lo:lo + 2 ** 21].float().t())


def _most_groups(gen, rows, groups=65536):
    """Offsets of 65536 groups of no, one or a few rows, and each row's group."""
    count = torch.bincount(torch.randint(0, groups, (rows,), generator=gen, device="cuda"), minlength=groups)
    count[1000:1200], count[-1] = 0, 40
    count[40000] += rows - 7 - int(count.sum())                 # seven rows behind the last group
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), count.cumsum(0)])
    return off.int(), torch.repeat_interleave(torch.arange(groups, device="cuda"), count)


@pytest.mark.parametrize("kernel", ["", "mfma16_128x128", "mfma16_256x256"])
def test_the_most_groups(kernel, monkeypatch):
    if kernel:
        monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    gen = torch.Generator(device="cuda").manual_seed(8)
    groups, rows, K, N, M = 65536, 70000, 32, 24, 16
    off, of_row = _most_groups(gen, rows)

    def ints_on(*shape):
        return torch.randint(-2, 3, shape, generator=gen, device="cuda").bfloat16()

    A, B, G = ints_on(rows, K), ints_on(groups, K, N), ints_on(rows, N)
    C = torch.full((rows, N), 9.0, device="cuda")
    dg.gemm_grouped(A, B, off, C)
    n = of_row.numel()
    assert n == rows - 7 and bool((C[n:] == 9.0).all())
    assert torch.equal(C[:n], torch.bmm(A[:n, None].float(), B[of_row].float())[:, 0])
    got = dg.gemm_grouped_k(A[:, :M].t(), G, off, out_dtype=torch.float32)
    ref = torch.zeros(groups, M, N, device="cuda")
    ref.index_add_(0, of_row, A[:n, :M, None].float() * G[:n, None].float())
    assert torch.equal(got, ref)
