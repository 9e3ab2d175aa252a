"""dg_gemm_grouped on the GPU against its definition in fp64: types, orders,
group patterns, strides, edges, epilogues, streams and graphs."""
import pytest
import torch

import dense_gemm_10_amd as dg
from grouped_util import DT, check, finish, groups_of, ints, offsets_like, sum_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _offsets(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _ref_m(A, B, off, out, C=None, alpha=1.0, beta=0.0, bias=None, act="none"):
    """(reference, tolerance, covered rows) on the CPU."""
    A, B = A.cpu().double(), B.cpu().double()
    rows, N = A.shape[0], B.shape[2]
    ref, tol = torch.zeros(rows, N, dtype=torch.float64), torch.zeros(rows, N, dtype=torch.float64)
    inside = torch.zeros(rows, dtype=torch.bool)
    for e, (lo, hi) in enumerate(groups_of(off, rows)):
        if lo == hi:
            continue
        y, mag = A[lo:hi] @ B[e], A[lo:hi].abs() @ B[e].abs()
        b = None if bias is None else bias.cpu()[e] if bias.dim() == 2 else bias.cpu()
        ref[lo:hi], tol[lo:hi] = finish(y, mag, sum_error(A.shape[1], mag), out, alpha=alpha, beta=beta,
                                        C=None if C is None else C[lo:hi].cpu(), bias=b, act=act)
        inside[lo:hi] = True
    return ref, tol, inside


def _ref_k(A, B, off, out, C=None, alpha=1.0, beta=0.0):
    A, B = A.cpu().double(), B.cpu().double()
    refs, tols = [], []
    for e, (lo, hi) in enumerate(groups_of(off, B.shape[0])):
        y, mag = A[:, lo:hi] @ B[lo:hi], A[:, lo:hi].abs() @ B[lo:hi].abs()
        r, t = finish(y, mag, sum_error(hi - lo, mag), out, alpha=alpha, beta=beta,
                      C=None if C is None else C[e].cpu())
        refs.append(r), tols.append(t)
    return torch.stack(refs), torch.stack(tols)


# groups, rows, K, N: single rows, odd sizes, sizes around the tiles (16, 64,
# 128, 256), more than 64 groups, K of no whole step
SIZES = [(1, 1, 8, 8), (3, 7, 40, 24), (4, 100, 72, 264), (5, 700, 128, 520), (70, 150, 64, 136),
         (130, 33, 200, 72), (8, 1100, 328, 264), (2, 300, 33, 17), (6, 90, 1000, 40)]


@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_integer_products_are_exact(size, dtype, order):
    groups, rows, K, N = size
    gen = torch.Generator().manual_seed(hash(size) % 1000)
    A = ints(gen, rows, K, dtype=DT[dtype])
    B = ints(gen, groups, K, N, dtype=DT[dtype])
    Bd = B.cuda() if order == "kn" else B.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    for pattern in ("random", "even", "one", "edges", "none"):
        off = offsets_like(pattern, groups, rows, gen)
        C = torch.full((rows, N), float("nan"), device="cuda")
        if dtype == "f32":
            got = dg.gemm_grouped(A.cuda(), Bd, _offsets(off), C)
        else:
            got = dg.gemm_grouped(A.cuda(), Bd, _offsets(off), C)
        assert got is C
        ref, _, inside = _ref_m(A, B, off, torch.float32)
        got = got.cpu().double()
        assert torch.equal(got[inside], ref[inside]), (pattern, off)
        assert bool(got[~inside].isnan().all()), pattern       # rows of no group: as they were


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "bf16"),
                                       ("f32", "f32")])
@pytest.mark.parametrize("act", ["none", "gelu_erf", "gelu_tanh"])
@pytest.mark.parametrize("size,order", [((4, 100, 72, 264), "kn"), ((5, 700, 128, 519), "nk"),
                                        ((9, 30, 256, 136), "nk"), ((9, 30, 256, 136), "kn"),
                                        ((3, 900, 96, 512), "kn"), ((2, 50, 31, 37), "kn")], ids=str)
def test_epilogue(size, order, dtype, out, act):
    groups, rows, K, N = size
    gen = torch.Generator().manual_seed(7)
    A = torch.randn(rows, K, generator=gen).to(DT[dtype])
    B = (torch.randn(groups, K, N, generator=gen) / K ** 0.5).to(DT[dtype])
    Bd = B.cuda() if order == "kn" else B.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    bias = torch.randn(groups, N, generator=gen).to(DT[dtype])
    C0 = torch.randn(rows, N, generator=gen).to(DT[out])
    off = offsets_like("edges", groups, rows, gen)
    for alpha, beta, b in ((1.0, 0.0, bias), (0.5, -1.5, bias[0]), (0.0, 2.0, None)):
        C = C0.cuda()
        dg.gemm_grouped(A.cuda(), Bd, _offsets(off), C, alpha=alpha, beta=beta,
                        bias=None if b is None else b.cuda(), act=act)
        ref, tol, inside = _ref_m(A, B, off, DT[out], C0, alpha, beta, b, act)
        got = C.cpu()
        check(got[inside], ref[inside], tol[inside], f"{alpha} {beta}")
        assert torch.equal(got[~inside], C0[~inside])


# groups, rows, M, N
SIZES_K = [(1, 1, 8, 8), (3, 7, 40, 24), (4, 300, 72, 264), (5, 700, 264, 136), (70, 150, 64, 40),
           (2, 2000, 520, 128), (2, 33, 17, 9), (6, 1100, 256, 512), (3, 129, 1, 264), (4, 260, 264, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", SIZES_K, ids=str)
def test_weight_gradient_of_integers_is_exact(size, dtype):
    groups, rows, M, N = size
    gen = torch.Generator().manual_seed(hash(size) % 1000)
    X, G = ints(gen, rows, M, dtype=DT[dtype]), ints(gen, rows, N, dtype=DT[dtype])
    for pattern in ("random", "even", "one", "edges", "none"):
        off = offsets_like(pattern, groups, rows, gen)
        got = dg.gemm_grouped_k(X.cuda().t(), G.cuda(), _offsets(off), out_dtype=torch.float32)
        ref, _ = _ref_k(X.t(), G, off, torch.float32)
        assert torch.equal(got.cpu().double(), ref), (pattern, off)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_weight_gradient_accumulates(dtype, out):
    gen = torch.Generator().manual_seed(5)
    groups, rows, M, N = 5, 400, 136, 264
    X, G = (torch.randn(rows, w, generator=gen).to(DT[dtype]) for w in (M, N))
    C0 = torch.randn(groups, M, N, generator=gen).to(DT[out])
    off = [0, 0, 120, 121, 390, 390]                    # two empty groups, rows behind the last
    for alpha, beta in ((1.0, 1.0), (0.25, 0.0), (0.0, 3.0)):
        C = C0.cuda()
        dg.gemm_grouped_k(X.cuda().t(), G.cuda(), _offsets(off), C, alpha=alpha, beta=beta)
        ref, tol = _ref_k(X.t(), G, off, DT[out], C0, alpha, beta)
        check(C, ref, tol, f"{alpha} {beta}")


@pytest.mark.parametrize("values", [[5, 3, 9, 2, 40], [-7, -1, 2, 2 ** 31 - 1, 0], [-2 ** 31] * 5,
                                    [2 ** 31 - 1] * 5, [50, 0, 10, 60, 61]], ids=str)
def test_any_offsets_stay_inside(values):
    """Decreasing, negative and too large offsets are clamped and made
    non-decreasing, as the header says; every operand is exactly as long as
    the call says."""
    gen = torch.Generator().manual_seed(3)
    rows, K, N, groups = 60, 64, 72, 4
    A, B = ints(gen, rows, K, dtype=torch.bfloat16), ints(gen, groups, K, N, dtype=torch.bfloat16)
    C = torch.full((rows, N), 7.0, device="cuda")
    dg.gemm_grouped(A.cuda(), B.cuda(), _offsets(values), C)
    ref, _, inside = _ref_m(A, B, values, torch.float32)
    ref[~inside] = 7.0
    assert torch.equal(C.cpu().double(), ref)
    G = ints(gen, rows, N, dtype=torch.bfloat16)
    got = dg.gemm_grouped_k(A.cuda().t(), G.cuda(), _offsets(values), out_dtype=torch.float32)
    assert torch.equal(got.cpu().double(), _ref_k(A.t(), G, values, torch.float32)[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,first", [(8, 0), (3, 1), (8, 1)])
def test_strides_and_alignment(dtype, pad, first):
    """Rows with padding between them (whole 16 bytes or not), operands that
    do not start on 16 bytes, one B and one bias for every group."""
    gen = torch.Generator().manual_seed(11)
    groups, rows, K, N = 3, 80, 72, 88
    dt = DT[dtype]

    def padded(*shape):
        t = ints(gen, *shape[:-1], shape[-1] + pad + first, dtype=dt).cuda()
        return t[..., first:first + shape[-1]]

    A, W, G = padded(rows, K), padded(groups, K, N), padded(rows, N)
    off = [2, 30, 30, 77]
    wide = torch.full((rows, N + pad), 3.0, device="cuda")
    C = wide[:, first:first + N] if first + N <= N + pad else wide[:, :N]
    dg.gemm_grouped(A, W, _offsets(off), C)
    ref, _, inside = _ref_m(A, W, off, torch.float32)
    assert torch.equal(C.cpu().double()[inside], ref[inside])
    mask = torch.ones_like(wide, dtype=torch.bool)
    mask[:, C.storage_offset():C.storage_offset() + N][inside.cuda()] = False
    assert bool((wide[mask] == 3.0).all())                      # padding and other rows untouched
    one = W[1:2].expand(groups, K, N)                           # broadcast
    C = torch.zeros(rows, N, device="cuda")
    dg.gemm_grouped(A, one, _offsets(off), C, bias=G[0])
    ref, _, inside = _ref_m(A, one, off, torch.float32, bias=G[0])
    assert torch.equal(C.cpu().double()[inside], ref[inside])
    got = dg.gemm_grouped_k(A.t(), G, _offsets(off), out_dtype=torch.float32)
    assert torch.equal(got.cpu().double(), _ref_k(A.t(), G, off, torch.float32)[0])


@pytest.mark.parametrize("rows", [24, 400])
@pytest.mark.parametrize("order", ["kn", "nk"])
def test_nan_rows_reach_no_other_row(rows, order):
    """NaN and infinity in rows of no group, and in other groups' rows and
    weights, stay there."""
    gen = torch.Generator().manual_seed(2)
    groups, K, N = 4, 64, 136
    A, B = ints(gen, rows, K, dtype=torch.bfloat16), ints(gen, groups, K, N, dtype=torch.bfloat16)
    G = ints(gen, rows, N, dtype=torch.bfloat16)
    off = [rows // 8, rows // 3, rows // 2, rows // 2, rows - 3]
    ref, _, inside = _ref_m(A, B, off, torch.float32)
    refk = _ref_k(A.t(), G, off, torch.float32)[0]
    lo, hi = off[1], off[2]
    A[~inside] = float("nan")
    G[~inside] = float("inf")
    B[2] = float("nan")                                          # an empty group's weights
    A[lo:hi] = float("inf")
    Bd = B.cuda() if order == "kn" else B.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    C = dg.gemm_grouped(A.cuda(), Bd, _offsets(off), out_dtype=torch.float32).cpu().double()
    keep = inside.clone()
    keep[lo:hi] = False
    assert torch.equal(C[keep], ref[keep])
    assert not bool(C[lo:hi].isfinite().any())
    A[lo:hi] = 1.0
    got = dg.gemm_grouped_k(A.cuda().t(), G.cuda(), _offsets(off), out_dtype=torch.float32).cpu().double()
    for e in (0, 2, 3):
        assert torch.equal(got[e], refk[e]), e


def test_replayed_graph_reads_the_offsets_anew():
    gen = torch.Generator().manual_seed(9)
    groups, rows, K, N = 5, 260, 72, 136
    A, B = ints(gen, rows, K, dtype=torch.bfloat16).cuda(), ints(gen, groups, K, N, dtype=torch.bfloat16).cuda()
    G = ints(gen, rows, N, dtype=torch.bfloat16).cuda()
    off = _offsets([0] * 6)
    C, D = torch.zeros(rows, N, device="cuda"), torch.zeros(groups, K, N, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dg.gemm_grouped(A, B, off, C)
        dg.gemm_grouped_k(A.t(), G, off, D)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.gemm_grouped(A, B, off, C)
        dg.gemm_grouped_k(A.t(), G, off, D)
    for pattern in ("random", "one", "edges", "none", "random"):
        values = offsets_like(pattern, groups, rows, gen)
        off.copy_(_offsets(values))
        C.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        eager = torch.full_like(C, -1.0)
        dg.gemm_grouped(A, B, off, eager)                       # the program's own work between replays
        torch.cuda.synchronize()
        assert torch.equal(C, eager), pattern
        ref, _, inside = _ref_m(A, B, values, torch.float32)
        assert torch.equal(C.cpu().double()[inside], ref[inside]), pattern
        assert torch.equal(D.cpu().double(), _ref_k(A.t(), G, values, torch.float32)[0]), pattern


def test_streams_at_once():
    """Calls on two streams, their own operands made on those streams."""
    gen = torch.Generator().manual_seed(4)
    groups, rows, K, N = 4, 200, 64, 72
    hA, hB = ints(gen, rows, K, dtype=torch.float16), ints(gen, groups, K, N, dtype=torch.float16)
    off = [0, 60, 61, 180, 200]
    ref = _ref_m(hA, hB, off, torch.float32)[0]
    outs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            A, B, o = hA.cuda() * (i + 1), hB.cuda(), _offsets(off)
            outs.append(dg.gemm_grouped(A, B, o, out_dtype=torch.float32))
            outs.append(dg.gemm_grouped(A, B, o, out_dtype=torch.float32, stream=s.cuda_stream))
    torch.cuda.synchronize()
    for i, C in enumerate(outs):
        assert torch.equal(C.cpu().double(), ref * (i // 2 + 1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_empty_sizes(dtype):
    """K = 0 gives act(beta C + bias), no rows gives beta C (0) weight
    gradients, no groups or columns change nothing."""
    dt = DT[dtype]

    def t(*shape):
        return torch.ones(shape, dtype=dt, device="cuda")

    off = _offsets([1, 3, 4])
    bias = torch.tensor([[1.0, 2.0, 3.0], [4.0, 5.0, 6.0]], dtype=dt, device="cuda")
    C = torch.full((5, 3), 7.0, dtype=dt, device="cuda")
    dg.gemm_grouped(t(5, 0), t(2, 0, 3), off, C, beta=2.0, bias=bias)
    want = [[7.0] * 3, [15.0, 16.0, 17.0], [15.0, 16.0, 17.0], [18.0, 19.0, 20.0], [7.0] * 3]
    assert C.tolist() == want
    D = torch.full((2, 4, 3), 2.0, dtype=dt, device="cuda")
    dg.gemm_grouped_k(t(0, 4).t(), t(0, 3), _offsets([0, 0, 0]), D, beta=1.5)
    assert bool((D == 3.0).all())
    assert bool((dg.gemm_grouped_k(t(0, 4).t(), t(0, 3), _offsets([0, 0, 0])) == 0.0).all())
    before = C.clone()
    dg.gemm_grouped(t(5, 2), t(0, 2, 3), _offsets([0]), C)
    assert torch.equal(C, before)
    assert dg.gemm_grouped(t(5, 2), t(2, 2, 0), off).shape == (5, 0)
    assert dg.gemm_grouped_k(t(5, 0).t(), t(5, 3), off).shape == (2, 0, 3)
    assert dg.gemm_grouped(t(0, 2), t(2, 2, 3), _offsets([0, 0, 0])).shape == (0, 3)


def test_one_group_longer_than_the_mean():
    """Many groups, one of which has nearly every row, on each kernel that
    the mean length chooses."""
    gen = torch.Generator().manual_seed(21)
    for groups, rows, K, N in ((40, 200, 96, 72), (30, 400, 64, 136), (12, 600, 72, 264), (9, 2400, 64, 136)):
        A, B = ints(gen, rows, K, dtype=torch.bfloat16), ints(gen, groups, K, N, dtype=torch.bfloat16)
        off = [0] * 3 + [2] + [rows - 1] * (groups - 4) + [rows]
        got = dg.gemm_grouped(A.cuda(), B.cuda(), _offsets(off), out_dtype=torch.float32)
        assert torch.equal(got.cpu().double(), _ref_m(A, B, off, torch.float32)[0]), groups


@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("rows,lengths", [
    (4200, [300, 0, 128, 129, 256, 1, 640, 512, 127, 1000, 255, 257, 300, 295]),   # every kind of last tile
    (2600, [2600]), (2560, [1280, 1280]), (3000, [1500, 100, 1400]),
    (5000, [90] * 10 + [100] * 10 + [1500, 1600]),
])
def test_whole_and_half_tiles(rows, lengths, order):
    """The 256 x 256 tile with its half-height tiles: last tiles of up to and
    over 128 rows, with and without a partly filled last wave to cut."""
    gen = torch.Generator().manual_seed(rows)
    groups, K = len(lengths), 64
    off = [0]
    for n in lengths:
        off.append(off[-1] + n)
    assert off[-1] <= rows
    A = ints(gen, rows, K, dtype=torch.bfloat16)
    for N in (264, 1100 if order == "nk" else 1104, 2048):
        B = ints(gen, groups, K, N, dtype=torch.bfloat16)
        Bd = B.cuda() if order == "kn" else B.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        C = torch.full((rows, N), float("nan"), device="cuda")
        with pytest.MonkeyPatch.context() as m:
            m.setenv("DG_FORCE_GROUPED", "mfma16_256x256")
            dg.gemm_grouped(A.cuda(), Bd, _offsets(off), C)
        ref, _, inside = _ref_m(A, B, off, torch.float32)
        got = C.cpu().double()
        assert torch.equal(got[inside], ref[inside]), N
        assert bool(got[~inside].isnan().all())


@pytest.mark.parametrize("kernel", ["mfma16_256x256", "mfma16_128x128", "mfma_f32_128x128", "stream_16x32",
                                    "stream_16x64", "stream_32x64"])
def test_every_kernel_takes_every_pattern(kernel, monkeypatch):
    """The kernel a problem gets depends on its sizes alone; each of them is
    right for any lengths."""
    monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    dtype = torch.float32 if "f32" in kernel else torch.bfloat16
    gen = torch.Generator().manual_seed(31)
    for groups, rows, K, N in ((3, 7, 40, 24), (70, 500, 96, 136), (5, 900, 72, 520)):
        A, B = ints(gen, rows, K, dtype=dtype), ints(gen, groups, K, N, dtype=dtype)
        G = ints(gen, rows, N, dtype=dtype)
        for pattern in ("random", "one", "edges", "none"):
            off = offsets_like(pattern, groups, rows, gen)
            C = torch.full((rows, N), 5.0, device="cuda")
            dg.gemm_grouped(A.cuda(), B.cuda(), _offsets(off), C)
            ref, _, inside = _ref_m(A, B, off, torch.float32)
            ref[~inside] = 5.0
            assert torch.equal(C.cpu().double(), ref), (pattern, off)
            got = dg.gemm_grouped_k(A.cuda().t(), G.cuda(), _offsets(off), out_dtype=torch.float32)
            assert torch.equal(got.cpu().double(), _ref_k(A.t(), G, off, torch.float32)[0])


@pytest.mark.parametrize("kernel", ["mfma16_256x256", "mfma16_128x128"])
@pytest.mark.parametrize("M,N", [(520, 648), (136, 3080), (3080, 136)])
def test_weight_gradient_of_many_tiles(kernel, M, N, monkeypatch):
    """More tiles than the chip holds at once, in bands that end anywhere."""
    monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    gen = torch.Generator().manual_seed(M + N)
    groups, rows = 60, 700
    A, G = ints(gen, rows, M, dtype=torch.bfloat16), ints(gen, rows, N, dtype=torch.bfloat16)
    off = offsets_like("random", groups, rows, gen)
    got = dg.gemm_grouped_k(A.cuda().t(), G.cuda(), _offsets(off), out_dtype=torch.float32).cpu()
    for e, (lo, hi) in enumerate(groups_of(off, rows)):
        assert torch.equal(got[e], A[lo:hi].float().t() @ G[lo:hi].float()), e


def test_weight_gradient_of_many_tiles_and_long_groups():
    gen = torch.Generator().manual_seed(12)
    groups, rows, M, N = 5, 2400, 1928, 1800
    A, G = ints(gen, rows, M, dtype=torch.bfloat16), ints(gen, rows, N, dtype=torch.bfloat16)
    off = [0, 1500, 1500, 1533, 2399, 2400]
    got = dg.gemm_grouped_k(A.cuda().t(), G.cuda(), _offsets(off), out_dtype=torch.float32).cpu()
    for e, (lo, hi) in enumerate(groups_of(off, rows)):
        assert torch.equal(got[e], A[lo:hi].float().t() @ G[lo:hi].float()), e


def test_runs_repeat_bit_for_bit():
    gen = torch.Generator().manual_seed(6)
    groups, rows, K, N = 6, 500, 264, 264
    A = torch.randn(rows, K, generator=gen).bfloat16().cuda()
    B = torch.randn(groups, K, N, generator=gen).bfloat16().cuda()
    G = torch.randn(rows, N, generator=gen).bfloat16().cuda()
    off = _offsets(offsets_like("random", groups, rows, gen))
    first = dg.gemm_grouped(A, B, off), dg.gemm_grouped_k(A.t(), G, off)
    for _ in range(5):
        assert torch.equal(dg.gemm_grouped(A, B, off), first[0])
        assert torch.equal(dg.gemm_grouped_k(A.t(), G, off), first[1])


@pytest.mark.parametrize("order", ["kn", "nk"])
def test_operands_past_2_31_elements(order):
    """The last group's weights and the last rows lie past 2^31 elements."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    K, N, groups = 4096, 4096, 130                               # 2.18e9 elements of B
    B = torch.zeros(groups, K, N, dtype=torch.bfloat16, device="cuda")
    last = torch.randint(-2, 3, (K, N), generator=gen, device="cuda").bfloat16()
    B[-1] = last
    A = torch.randint(-2, 3, (20, K), generator=gen, device="cuda").bfloat16()
    off = _offsets([0] * 130 + [20])
    W = B if order == "kn" else B.transpose(1, 2)
    C = dg.gemm_grouped(A, W, off, out_dtype=torch.float32)
    w = last if order == "kn" else last.t()
    assert torch.equal(C.double(), A.double() @ w.double())
    del B, W
    # rows 2^16 apart by 2^15 + 8 elements
    rows = 66000
    X = torch.zeros(rows, 32776, dtype=torch.bfloat16, device="cuda")
    X[-300:] = torch.randint(-2, 3, (300, 32776), generator=gen, device="cuda").bfloat16()
    V = torch.randint(-2, 3, (2, 64, 72), generator=gen, device="cuda").bfloat16()
    off = _offsets([0, rows - 300, rows])
    C = dg.gemm_grouped(X[:, 32704:32768], V, off, out_dtype=torch.float32)
    assert torch.equal(C[-300:].double(), X[-300:, 32704:32768].double() @ V[1].double())
    D = dg.gemm_grouped_k(X[:, 32704:32768].t(), X[:, :72], off, out_dtype=torch.float32)
    assert torch.equal(D[1].double(), X[-300:, 32704:32768].double().t() @ X[-300:, :72].double())
    assert bool((D[0] == 0).all())


def test_gradients_against_differences():
    """L = sum(R * (A . B)): dA = R . B^T and dB = A^T . R by the two
    products, against central differences of L in fp64 (L is bilinear, so
    they are exact) and against the formula."""
    gen = torch.Generator().manual_seed(8)
    groups, rows, K, N = 3, 40, 24, 16
    A, B = ints(gen, rows, K), ints(gen, groups, K, N)
    R = ints(gen, rows, N)
    off = [0, 11, 11, 40]
    o = _offsets(off)
    dA = dg.gemm_grouped(R.cuda(), B.cuda().transpose(1, 2), o).cpu().double()
    dB = dg.gemm_grouped_k(A.cuda().t(), R.cuda(), o).cpu().double()
    ones = torch.ones(rows, 1, device="cuda")
    dbias = dg.gemm_grouped_k(ones.t(), R.cuda(), o).cpu().double()[:, 0]

    def loss(A, B):
        return sum(((A[lo:hi] @ B[e]) * R[lo:hi].double()).sum()
                   for e, (lo, hi) in enumerate(groups_of(off, rows)))

    A64, B64 = A.double(), B.double()
    for i, k in ((0, 0), (10, 23), (11, 5), (39, 7)):
        d = torch.zeros_like(A64)
        d[i, k] = 0.5
        assert float(loss(A64 + d, B64) - loss(A64 - d, B64)) == float(dA[i, k])
    for e, k, n in ((0, 3, 4), (1, 0, 0), (2, 23, 15)):
        d = torch.zeros_like(B64)
        d[e, k, n] = 0.5
        assert float(loss(A64, B64 + d) - loss(A64, B64 - d)) == float(dB[e, k, n])
    for e, (lo, hi) in enumerate(groups_of(off, rows)):
        assert torch.equal(dA[lo:hi], R[lo:hi].double() @ B64[e].t())
        assert torch.equal(dbias[e], R[lo:hi].double().sum(0))
