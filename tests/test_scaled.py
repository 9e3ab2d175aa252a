"""dg_gemm_scaled on the GPU against its definition: every kernel on every
pattern of lengths, exact sums, epilogues, any alignment, float operands,
extremes, streams and graphs.

Tolerance: the sum is exact; converting it to fp32 and multiplying by two
scales are three roundings, 2^-24 each, of a value y: 3.01 * 2^-24 |y|; the
epilogue and the output as in grouped_util."""
import pytest
import torch

import dense_gemm_10_amd as dg
from grouped_util import DT, check, finish, groups_of, offsets_like
from tokens_util import codes64, same_bits

pytestmark = pytest.mark.gpu

KERNELS = ["i8_stream_16x16", "i8_stream_16x32", "i8_stream_16x32_short", "i8_stream_16x64", "i8_stream_32x32",
           "i8_any_64x128", "i8_tile_64x128", "i8_any_128x128", "i8_tile_128x128_deep", "i8_tile_128x128", "i8_tile_256x256"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _i8(gen, *shape):
    return torch.randint(-128, 128, shape, generator=gen, dtype=torch.int8)


def _padded(t, pad, lead=0):
    """t on the GPU with rows `pad` bytes apart from their end, `lead` bytes into its storage."""
    ld = t.shape[-1] + pad
    n = torch.Size(t.shape[:-1]).numel() * ld
    flat = torch.full((lead + n,), 77, dtype=torch.int8, device="cuda")
    strides, step = [1, ld], ld
    for size in reversed(t.shape[1:-1]):
        step *= size
        strides.append(step)
    out = torch.as_strided(flat, t.shape, strides[::-1][-t.dim():], lead)
    out.copy_(t)
    return out


def _ref(A, B, sa, sb, out, off=None, C=None, alpha=1.0, beta=0.0, bias=None, act="none"):
    """(reference, tolerance, covered rows) on the CPU."""
    M, N = A.shape[0], B.shape[-2]
    ref, tol = torch.zeros(M, N, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    inside = torch.zeros(M, dtype=torch.bool)
    for e, (lo, hi) in enumerate([(0, M)] if off is None else groups_of(off, M)):
        if lo == hi:
            continue
        pick = (lambda t: t) if off is None else (lambda t: t[e])
        y = A[lo:hi].double() @ pick(B).double().t()
        if sa is not None:
            y = y * sa[lo:hi, None].double()
        if sb is not None:
            y = y * pick(sb).double()
        b = None if bias is None else pick(bias) if bias.dim() == 2 else bias
        ref[lo:hi], tol[lo:hi] = finish(y, None, 3.01 * 2.0 ** -24 * y.abs(), out, alpha=alpha, beta=beta,
                                        C=None if C is None else C[lo:hi], bias=b, act=act)
        inside[lo:hi] = True
    return ref, tol, inside


# groups, M, N, K: one row, sizes around the tiles (16 to 256), more than 64 groups, K from 0 over parts of a step
SIZES = [(1, 1, 16, 16), (3, 7, 40, 48), (4, 100, 72, 256), (5, 700, 260, 144), (70, 150, 33, 128), (2, 40, 300, 1026),
         (130, 33, 64, 2), (3, 600, 520, 400), (1, 300, 257, 0)]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sums_are_exact_on_every_kernel(size, kernel, monkeypatch):
    groups, M, N, K = size
    monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    desc = dg.make_scaled_desc(M, N, K, groups=groups, lda=K + -K % 16 or 16, ldb=K + -K % 16 or 16,
                               stride_b=N * (K + -K % 16))
    assert f"kernel={kernel} " in dg.dg_gemm_scaled_describe(desc)
    gen = torch.Generator().manual_seed(M + N)
    A, B = _i8(gen, M, K), _i8(gen, groups, N, K)
    Ad, Bd = _padded(A, -K % 16 or 16 * (K == 0)), _padded(B, -K % 16 or 16 * (K == 0))
    for pattern in ("random", "even", "one", "edges", "none"):
        off = offsets_like(pattern, groups, M, gen)
        C = torch.full((M, N), float("nan"), device="cuda")
        dg.gemm_scaled(Ad, Bd, None, None, C, offsets=torch.tensor(off, dtype=torch.int32).cuda())
        ref, _, inside = _ref(A, B, None, None, torch.float32, off)
        got = C.cpu()
        assert torch.equal(got[inside], ref[inside].float()), pattern
        assert bool(got[~inside].isnan().all()), pattern         # rows of no group: as they were
    got = dg.gemm_scaled(Ad, Bd[0], out_dtype=torch.float32).cpu()
    assert torch.equal(got, _ref(A, B[0], None, None, torch.float32)[0].float())


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", ["none", "gelu_erf", "gelu_tanh"])
def test_epilogue(act, out, kernel, monkeypatch):
    monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    gen = torch.Generator().manual_seed(7)
    for groups, M, N, K, st in ((4, 270, 300, 256, "f32"), (3, 50, 264, 96, "bf16")):
        A, B = _i8(gen, M, K), _i8(gen, groups, N, K)
        sa = torch.rand(M, generator=gen) / 80
        sb = ((0.5 + torch.rand(groups, N, generator=gen)) / (80 * K ** 0.5)).to(DT[st])
        bias = torch.randn(groups, N, generator=gen).to(DT[out])
        C0 = torch.randn(M, N, generator=gen).to(DT[out])
        off = offsets_like("edges", groups, M, gen)
        offd = torch.tensor(off, dtype=torch.int32).cuda()
        for alpha, beta, b in ((1.0, 0.0, bias), (0.5, -1.5, bias[0]), (0.0, 2.0, None)):
            C = C0.cuda()
            dg.gemm_scaled(A.cuda(), B.cuda(), sa.cuda(), sb.cuda(), C, offsets=offd, alpha=alpha, beta=beta,
                           bias=None if b is None else b.cuda(), act=act)
            ref, tol, inside = _ref(A, B, sa, sb, DT[out], off, C0, alpha, beta, b, act)
            got = C.cpu()
            check(got[inside], ref[inside], tol[inside], f"{alpha} {beta}")
            assert torch.equal(got[~inside], C0[~inside])
        C = C0.cuda()
        dg.gemm_scaled(A.cuda(), B[1].cuda(), sa.cuda(), sb[1].cuda(), C, beta=1.0, bias=bias[1].cuda(), act=act)
        ref, tol, _ = _ref(A, B[1], sa, sb[1], DT[out], None, C0, 1.0, 1.0, bias[1], act)
        check(C.cpu(), ref, tol, "one matrix")


@pytest.mark.parametrize("M", [1, 5, 16, 17, 40, 300])
@pytest.mark.parametrize("K,pad,lead", [(1, 0, 0), (15, 0, 0), (33, 0, 3), (127, 1, 0), (129, 0, 1), (1001, 0, 0),
                                        (256, 1, 0), (250, 6, 5), (1040, 0, 8), (143, 1, 0)])
def test_any_alignment(M, K, pad, lead):
    """Rows that start on any byte, of any length; C's rows too."""
    gen = torch.Generator().manual_seed(K)
    groups, N = 3, 70
    A, B = _i8(gen, M, K), _i8(gen, groups, N, K)
    sa, sb = torch.rand(M, generator=gen), torch.rand(groups, N, generator=gen)
    off = offsets_like("random", groups, M, gen)
    wide = torch.zeros(M, N + 3, dtype=torch.bfloat16, device="cuda")
    for a_pad, b_pad in ((pad, pad), (-K % 16, pad), (pad, -K % 16)):
        got = dg.gemm_scaled(_padded(A, a_pad, lead if a_pad == pad else 0),
                             _padded(B, b_pad, lead if b_pad == pad else 0), sa.cuda(), sb.cuda(), wide[:, 1:N + 1],
                             offsets=torch.tensor(off, dtype=torch.int32).cuda())
        ref, tol, inside = _ref(A, B, sa, sb, torch.bfloat16, off)
        check(got.cpu()[inside], ref[inside], tol[inside])
        assert bool((wide[:, 0] == 0).all()) and bool((wide[:, N + 1:] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 4096), (13, 1001), (300, 64), (40, 20000), (5, 0)])
def test_float_operand(M, K, dtype):
    """The codes and scales are quantize_rows', bit for bit; the product is that of the definition."""
    gen = torch.Generator().manual_seed(M)
    N = 96
    x = torch.randn(M, K, generator=gen).to(DT[dtype])
    B, sb = _i8(gen, N, K), torch.rand(N, generator=gen) / 1000
    got = dg.gemm_scaled(x.cuda(), B.cuda(), None, sb.cuda())
    assert got.dtype == DT[dtype]
    q, s = dg.quantize_rows(x.cuda())
    assert same_bits(got, dg.gemm_scaled(q, B.cuda(), s, sb.cuda(), out_dtype=DT[dtype]))
    codes, scales = codes64(x)
    ref, tol, _ = _ref(codes, B, scales, sb, DT[dtype])
    check(got.cpu(), ref, tol)


@pytest.mark.parametrize("kernel", ["i8_stream_16x16", "i8_stream_16x32", "i8_stream_16x64"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_few_float_rows_need_no_workspace(dtype, kernel, monkeypatch):
    """Up to four rows and 8192 elements: one launch, the same bits as quantize_rows and
    the product, whatever K, alignment and offsets of one group."""
    monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    gen = torch.Generator().manual_seed(21)
    for M, K, N, pad in ((1, 4096, 48, 0), (1, 8192, 33, 0), (3, 1001, 70, 1), (4, 7, 100, 0), (4, 128, 20, 5),
                         (1, 130, 64, 0), (2, 4095, 17, 2), (4, 2040, 300, 8), (4, 2048, 30, 0)):
        desc = dg.make_scaled_desc(M, N, K, a_type=dtype)
        assert dg.dg_gemm_scaled_workspace_size(desc) == 0
        assert f"kernel={kernel} " in dg.dg_gemm_scaled_describe(desc)
        x = torch.zeros(M, K + pad)
        x[:, :K] = torch.randn(M, K, generator=gen)
        if M > 2:
            x[1], x[2, K // 2] = 0, float("nan")
        x = x.to(DT[dtype]).cuda()[:, :K]
        B, sb = _padded(_i8(gen, N, K), pad), torch.rand(N, generator=gen).cuda() / 100
        bias = torch.randn(N, generator=gen).cuda()
        q, s = dg.quantize_rows(x)
        for kw in ({}, dict(act="gelu_erf", bias=bias, alpha=0.5), dict(out_dtype=torch.float32)):
            got = dg.gemm_scaled(x, B, None, sb, **kw)
            want = dg.gemm_scaled(q, B, s, sb, **dict(dict(out_dtype=DT[dtype]), **kw))
            assert same_bits(got.nan_to_num(nan=5.0), want.nan_to_num(nan=5.0)), (M, K)
        for lo, hi in ((0, M), (1, M), (1, M - 1), (0, 0)):
            off = torch.tensor([lo, hi], dtype=torch.int32).cuda()
            a, b = torch.full((2, M, N), 9.0, device="cuda")
            dg.gemm_scaled(x, B[None], None, sb[None], a, offsets=off)
            dg.gemm_scaled(q, B[None], s, sb[None], b, offsets=off)
            assert same_bits(a.nan_to_num(nan=5.0), b.nan_to_num(nan=5.0)), (M, K, lo, hi)


def test_largest_sums():
    K = 131071
    for kernel_rows in (1, 300):
        A = torch.full((kernel_rows, K + 1), -128, dtype=torch.int8, device="cuda")[:, :K]
        B = torch.full((64, K + 1), -128, dtype=torch.int8, device="cuda")[:, :K]
        B[1].fill_(127)
        got = dg.gemm_scaled(A, B, out_dtype=torch.float32).cpu()
        assert bool((got[:, 0] == float(K * 16384)).all())      # 2^31 - 2^14: a fp32 value
        want = torch.tensor(-128 * 127 * K, dtype=torch.float64).float()
        assert bool((got[:, 1] == want).all())
    A, B = (torch.full((300, 131056), -128, dtype=torch.int8, device="cuda") for _ in range(2))
    assert bool((dg.gemm_scaled(A, B, out_dtype=torch.float32) == float(131056 * 16384)).all())


@pytest.mark.parametrize("kernel", KERNELS)
def test_nan_scales_stay_in_their_row_and_column(kernel, monkeypatch):
    monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    gen = torch.Generator().manual_seed(1)
    M, N, K = 140, 150, 128
    A, B = _i8(gen, M, K).cuda(), _i8(gen, N, K).cuda()
    sa, sb = torch.ones(M), torch.ones(N)
    sa[7], sb[11], sa[100] = float("nan"), float("inf"), 0.0
    got = dg.gemm_scaled(A, B, sa.cuda(), sb.cuda(), out_dtype=torch.float32).cpu()
    plain = dg.gemm_scaled(A, B, out_dtype=torch.float32).cpu()
    assert bool(got[7].isnan().all()) and bool(got[100, 11].isnan())
    rest = torch.ones(M, N, dtype=torch.bool)
    rest[7], rest[100], rest[:, 11] = False, False, False
    assert torch.equal(got[rest], plain[rest])
    assert bool((got[100, :11] == 0).all())
    big = torch.tensor([float("inf"), 3.0, float("nan")]).repeat(2)[:, None] * torch.ones(1, 32)
    got = dg.gemm_scaled(big.cuda(), B[:, :32].contiguous(), out_dtype=torch.float32).cpu()
    assert bool(got[[0, 2, 3, 5]].isnan().all()) and bool(got[[1, 4]].isfinite().all())


@pytest.mark.parametrize("kernel", KERNELS)
def test_offsets_of_any_content(kernel, monkeypatch):
    monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    gen = torch.Generator().manual_seed(4)
    groups, M, N, K = 5, 90, 48, 64
    A, B = _i8(gen, M, K), _i8(gen, groups, N, K)
    for off in ([-5, 20, 10, 2 ** 31 - 1, 3, 7], [2 ** 31 - 1] * 6, [-2 ** 31] * 6, [50, 40, 30, 20, 60, 0]):
        C = torch.full((M, N), 3.0, device="cuda")
        dg.gemm_scaled(A.cuda(), B.cuda(), None, None, C, offsets=torch.tensor(off, dtype=torch.int32).cuda())
        ref, _, inside = _ref(A, B, None, None, torch.float32, off)
        got = C.cpu()
        assert torch.equal(got[inside], ref[inside].float()) and bool((got[~inside] == 3).all())


def test_operands_past_4_gib():
    N, K, far = 40, 256, 3_000_000_000
    flat = torch.empty(2 * far, dtype=torch.int8, device="cuda")
    B = torch.as_strided(flat, (3, N, K), (far - 2 ** 20, K, 1))
    gen = torch.Generator().manual_seed(3)
    small = _i8(gen, 3, N, K)
    B.copy_(small)
    A = _i8(gen, 30, K)
    off = [0, 10, 11, 30]
    got = dg.gemm_scaled(A.cuda(), B, offsets=torch.tensor(off, dtype=torch.int32).cuda(), out_dtype=torch.float32)
    assert torch.equal(got.cpu(), _ref(A, small, None, None, torch.float32, off)[0].float())


def test_empty_sizes():
    new = lambda *s, dt=torch.int8: torch.empty(s, dtype=dt, device="cuda")
    assert dg.gemm_scaled(new(0, 16), new(8, 16)).shape == (0, 8)
    assert dg.gemm_scaled(new(4, 16), new(0, 16)).shape == (4, 0)
    bias = torch.arange(8.0, device="cuda")
    got = dg.gemm_scaled(new(4, 0), new(8, 0), bias=bias, out_dtype=torch.float32)
    assert torch.equal(got, bias.expand(4, 8))
    assert torch.equal(dg.gemm_scaled(new(4, 0, dt=torch.float32), new(8, 0), bias=bias), bias.expand(4, 8))


def test_other_stream_and_explicit_stream():
    gen = torch.Generator().manual_seed(9)
    x = torch.randn(200, 512, generator=gen).bfloat16().cuda()
    B, sb = _i8(gen, 300, 512).cuda(), torch.rand(300, generator=gen).cuda()
    want = dg.gemm_scaled(x, B, None, sb)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        here = dg.gemm_scaled(x, B, None, sb)
    there = [dg.gemm_scaled(x, B, None, sb, stream=side.cuda_stream) for _ in range(4)]
    torch.cuda.synchronize()
    for got in [here] + there:
        assert same_bits(got, want)


def test_8_bit_layer_of_experts_captured():
    """dispatch -> codes at their places -> two grouped products -> combine, eager
    and as two graphs replayed on new inputs and routing in turn."""
    gen = torch.Generator().manual_seed(12)
    tokens, top_k, groups, D, H = 50, 2, 6, 192, 320
    x = torch.randn(tokens, D, generator=gen).bfloat16().cuda()
    index = torch.randint(0, groups, (tokens, top_k), generator=gen).cuda()
    w = torch.rand(tokens, top_k, generator=gen).cuda()
    W1, W2 = _i8(gen, groups, H, D).cuda(), _i8(gen, groups, D, H).cuda()
    s1, s2 = (torch.rand(groups, n, generator=gen).cuda() / 1000 for n in (H, D))

    def layer():
        off, _, place = dg.sort_tokens(index, groups)
        q, s = dg.quantize_rows(x, place)
        h = dg.gemm_scaled(q, W1, s, s1, offsets=off, act="gelu_tanh")
        return off, place, h, dg.combine_tokens(dg.gemm_scaled(h, W2, None, s2, offsets=off), place, w)

    off, place, h, y = layer()
    codes, scales = codes64(x.cpu())
    src = torch.empty(tokens * top_k, dtype=torch.long)
    src[place.cpu().reshape(-1).long()] = torch.arange(tokens * top_k) // top_k
    ref, tol, _ = _ref(codes[src], W1.cpu(), scales[src], s1.cpu(), torch.bfloat16, off.tolist(), act="gelu_tanh")
    check(h.cpu(), ref, tol, "first product")
    codes, scales = codes64(h.cpu())
    z, ztol, _ = _ref(codes, W2.cpu(), scales, s2.cpu(), torch.bfloat16, off.tolist())
    p = place.cpu().long()
    want = (z[p] * w.cpu().double()[..., None]).sum(1)
    slack = (ztol[p] * w.cpu().double()[..., None]).sum(1) + (2.0 ** -8 + 2.0 ** -20) * want.abs() + 2.0 ** -20
    assert bool(((y.cpu().double() - want).abs() <= slack * 1.01).all())

    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer()
        graphs.append((graph, out))
    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        index.copy_(torch.randint(0, groups, (tokens, top_k), generator=g))
        x.copy_(torch.randn(tokens, D, generator=g).bfloat16())
        for graph, _ in graphs:
            graph.replay()
        for a in layer():
            pass
        for graph, out in graphs:
            for a, b in zip(out, layer()):
                assert same_bits(a, b)
        torch.cuda.synchronize()


def test_explicit_stream_leaves_the_current_streams_memory_alone():
    """With stream=, what the call allocates must not be a block that the
    current stream freed while work on it is still pending there."""
    M, N, K = 512, 256, 4096
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(M, K, device="cuda", generator=gen).bfloat16()
    B = torch.randint(-127, 128, (N, K), device="cuda", generator=gen, dtype=torch.int8)
    sb = torch.rand(N, device="cuda", generator=gen)
    at = torch.randint(0, 8, (M, 2), device="cuda", generator=gen)
    want = dg.gemm_scaled(x, B, None, sb)
    ones = torch.ones(M, 2, device="cuda")
    side = torch.cuda.Stream()
    sizes = (M * (K + 4), M * N * 2, 2 * M * K * 2, 2 * M * 4, M * K)     # workspace, C, rows, maps, codes
    torch.cuda.synchronize()
    freed = [torch.full((n,), 85, dtype=torch.uint8, device="cuda") for n in sizes]
    spans = [(f.data_ptr(), f.data_ptr() + n) for f, n in zip(freed, sizes)]
    kept = [torch.empty_like(f) for f in freed]
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(20_000_000)
    for k, f in zip(kept, freed):
        k.copy_(f)
    freed = f = None
    got = dg.gemm_scaled(x, B, None, sb, stream=side.cuda_stream)
    rows, offsets, order, place = dg.dispatch_tokens(x, at, 8, stream=side.cuda_stream)
    q, s = dg.quantize_rows(x, stream=side.cuda_stream)
    y = dg.combine_tokens(rows, place, stream=side.cuda_stream)
    dz, dw = dg.combine_tokens_grad(x, rows, place, ones, stream=side.cuda_stream)
    maps = dg.sort_tokens(at, 8, stream=side.cuda_stream)
    spread = dg.spread_tokens(x, place, stream=side.cuda_stream)
    torch.cuda.synchronize()
    for t in (got, rows, offsets, order, place, q, s, y, dz, dw, *maps, spread):
        assert not any(lo <= t.data_ptr() < hi for lo, hi in spans)
    for k in kept:
        assert bool((k == 85).all())
    assert torch.equal(got, want)
    assert torch.equal(spread, rows)
    assert all(torch.equal(a, b) for a, b in zip(maps, (offsets, order, place)))
