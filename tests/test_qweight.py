"""dg_gemm_qweight on the GPU against its definition in fp64, and a run of
the expert products as a layer uses them: trained with the grouped products,
served from 4-bit weights."""
import pytest
import torch

import dense_gemm_10_amd as dg
from grouped_util import DT, check, finish, groups_of, ints, offsets_like, sum_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _pack(q):
    if q.shape[-1] % 2:
        q = torch.cat([q, torch.zeros_like(q[..., :1])], -1)
    return q[..., 0::2] | (q[..., 1::2] << 4)


def _weights(q, scales, zeros, g):
    at = torch.arange(q.shape[-1]) // g
    zero = 8.0 if zeros is None else zeros.double()[..., at]
    return (q.double() - zero) * scales.double()[..., at]


def _make(gen, lead, N, K, g, scale_dtype, with_zeros, exact):
    q = torch.randint(0, 16, (*lead, N, K), generator=gen, dtype=torch.uint8)
    S = -(-K // g)
    if exact:                                            # powers of two
        scales = 2.0 ** torch.randint(-2, 2, (*lead, N, S), generator=gen)
    else:
        scales = (0.5 + torch.rand(*lead, N, S, generator=gen)) / K ** 0.5
    zeros = torch.randint(0, 16, (*lead, N, S), generator=gen, dtype=torch.uint8) if with_zeros else None
    return q, scales.to(scale_dtype), zeros


def _dev(t):
    return None if t is None else t.cuda()


def _offsets(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# M, N, K, group size: one row, odd rows and columns, around the tiles, K of
# no whole step, last group shorter
SIZES = [(1, 16, 32, 32), (1, 40, 256, 128), (3, 17, 96, 32), (13, 129, 544, 32), (16, 64, 192, 64),
         (17, 72, 640, 128), (33, 264, 512, 256), (65, 100, 1024, 64), (130, 136, 256, 128),
         (300, 520, 384, 128), (5, 33, 100, 32), (2, 20, 77, 64), (4, 24, 1, 32), (7, 48, 160, 64),
         (1, 1, 128, 128), (260, 33, 96, 96)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("with_zeros", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_integer_products_are_exact(size, with_zeros, dtype):
    M, N, K, g = size
    gen = torch.Generator().manual_seed(M + N + K)
    q, scales, zeros = _make(gen, (), N, K, g, DT[dtype], with_zeros, True)
    A = ints(gen, M, K, dtype=DT[dtype])
    got = dg.gemm_qweight(A.cuda(), _pack(q).cuda(), scales.cuda(), _dev(zeros), group_size=g,
                          out_dtype=torch.float32)
    ref = A.double() @ _weights(q, scales, zeros, g).t()
    assert torch.equal(got.cpu().double(), ref)


def _error(A, q, scales, zeros, g, K):
    """Bound of the fp32 error of one product (grouped_util), and the
    product's own terms."""
    at = torch.arange(K) // g
    s = scales.double()[..., at]
    mag = A.double().abs() @ (62 * s).t()
    return (K + K // g + 8) * 2.0 ** -23 * mag


@pytest.mark.parametrize("dtype,out,scale", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"),
                                             ("f16", "f16", "f16"), ("f16", "bf16", "f32")])
@pytest.mark.parametrize("size", [(1, 264, 512, 128), (5, 100, 160, 32), (40, 72, 256, 64),
                                  (200, 136, 256, 128), (3, 50, 99, 32)], ids=str)
def test_epilogue(size, dtype, out, scale):
    M, N, K, g = size
    gen = torch.Generator().manual_seed(1)
    q, scales, zeros = _make(gen, (), N, K, g, DT[scale], True, False)
    A, C0 = torch.randn(M, K, generator=gen).to(DT[dtype]), torch.randn(M, N, generator=gen).to(DT[out])
    bias = torch.randn(N, generator=gen).to(DT[dtype])
    y, err = A.double() @ _weights(q, scales, zeros, g).t(), _error(A, q, scales, zeros, g, K)
    for alpha, beta, b, act in ((1.0, 0.0, None, "none"), (0.5, 1.0, bias, "gelu_erf"),
                                (1.0, -2.0, bias, "gelu_tanh"), (0.0, 1.0, None, "none")):
        C = C0.cuda()
        dg.gemm_qweight(A.cuda(), _pack(q).cuda(), scales.cuda(), zeros.cuda(), C, group_size=g,
                        alpha=alpha, beta=beta, bias=_dev(b), act=act)
        ref, tol = finish(y, None, err, DT[out], alpha=alpha, beta=beta, C=C0, bias=b, act=act)
        check(C, ref, tol, f"{alpha} {beta} {act}")


# groups, rows, N, K, group size
EXPERTS = [(4, 9, 40, 128, 32), (9, 30, 72, 256, 128), (70, 40, 24, 64, 64), (3, 300, 136, 512, 128),
           (2, 100, 33, 96, 32), (5, 50, 20, 70, 32), (6, 900, 264, 256, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("with_zeros", [False, True])
@pytest.mark.parametrize("size", EXPERTS, ids=str)
def test_experts_exact(size, with_zeros, dtype):
    groups, rows, N, K, g = size
    gen = torch.Generator().manual_seed(rows)
    q, scales, zeros = _make(gen, (groups,), N, K, g, DT[dtype], with_zeros, True)
    A, bias = ints(gen, rows, K, dtype=DT[dtype]), ints(gen, groups, N)
    W = _weights(q, scales, zeros, g)
    for pattern in ("random", "one", "edges", "none"):
        off = offsets_like(pattern, groups, rows, gen)
        C = torch.full((rows, N), float("nan"), device="cuda")
        dg.gemm_qweight(A.cuda(), _pack(q).cuda(), scales.cuda(), _dev(zeros), C, group_size=g,
                        offsets=_offsets(off), bias=bias.cuda())
        got, inside = C.cpu().double(), torch.zeros(rows, dtype=torch.bool)
        for e, (lo, hi) in enumerate(groups_of(off, rows)):
            assert torch.equal(got[lo:hi], A[lo:hi].double() @ W[e].t() + bias[e].double()), (pattern, e)
            inside[lo:hi] = True
        assert bool(got[~inside].isnan().all()), pattern


@pytest.mark.parametrize("values", [[5, 3, 9, 2, 40], [-7, -1, 2, 2 ** 31 - 1, 0], [50, 0, 10, 60, 61]],
                         ids=str)
def test_any_offsets_stay_inside(values):
    gen = torch.Generator().manual_seed(3)
    rows, K, N, groups, g = 60, 64, 72, 4, 32
    q, scales, _ = _make(gen, (groups,), N, K, g, torch.float32, False, True)
    A, W = ints(gen, rows, K, dtype=torch.bfloat16), _weights(q, scales, None, g)
    C = torch.full((rows, N), 7.0, device="cuda")
    dg.gemm_qweight(A.cuda(), _pack(q).cuda(), scales.cuda(), None, C, group_size=g,
                    offsets=_offsets(values))
    ref = torch.full((rows, N), 7.0, dtype=torch.float64)
    for e, (lo, hi) in enumerate(groups_of(values, rows)):
        ref[lo:hi] = A[lo:hi].double() @ W[e].t()
    assert torch.equal(C.cpu().double(), ref)


@pytest.mark.parametrize("M", [1, 20, 150])
@pytest.mark.parametrize("first,pad", [(0, 16), (1, 0), (3, 5)])
def test_strides_and_alignment(M, first, pad):
    """Rows of every operand with padding, and starts off the 16-byte grid."""
    gen = torch.Generator().manual_seed(M)
    N, K, g = 40, 256, 64

    def wide(t):
        full = torch.zeros(*t.shape[:-1], t.shape[-1] + first + pad, dtype=t.dtype, device="cuda")
        part = full[..., first:first + t.shape[-1]]
        part.copy_(t)
        return part

    q, scales, zeros = _make(gen, (), N, K, g, torch.bfloat16, True, True)
    A = ints(gen, M, K, dtype=torch.bfloat16)
    full = torch.full((M, N + first + pad), 3.0, device="cuda")
    C = full[:, first:first + N]
    dg.gemm_qweight(wide(A), wide(_pack(q)), wide(scales), wide(zeros), C, group_size=g)
    assert torch.equal(C.cpu().double(), A.double() @ _weights(q, scales, zeros, g).t())
    assert bool((full[:, :first] == 3.0).all()) and bool((full[:, first + N:] == 3.0).all())


@pytest.mark.parametrize("M", [3, 40])
def test_nan_rows_and_scales_stay_where_they_are(M):
    gen = torch.Generator().manual_seed(0)
    N, K, g = 48, 128, 32
    q, scales, _ = _make(gen, (), N, K, g, torch.float32, False, True)
    A = ints(gen, M, K, dtype=torch.bfloat16)
    ref = A.double() @ _weights(q, scales, None, g).t()
    A[1, 5] = float("nan")
    scales[7, 2] = float("inf")
    got = dg.gemm_qweight(A.cuda(), _pack(q).cuda(), scales.cuda(), group_size=g,
                          out_dtype=torch.float32).cpu().double()
    keep = torch.ones(M, N, dtype=torch.bool)
    keep[1], keep[:, 7] = False, False
    assert torch.equal(got[keep], ref[keep])
    assert not bool(got[1].isfinite().any()) and not bool(got[0, 7].isfinite())


@pytest.mark.parametrize("kernel", ["qstream_16x16", "qstream_16x32", "qstream_16x64", "qstream_32x32",
                                    "qstream_32x64", "qstream_32x128", "qtile_64x256", "qtile_64x512"])
def test_every_kernel(kernel, monkeypatch):
    """The kernel depends on the sizes alone; each is right for any rows,
    columns, K, group size and lengths."""
    monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    gen = torch.Generator().manual_seed(17)
    for M, N, K, g, dt, with_zeros in ((1, 300, 4384, 128, torch.bfloat16, False), (70, 130, 288, 96, torch.float16, True),
                                       (33, 16, 64, 64, torch.bfloat16, True), (130, 520, 1056, 32, torch.float16, False),
                                       (130, 1040, 1056, 256, torch.bfloat16, True)):
        q, scales, zeros = _make(gen, (), N, K, g, dt, with_zeros, True)
        A = ints(gen, M, K, dtype=dt)
        got = dg.gemm_qweight(A.cuda(), _pack(q).cuda(), scales.cuda(), _dev(zeros), group_size=g,
                              out_dtype=torch.float32)
        assert torch.equal(got.cpu().double(), A.double() @ _weights(q, scales, zeros, g).t()), (M, N, K)
    groups, rows, N, K, g = 70, 300, 72, 192, 128 if kernel == "qtile_64x512" else 64
    q, scales, zeros = _make(gen, (groups,), N, K, g, torch.bfloat16, True, True)
    A, W = ints(gen, rows, K, dtype=torch.bfloat16), _weights(q, scales, zeros, g)
    for pattern in ("random", "one", "edges"):
        off = offsets_like(pattern, groups, rows, gen)
        C = torch.full((rows, N), 5.0, device="cuda")
        dg.gemm_qweight(A.cuda(), _pack(q).cuda(), scales.cuda(), zeros.cuda(), C, group_size=g,
                        offsets=_offsets(off))
        ref = torch.full((rows, N), 5.0, dtype=torch.float64)
        for e, (lo, hi) in enumerate(groups_of(off, rows)):
            ref[lo:hi] = A[lo:hi].double() @ W[e].t()
        assert torch.equal(C.cpu().double(), ref), pattern


@pytest.mark.parametrize("kernel", ["qstream_32x128", "qtile_64x256", "qtile_64x512"])
@pytest.mark.parametrize("out,scale", [("bf16", "f32"), ("f16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("first,pad", [(0, 2), (4, 2), (2, 0), (1, 3), (0, 1)])
def test_output_at_any_alignment(kernel, out, scale, first, pad, monkeypatch):
    """C a part of a wider matrix: rows on four columns or not; nothing
    beside it is written."""
    monkeypatch.setenv("DG_FORCE_GROUPED", kernel)
    gen = torch.Generator().manual_seed(first + pad)
    M, N, K, g = 75, 522, 416, 128
    q, scales, zeros = _make(gen, (), N, K, g, DT[scale], True, False)
    A, bias = torch.randn(M, K, generator=gen).bfloat16(), torch.randn(N, generator=gen).bfloat16()
    y, err = A.double() @ _weights(q, scales, zeros, g).t(), _error(A, q, scales, zeros, g, K)
    wide = torch.randn(M, first + N + pad, generator=gen).to(DT[out])
    for beta, b, act in ((0.0, None, "none"), (1.0, bias, "gelu_erf")):
        W = wide.cuda()
        C = W[:, first:first + N]
        dg.gemm_qweight(A.cuda(), _pack(q).cuda(), scales.cuda(), zeros.cuda(), C, group_size=g,
                        beta=beta, bias=_dev(b), act=act)
        ref, tol = finish(y, None, err, DT[out], beta=beta, C=wide[:, first:first + N], bias=b, act=act)
        check(C, ref, tol, f"{beta} {act}")
        assert torch.equal(W[:, :first].cpu(), wide[:, :first])
        assert torch.equal(W[:, first + N:].cpu(), wide[:, first + N:])


def test_empty_sizes():
    def z(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    C = torch.full((2, 3), 4.0, device="cuda")
    dg.gemm_qweight(z(2, 0), z(3, 0, dtype=torch.uint8), z(3, 0), None, C, group_size=32, beta=0.5,
                    bias=torch.tensor([1.0, 2.0, 3.0], device="cuda"))
    assert C.tolist() == [[3.0, 4.0, 5.0]] * 2
    assert dg.gemm_qweight(z(0, 64), z(3, 32, dtype=torch.uint8), z(3, 2), group_size=32).shape == (0, 3)
    assert dg.gemm_qweight(z(2, 64), z(0, 32, dtype=torch.uint8), z(0, 2), group_size=32).shape == (2, 0)
    dg.gemm_qweight(z(2, 64), z(0, 3, 32, dtype=torch.uint8), z(0, 3, 2), None, C, group_size=32,
                    offsets=_offsets([0]))
    assert C.tolist() == [[3.0, 4.0, 5.0]] * 2


def test_runs_repeat_bit_for_bit():
    gen = torch.Generator().manual_seed(6)
    for M, N, K, g in ((1, 264, 4352, 128), (40, 520, 1024, 32), (700, 264, 512, 64)):
        q, scales, zeros = _make(gen, (), N, K, g, torch.bfloat16, True, False)
        A = torch.randn(M, K, generator=gen).bfloat16().cuda()
        args = A, _pack(q).cuda(), scales.cuda(), zeros.cuda()
        first = dg.gemm_qweight(*args, group_size=g)
        for _ in range(5):
            assert torch.equal(dg.gemm_qweight(*args, group_size=g), first)


@pytest.mark.parametrize("size", [(600, 2000, 288, 96), (1024, 1040, 512, 128), (2050, 264, 160, 32)], ids=str)
def test_many_rows(size):
    """Sizes that the 64 x 256 tile takes, and its edges."""
    M, N, K, g = size
    gen = torch.Generator().manual_seed(M)
    q, scales, zeros = _make(gen, (), N, K, g, torch.float16, True, True)
    A = ints(gen, M, K, dtype=torch.float16)
    got = dg.gemm_qweight(A.cuda(), _pack(q).cuda(), scales.cuda(), zeros.cuda(), group_size=g,
                          out_dtype=torch.float32)
    assert torch.equal(got.cpu().double(), A.double() @ _weights(q, scales, zeros, g).t())


def test_weights_past_2_31_bytes():
    gen = torch.Generator(device="cuda").manual_seed(1)
    N, K, g, groups = 4096, 8192, 128, 130                       # 2.18e9 bytes of Q
    Q = torch.zeros(groups, N, K // 2, dtype=torch.uint8, device="cuda")
    Q[-1] = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.ones(groups, N, K // g, dtype=torch.bfloat16, device="cuda")
    A = torch.randint(-2, 3, (5, K), generator=gen, device="cuda").bfloat16()
    C = dg.gemm_qweight(A, Q, scales, group_size=g, offsets=_offsets([0] * 130 + [5]),
                        out_dtype=torch.float32)
    w = torch.empty(N, K, dtype=torch.float64, device="cuda")
    w[:, 0::2], w[:, 1::2] = (Q[-1] & 15).double() - 8, (Q[-1] >> 4).double() - 8
    assert torch.equal(C.double(), A.double() @ w.t())


def test_graph_and_streams():
    gen = torch.Generator().manual_seed(9)
    N, K, g, groups, rows = 72, 256, 64, 5, 37
    q, scales, zeros = _make(gen, (groups,), N, K, g, torch.float16, True, True)
    A, Q, S, Z = ints(gen, rows, K, dtype=torch.float16).cuda(), _pack(q).cuda(), scales.cuda(), zeros.cuda()
    W = _weights(q, scales, zeros, g)
    off, C, one = _offsets([0] * 6), torch.zeros(rows, N, device="cuda"), torch.zeros(1, N, device="cuda")

    def step():
        dg.gemm_qweight(A, Q, S, Z, C, group_size=g, offsets=off)
        dg.gemm_qweight(A[:1], Q[2], S[2], Z[2], one, group_size=g)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for pattern in ("random", "edges", "one", "random"):
        values = offsets_like(pattern, groups, rows, gen)
        off.copy_(_offsets(values))
        C.fill_(-1.0), one.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        got = C.cpu().double()
        for e, (lo, hi) in enumerate(groups_of(values, rows)):
            assert torch.equal(got[lo:hi], A[lo:hi].cpu().double() @ W[e].t())
        assert torch.equal(one.cpu().double(), A[:1].cpu().double() @ W[2].t())
        step()                                                   # eager work between the replays
        torch.cuda.synchronize()
        assert torch.equal(C.cpu().double(), got)


def _quantise(W, g):
    """Symmetric 4-bit codes of W (..., N, K): scale = max |w| / 7 per group."""
    w = W.unflatten(-1, (-1, g))
    scale = (w.abs().amax(-1) / 7).clamp(min=1e-8).bfloat16()
    q = (w / scale.float()[..., None]).round().clamp(-8, 7) + 8
    return q.flatten(-2).to(torch.uint8), scale


def test_an_expert_layer_trained_and_served():
    """Forward (bias, GELU), input and weight gradients of a two-product
    expert layer in bf16, one step on fp32 weights, 4-bit codes of the result,
    and one generation step from the codes: every product against fp64 on the
    values it was given."""
    gen = torch.Generator().manual_seed(12)
    E, rows, D, H, g = 6, 330, 128, 264, 32
    off = offsets_like("random", E, rows, gen)
    o, spans = _offsets(off), groups_of(off, rows)
    X = torch.randn(rows, D, generator=gen).bfloat16()
    W1 = torch.randn(E, D, H, generator=gen) / D ** 0.5
    W2 = torch.randn(E, H, D, generator=gen) / H ** 0.5
    b1 = torch.randn(E, H, generator=gen) * 0.1

    def each(A, B):
        return torch.cat([A[lo:hi].double() @ B[e].double() for e, (lo, hi) in enumerate(spans)])

    def tol_of(A, B):
        mag = torch.cat([A[lo:hi].double().abs() @ B[e].double().abs() for e, (lo, hi) in enumerate(spans)])
        return sum_error(A.shape[1], mag)

    by_row = torch.cat([torch.full((hi - lo,), e) for e, (lo, hi) in enumerate(spans)]).long()
    w1, w2 = W1.bfloat16(), W2.bfloat16()
    Xd, w1d, w2d = X.cuda(), w1.cuda(), w2.cuda()
    h = dg.gemm_grouped(Xd, w1d, o, bias=b1.cuda(), act="gelu_tanh")
    ref, tol = finish(each(X, w1), None, tol_of(X, w1), torch.bfloat16, bias=b1[by_row], act="gelu_tanh")
    check(h, ref, tol, "first product")
    y = dg.gemm_grouped(h, w2d, o)
    hc = h.cpu()
    check(y, *finish(each(hc, w2), None, tol_of(hc, w2), torch.bfloat16), "second product")
    dy = y                                                       # of L = sum(y^2) / 2
    dh = dg.gemm_grouped(dy, w2d.transpose(1, 2), o)
    dc, w2t = dy.cpu(), w2.transpose(1, 2)
    check(dh, *finish(each(dc, w2t), None, tol_of(dc, w2t), torch.bfloat16), "input gradient")
    dW2 = dg.gemm_grouped_k(h.t(), dy, o, out_dtype=torch.float32)
    for e, (lo, hi) in enumerate(spans):
        a, b = hc[lo:hi].double().t(), dc[lo:hi].double()
        check(dW2[e], *finish(a @ b, None, sum_error(hi - lo, a.abs() @ b.abs()), torch.float32), f"dW2 {e}")
    W2 = W2 - 0.01 * dW2.cpu()
    q, scale = _quantise(W2.transpose(1, 2).contiguous()[..., :256], g)      # (E, D, 256)
    step = hc[:9, :256].contiguous()
    off9 = [min(v, 9) for v in off]
    got = dg.gemm_qweight(step.cuda(), _pack(q).cuda(), scale.cuda(), group_size=g, offsets=_offsets(off9),
                          out_dtype=torch.float32)
    W4 = _weights(q, scale, None, g)
    for e, (lo, hi) in enumerate(groups_of(off9, 9)):
        if hi > lo:
            ref, tol = finish(step[lo:hi].double() @ W4[e].t(), None,
                              _error(step[lo:hi], q[e], scale[e], None, g, 256), torch.float32)
            check(got[lo:hi], ref, tol, f"expert {e}")
