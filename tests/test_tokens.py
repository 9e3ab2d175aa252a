"""Tokens sorted by group and back, and 8-bit codes, on the GPU against plain
forms: maps and copies exactly, sums and gradients in fp64 and by differences,
strides, empty sizes, places of any content, streams and graphs."""
import pytest
import torch

import dense_gemm_10_amd as dg
from tokens_util import DT, codes64, combine64, maps, random_index, rounded, same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# tokens, top_k, groups: both sides of a wavefront, a workgroup, the launch for
# few slots and a round of the sort; one group, more groups than slots, no top_k
MAPS = [(1, 1, 1), (1, 2, 64), (16, 2, 64), (7, 5, 3), (64, 1, 2), (65, 1, 8), (128, 8, 16), (257, 4, 300),
        (512, 2, 17), (1025, 1, 5), (1000, 8, 512), (3000, 6, 1), (4097, 3, 8192), (20000, 2, 24), (140000, 2, 60),
        (5, 0, 4), (0, 3, 4), (9, 2, 0)]


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64], ids=["i32", "i64"])
@pytest.mark.parametrize("size", MAPS, ids=str)
def test_maps(size, dtype):
    tokens, top_k, groups = size
    gen = torch.Generator().manual_seed(tokens + groups)
    for drop in (0.0, 0.3):
        index = random_index(tokens, top_k, groups, gen, drop, dtype)
        want = maps(index, groups)
        for got, ref in zip(dg.sort_tokens(index.cuda(), groups), want):
            assert torch.equal(got.cpu(), ref)
        x = torch.randn(tokens, 24, generator=gen).bfloat16()
        out = torch.full((tokens * top_k, 24), 5.0).bfloat16()
        rows, *got = dg.dispatch_tokens(x.cuda(), index.cuda(), groups, out=out.cuda())
        for g, ref in zip(got, want):
            assert torch.equal(g.cpu(), ref)
        kept = want[1] >= 0
        out[kept] = x[want[1][kept].long() // max(top_k, 1)]
        assert same_bits(rows, out)


@pytest.mark.parametrize("size", [(40, 2, 9), (600, 3, 9)], ids=str)
def test_index_values_outside_the_groups(size):
    """Any 32- or 64-bit value names a group or none; strided index tensors."""
    tokens, top_k, groups = size
    gen = torch.Generator().manual_seed(3)
    for dtype, extremes in ((torch.int32, (-1, -2 ** 31, 2 ** 31 - 1, groups)),
                            (torch.int64, (-1, -2 ** 63, 2 ** 63 - 1, 2 ** 32, 2 ** 32 + 1, groups))):
        wide = random_index(tokens, top_k + 2, groups, gen, dtype=dtype)
        for i, v in enumerate(extremes):
            wide[i::11] = v
        index = wide.cuda()[:, :top_k]
        assert not index.is_contiguous()
        want = maps(wide[:, :top_k], groups)
        for got, ref in zip(dg.sort_tokens(index, groups), want):
            assert torch.equal(got.cpu(), ref)
        x = torch.randn(tokens, 8, generator=gen)
        rows, _, order, _ = dg.dispatch_tokens(x.cuda(), index, groups)
        kept = want[1] >= 0
        assert torch.equal(rows.cpu()[kept], x[want[1][kept].long() // top_k])


# rows of no whole number of 16-byte pieces, rows at any element, long rows
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("width,pad", [(1, 0), (7, 2), (8, 0), (129, 3), (1037, 0), (4096, 8), (20003, 1), (0, 4)])
@pytest.mark.parametrize("tokens", [6, 700])
def test_rows_are_copied_bit_for_bit(tokens, width, pad, dtype):
    gen = torch.Generator().manual_seed(width)
    groups, top_k = 5, 2
    wide = torch.randint(-2 ** 15, 2 ** 15, (tokens, width + pad, 2), generator=gen).to(torch.int16)
    wide = (wide.view(torch.int32).squeeze(-1).view(torch.float32) if dtype == "f32"
            else wide[..., 0].contiguous().view(DT[dtype]))               # NaN patterns among them
    x = wide.cuda()[:, :width]
    index = random_index(tokens, top_k, groups, gen, 0.2)
    out = torch.zeros(tokens * top_k, width + pad, dtype=DT[dtype])
    ref, got = out.clone(), out.cuda()
    rows, offsets, order, place = dg.dispatch_tokens(x, index.cuda(), groups, out=got[:, :width])
    _, want, _ = maps(index, groups)
    kept = want >= 0
    ref[kept, :width] = wide[want[kept].long() // top_k, :width]
    assert same_bits(got, ref)                                            # the padding too
    again = torch.zeros_like(got)
    dg.spread_tokens(x, place, out=again[:, :width])
    assert same_bits(again, ref)


def _combine_case(tokens, top_k, width, dtype, gen, drop=0.2, extra=3):
    rows = tokens * top_k + extra
    place = torch.randperm(rows, generator=gen)[:tokens * top_k].view(tokens, top_k).to(torch.int32)
    place[torch.rand(tokens, top_k, generator=gen) < drop] = -1
    z = torch.randn(rows, width, generator=gen).to(DT[dtype])
    w = torch.rand(tokens, top_k, generator=gen)
    return z, place, w


# one row to more than the eight that are loaded at once; widths around pieces and segments
SIZES = [(1, 1, 8), (3, 2, 1), (5, 3, 129), (33, 4, 1000), (4, 8, 1037), (9, 9, 520), (2, 19, 40), (70, 2, 4096),
         (2, 6, 9001)]


@pytest.mark.parametrize("dtype,out,wt", [("bf16", "bf16", "f32"), ("bf16", "f32", "bf16"), ("f16", "f16", "f16"),
                                          ("f16", "f32", "f32"), ("f32", "f32", "f32"), ("f32", "f32", "bf16")])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_combine(size, dtype, out, wt):
    tokens, top_k, width = size
    gen = torch.Generator().manual_seed(width)
    z, place, w = _combine_case(tokens, top_k, width, dtype, gen)
    w = w.to(DT[wt])
    y0 = torch.randn(tokens, width, generator=gen).to(DT[out])
    for weights, beta in ((w, 0.0), (None, 0.0), (w, -1.5)):
        y = y0.cuda()
        got = dg.combine_tokens(z.cuda(), place.cuda(), None if weights is None else weights.cuda(), y, beta=beta)
        assert got is y
        ref, mag = combine64(z, place, weights, y0 if beta else None, beta)
        tol = rounded(ref, (top_k + 2) * 2.0 ** -23 * mag, DT[out])
        assert bool(((got.cpu().double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("dtype,gt,wt", [("bf16", "bf16", "f32"), ("bf16", "f32", "bf16"), ("f16", "f16", "f16"),
                                         ("f16", "f32", "f32"), ("f32", "f32", "f32")])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_combine_grad(size, dtype, gt, wt):
    tokens, top_k, width = size
    gen = torch.Generator().manual_seed(width + 1)
    z, place, w = _combine_case(tokens, top_k, width, dtype, gen)
    w = w.to(DT[wt])
    dy = torch.randn(tokens, width, generator=gen).to(DT[gt])
    dz = torch.full_like(z, 7.0).cuda()
    got_z, got_w = dg.combine_tokens_grad(dy.cuda(), z.cuda(), place.cuda(), w.cuda(), dz=dz)
    assert got_z is dz and got_w.dtype == DT[wt]
    ref_z = torch.full(z.shape, 7.0, dtype=torch.float64)
    err_z = torch.zeros_like(ref_z)
    ref_w, mag_w = torch.zeros(tokens, top_k, dtype=torch.float64), torch.zeros(tokens, top_k, dtype=torch.float64)
    for t in range(tokens):
        for j in range(top_k):
            p = int(place[t, j])
            if p < 0:
                continue
            ref_z[p] = float(w[t, j]) * dy[t].double()
            err_z[p] = 2.0 ** -24 * ref_z[p].abs()
            v = dy[t].double() * z[p].double()
            ref_w[t, j], mag_w[t, j] = v.sum(), v.abs().sum()
    assert bool(((got_z.cpu().double() - ref_z).abs() <= rounded(ref_z, err_z, DT[dtype])).all())
    tol = rounded(ref_w, (width + 8) * 2.0 ** -23 * mag_w, DT[wt])
    assert bool(((got_w.cpu().double() - ref_w).abs() <= tol).all())
    assert bool((got_w.cpu()[place < 0] == 0).all())


def test_gradients_against_differences():
    """The layer x -> dispatch -> c * rows -> combine, L = <y, v>: its gradients
    of x and of the weights against central differences.  L is quadratic in
    neither (linear in x for given weights, and the other way), so a difference
    is exact but for fp32 rounding: 64 terms of about 1 with 2^-23 each, over a
    step of 2^-3."""
    gen = torch.Generator().manual_seed(5)
    tokens, top_k, width, groups = 6, 2, 16, 3
    index = random_index(tokens, top_k, groups, gen, 0.2).cuda()
    x = torch.randn(tokens, width, generator=gen).cuda()
    w = torch.rand(tokens, top_k, generator=gen).cuda()
    v = torch.randn(tokens, width, generator=gen).cuda()
    c = torch.randn(tokens * top_k, 1, generator=gen).cuda()

    def forward(x, w):
        rows, _, _, place = dg.dispatch_tokens(x, index, groups, out=torch.zeros_like(x).repeat(top_k, 1))
        return rows * c, place

    z, place = forward(x, w)
    dz, dw = dg.combine_tokens_grad(v, z, place, w, dz=torch.zeros_like(z))
    dx = dg.combine_tokens(dz * c, place)

    def loss(x, w):
        z, place = forward(x, w)
        return float((dg.combine_tokens(z, place, w).double() * v.double()).sum())

    h = 2.0 ** -3
    for t in range(tokens):
        for leaf, grad, width_of in ((x, dx, width), (w, dw, top_k)):
            for i in range(0, width_of, 5):
                d = torch.zeros_like(leaf)
                d[t, i] = h
                a = (loss(x + d, w) if leaf is x else loss(x, w + d))
                b = (loss(x - d, w) if leaf is x else loss(x, w - d))
                scale = float((z.abs().amax() + 1) * (v.abs().amax() + 1) * 64)
                assert abs((a - b) / (2 * h) - float(grad[t, i])) <= scale * 2.0 ** -23 / h * 4


def test_places_of_any_content():
    """Rows outside the operands are skipped; equal places are read twice."""
    gen = torch.Generator().manual_seed(8)
    z = torch.randn(10, 40, generator=gen)
    place = torch.tensor([[3, 3], [-1, 10], [2 ** 31 - 1, -2 ** 31], [9, 0]], dtype=torch.int32)
    w = torch.rand(4, 2, generator=gen)
    got = dg.combine_tokens(z.cuda(), place.cuda(), w.cuda()).cpu().double()
    ref, mag = combine64(z, place, w)
    assert bool(((got - ref).abs() <= rounded(ref, 4 * 2.0 ** -23 * mag, torch.float32)).all())
    assert bool((got[1:3] == 0).all())
    place[0, 1] = 5
    dy = torch.randn(4, 40, generator=gen)
    dz, dw = dg.combine_tokens_grad(dy.cuda(), z.cuda(), place.cuda(), w.cuda(), dz=torch.zeros(10, 40).cuda())
    touched = sorted(int(p) for p in place.reshape(-1) if 0 <= p < 10)
    assert sorted(dz.abs().sum(1).nonzero().flatten().tolist()) == touched
    assert bool((dw.cpu()[1:3] == 0).all())
    out = torch.zeros(10, 40).cuda()
    dg.spread_tokens(dy.cuda(), place.cuda(), out=out)
    assert sorted(out.abs().sum(1).nonzero().flatten().tolist()) == touched
    q, s = torch.zeros(10, 40, dtype=torch.int8).cuda(), torch.full((10,), -1.0).cuda()
    dg.quantize_rows(dy.cuda(), place.cuda(), q, s)
    assert sorted((s >= 0).nonzero().flatten().tolist()) == touched


def test_nan_and_infinity_stay_where_the_formula_has_them():
    z = torch.ones(4, 16)
    z[1, 3], z[2] = float("nan"), float("inf")
    place = torch.tensor([[0, 3], [1, -1], [2, 0]], dtype=torch.int32)
    w = torch.tensor([[1.0, 2.0], [1.0, float("nan")], [0.5, 1.0]])
    y = dg.combine_tokens(z.cuda(), place.cuda(), w.cuda()).cpu()
    assert bool((y[0] == 3).all()) and bool((y[2] == float("inf")).all())
    assert y[1].isnan().nonzero().flatten().tolist() == [3] and float(y[1, 0]) == 1.0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("width", [1, 8, 15, 1000, 2048, 2049, 4096, 8191, 8192, 8200, 20000])
def test_codes_are_exact(width, dtype):
    gen = torch.Generator().manual_seed(width)
    x = torch.randn(9, width, generator=gen)
    x[1] *= 2.0 ** -130 if dtype != "f16" else 2.0 ** -20          # subnormals
    x[2] *= 2.0 ** 124 if dtype != "f16" else 2.0 ** 13
    x[3] = 0.0
    x[4, width // 2] = float("inf")
    x[5, 0] = float("nan")
    # every half integer: 127 x / max with max 127
    x[6] = torch.arange(width) % 254 / 2 - 63.5
    x[6, -1] = 127.0
    x[7] = (torch.arange(width) % 509 - 254) / 2.0 * 2.0 ** -9    # max 127: halves at 1/2 steps
    x = x.to(DT[dtype])
    wide = torch.zeros(9, width + 3, dtype=DT[dtype])
    wide[:, :width] = x
    q, s = dg.quantize_rows(wide.cuda()[:, :width])
    want_q, want_s = codes64(x)
    assert q.stride(0) % 16 == 0 and q.data_ptr() % 16 == 0
    assert torch.equal(q.cpu(), want_q)
    assert torch.equal(s.cpu().nan_to_num(nan=-1.0), want_s.nan_to_num(nan=-1.0))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_codes_next_to_a_half(dtype):
    """Quotients as close to n + 1/2 as the type has them, for many maxima."""
    eps = torch.finfo(DT[dtype]).eps
    tops = (1 + torch.arange(0, 64) * (1 / 64)).to(DT[dtype])
    n = torch.arange(0, 127).double() + 0.5
    rows = []
    for top in tops:
        mid = n * float(top) / 127
        near = mid.to(DT[dtype])
        x = torch.cat([near, (near.double() * (1 + eps)).to(DT[dtype]), (near.double() * (1 - eps)).to(DT[dtype])])
        rows.append(torch.cat([x, -x, top[None]]))
    x = torch.stack(rows)
    q, s = dg.quantize_rows(x.cuda())
    want_q, want_s = codes64(x)
    assert torch.equal(q.cpu(), want_q) and torch.equal(s.cpu(), want_s)


def test_codes_at_their_places():
    gen = torch.Generator().manual_seed(2)
    tokens, top_k, groups, width = 50, 3, 7, 300
    x = torch.randn(tokens, width, generator=gen).bfloat16()
    index = random_index(tokens, top_k, groups, gen, 0.2)
    _, _, place = dg.sort_tokens(index.cuda(), groups)
    q = torch.full((tokens * top_k + 2, width + 5), 99, dtype=torch.int8).cuda()
    s = torch.full((tokens * top_k + 2,), -1.0).cuda()
    dg.quantize_rows(x.cuda(), place, q[:, :width], s)
    codes, scales = codes64(x)
    want_q, want_s = torch.full(q.shape, 99, dtype=torch.int8), torch.full(s.shape, -1.0)
    for t in range(tokens):
        for p in place[t].tolist():
            if p >= 0:
                want_q[p, :width], want_s[p] = codes[t], scales[t]
    assert torch.equal(q.cpu(), want_q) and torch.equal(s.cpu(), want_s)


def test_empty_sizes():
    new = lambda *shape, dt=torch.float32: torch.empty(shape, dtype=dt, device="cuda")
    place = torch.zeros(3, 0, dtype=torch.int32, device="cuda")
    assert bool((dg.combine_tokens(new(5, 8), place) == 0).all())
    y = torch.ones(3, 8, device="cuda")
    assert bool((dg.combine_tokens(new(0, 8), torch.zeros(3, 2, dtype=torch.int32, device="cuda"), None, y,
                                   beta=2.0) == 2).all())
    dz, dw = dg.combine_tokens_grad(new(3, 0), new(6, 0), torch.zeros(3, 2, dtype=torch.int32, device="cuda"),
                                    new(3, 2))
    assert dz.shape == (6, 0) and bool((dw == 0).all())
    q, s = dg.quantize_rows(new(4, 0))
    assert q.shape == (4, 0) and bool((s == 0).all())
    q, s = dg.quantize_rows(new(0, 9))
    assert q.shape == (0, 9) and s.shape == (0,)
    assert dg.spread_tokens(new(0, 9), torch.zeros(0, 2, dtype=torch.int32, device="cuda")).shape == (0, 9)


def test_rows_past_4_gib():
    width, last = 1 << 16, 20000
    rows = torch.empty(last + 1, width, device="cuda")               # 5.2 GB
    rows[last] = 0
    x = torch.arange(width, dtype=torch.float32, device="cuda")[None]
    place = torch.tensor([[last]], dtype=torch.int32, device="cuda")
    dg.spread_tokens(x, place, out=rows)
    assert torch.equal(rows[last], x[0])
    assert torch.equal(dg.combine_tokens(rows, place), x)
    w = torch.ones(1, 1, device="cuda")
    dz, dw = dg.combine_tokens_grad(2 * x, rows, place, w, dz=rows.clone())
    assert torch.equal(dz[last], 2 * x[0])


@pytest.mark.parametrize("tokens", [40, 3000])
def test_streams_and_graphs(tokens):
    """The same calls on another stream, captured and replayed on new routing."""
    gen = torch.Generator().manual_seed(6)
    top_k, groups, width = 2, 8, 200
    x = torch.randn(tokens, width, generator=gen).bfloat16().cuda()
    index = random_index(tokens, top_k, groups, gen).cuda()
    w = torch.rand(tokens, top_k, generator=gen).cuda()
    dy = torch.randn(tokens, width, generator=gen).bfloat16().cuda()

    def step():
        rows, offsets, order, place = dg.dispatch_tokens(x, index, groups)
        q, s = dg.quantize_rows(x, place)
        return (rows, offsets, order, place, dg.combine_tokens(rows, place, w),
                *dg.combine_tokens_grad(dy, rows, place, w), q, s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        here = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(here, step()):
        assert same_bits(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(3):
        index.copy_(random_index(tokens, top_k, groups, torch.Generator().manual_seed(seed)))
        x.normal_()
        graph.replay()
        for a, b in zip(held, step()):
            assert same_bits(a, b)
        torch.cuda.synchronize()


def test_layer_of_experts_and_its_gradients():
    """dispatch -> grouped product -> combine and back, against fp64 autograd of
    the plain layer.  Each 16-bit rounding is off by 2^-8 at most: rows of z,
    of dz and the outputs; three of them and fp32 sums stay
    below 3.1 * 2^-8 of the sums of absolute values."""
    gen = torch.Generator().manual_seed(11)
    tokens, top_k, groups, D, H = 60, 2, 5, 64, 96
    x = torch.randn(tokens, D, generator=gen).bfloat16()
    W = (torch.randn(groups, D, H, generator=gen) / 8).bfloat16()
    index = random_index(tokens, top_k, groups, gen, 0.1)
    w = torch.rand(tokens, top_k, generator=gen)
    dy = torch.randn(tokens, H, generator=gen).bfloat16()
    xc, Wc, wc = x.cuda(), W.cuda(), w.cuda()
    rows, off, order, place = dg.dispatch_tokens(xc, index.cuda(), groups)
    z = dg.gemm_grouped(rows, Wc, off)
    y = dg.combine_tokens(z, place, wc)
    dz, dw = dg.combine_tokens_grad(dy.cuda(), z, place, wc)
    dx = dg.combine_tokens(dg.gemm_grouped(dz, Wc.transpose(1, 2), off), place)
    dW = dg.gemm_grouped_k(rows.t(), dz, off, out_dtype=torch.float32)

    x64, W64, w64 = (t.double().requires_grad_() for t in (x, W, w))
    mag = lambda t: t.abs()

    def layer(x, W, w):
        y = torch.zeros(tokens, H, dtype=torch.float64)
        parts = []
        for t in range(tokens):
            terms = [w[t, j] * (x[t] @ W[index[t, j]]) for j in range(top_k) if index[t, j] >= 0]
            parts.append(sum(terms) if terms else torch.zeros(H, dtype=torch.float64))
        return torch.stack(parts)

    ref = layer(x64, W64, w64)
    ref.backward(dy.double())
    with torch.no_grad():
        big = layer(mag(x.double()), mag(W.double()), w.double())
    xm, Wm, wm = (t.double().abs().requires_grad_() for t in (x, W, w))
    layer(xm, Wm, wm).backward(dy.double().abs())
    u = 2.0 ** -8
    for got, want, size in ((y, ref, big), (dx, x64.grad, xm.grad), (dW, W64.grad, Wm.grad), (dw, w64.grad, wm.grad)):
        err = (got.cpu().double() - want.detach()).abs()
        assert bool((err <= 3.1 * u * size.detach() + 1e-30).all())


def test_many_tokens():
    """More tokens than the launches have workgroups, slots in chunks of many rounds."""
    tokens, width, groups = 4_400_000, 8, 40
    gen = torch.Generator(device="cuda").manual_seed(3)
    index = torch.randint(-1, groups, (tokens, 1), device="cuda", generator=gen)
    x = torch.randn(tokens, width, device="cuda", generator=gen).bfloat16()
    rows, off, order, place = dg.dispatch_tokens(x, index, groups, out=torch.zeros_like(x))
    key = torch.where(index[:, 0] < 0, groups, index[:, 0])
    want = torch.sort(key, stable=True).indices
    n = int((index >= 0).sum())
    assert int(off[groups]) == n and torch.equal(order[:n].long(), want[:n]) and bool((order[n:] == -1).all())
    assert torch.equal(off.long()[1:], torch.bincount(key, minlength=groups + 1)[:groups].cumsum(0))
    assert torch.equal(rows[:n], x[want[:n]]) and bool((rows[n:] == 0).all())
    kept = (index >= 0).expand_as(x)
    assert torch.equal(dg.combine_tokens(rows, place), torch.where(kept, x, 0))
    w = torch.full((tokens, 1), 2.0, device="cuda")
    dz, dw = dg.combine_tokens_grad(x, rows, place, w, dz=torch.zeros_like(x))
    assert torch.equal(dz, 2 * rows)
    norm = torch.where(kept, x, 0).double().square().sum(1, keepdim=True)
    assert bool(((dw.double() - norm).abs() <= 16 * 2.0 ** -23 * norm).all())
    q, s = dg.quantize_rows(x, place, torch.zeros(tokens, width, dtype=torch.int8, device="cuda"),
                            torch.zeros(tokens, device="cuda"))
    top = rows.double().abs().amax(1, keepdim=True)
    codes = torch.where(top > 0, 127 * rows.double() / top, 0.0).round()
    assert torch.equal(q, codes.to(torch.int8)) and torch.equal(s, (top[:, 0] / 127).float())


def test_two_streams_at_once():
    gen = torch.Generator().manual_seed(13)
    tokens, top_k, groups, width = 1500, 2, 16, 512
    cases = []
    for _ in range(2):
        x = torch.randn(tokens, width, generator=gen).bfloat16().cuda()
        index = random_index(tokens, top_k, groups, gen).cuda()
        w = torch.rand(tokens, top_k, generator=gen).cuda()
        B = torch.randint(-127, 128, (groups, 300, width), generator=gen, dtype=torch.int8).cuda()
        cases.append((x, index, w, B))

    def layer(x, index, w, B):
        rows, off, _, place = dg.dispatch_tokens(x, index, groups)
        return dg.combine_tokens(dg.gemm_scaled(rows, B, offsets=off), place, w), dg.combine_tokens(rows, place)

    want = [layer(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(10):
        for i, (stream, c) in enumerate(zip(streams, cases)):
            with torch.cuda.stream(stream):
                got[i].append(layer(*c))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for out in g:
            assert all(same_bits(a, b) for a, b in zip(out, w))
