"""Routed tokens on rows that start on any element, with other data between
them, and with many choices per token: bit for bit what packed operands give,
and nothing written beside the rows."""
import pytest
import torch

import dense_gemm_10_amd as dg
from tokens_util import DT, maps, random_index, same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class _Wide:
    """A matrix as columns [lead, lead + n) of a wider one."""

    def __init__(self, t, lead, tail, fill=3.0):
        self.all = torch.full((t.shape[0], lead + t.shape[1] + tail), fill, dtype=t.dtype, device="cuda")
        self.t = self.all[:, lead:lead + t.shape[1]]
        self.t.copy_(t)
        self.lead, self.n, self.fill = lead, t.shape[1], fill

    def beside_is_untouched(self):
        return bool((self.all[:, :self.lead] == self.fill).all()) and \
            bool((self.all[:, self.lead + self.n:] == self.fill).all())


@pytest.mark.parametrize("dtype,yt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("tokens,top_k,width", [(5, 2, 40), (70, 3, 1001), (33, 9, 2055), (9, 1, 4103)])
@pytest.mark.parametrize("lead,tail", [(1, 0), (3, 6), (0, 1)])
def test_combine_and_its_gradients(lead, tail, tokens, top_k, width, dtype, yt):
    gen = torch.Generator().manual_seed(width + lead)
    rows = tokens * top_k + 4
    place = torch.randperm(rows, generator=gen)[:tokens * top_k].view(tokens, top_k).to(torch.int32)
    place[torch.rand(tokens, top_k, generator=gen) < 0.2] = -1
    place = place.cuda()
    z = torch.randn(rows, width, generator=gen).to(DT[dtype]).cuda()
    w = torch.rand(tokens, top_k, generator=gen).to(DT[dtype]).cuda()
    y0, dy = (torch.randn(tokens, width, generator=gen).to(DT[yt]).cuda() for _ in range(2))
    zw, ww, yw, dyw = (_Wide(t, lead, tail) for t in (z, w, y0, dy))
    dzw = _Wide(torch.zeros_like(z), lead, tail)
    for weights, wide_weights in ((w, ww.t), (None, None)):
        yw.t.copy_(y0)
        want = dg.combine_tokens(z, place, weights, y0.clone(), beta=0.5)
        assert same_bits(dg.combine_tokens(zw.t, place, wide_weights, yw.t, beta=0.5), want)
    want_dz, want_dw = dg.combine_tokens_grad(dy, z, place, w, dz=torch.zeros_like(z))
    got_dz, got_dw = dg.combine_tokens_grad(dyw.t, zw.t, place, ww.t, dz=dzw.t)
    assert same_bits(got_dz, want_dz) and same_bits(got_dw, want_dw)
    assert all(t.beside_is_untouched() for t in (zw, ww, yw, dyw, dzw))


@pytest.mark.parametrize("tokens,top_k", [(1, 100), (7, 65), (40, 130), (3, 4097)])
def test_many_choices(tokens, top_k):
    """Maps, rows and sums of more choices than any kernel takes at once."""
    gen = torch.Generator().manual_seed(top_k)
    groups, width = 11, 33
    index = random_index(tokens, top_k, groups, gen, 0.1)
    x = torch.randn(tokens, width, generator=gen)
    want = maps(index, groups)
    out = torch.zeros(tokens * top_k, width)
    rows, *got = dg.dispatch_tokens(x.cuda(), index.cuda(), groups, out=out.cuda())
    for a, b in zip(got, want):
        assert torch.equal(a.cpu(), b)
    kept = want[1] >= 0
    out[kept] = x[want[1][kept].long() // top_k]
    assert torch.equal(rows.cpu(), out)
    # ones and small integers: every sum is exact
    z = torch.randint(-4, 5, rows.shape, generator=gen).float()
    place = want[2].long()
    ref = torch.where((place >= 0)[..., None], z[place.clamp(min=0)], 0.0).sum(1)
    assert torch.equal(dg.combine_tokens(z.cuda(), got[2]).cpu(), ref)
    w = torch.randint(-3, 4, (tokens, top_k), generator=gen).float()
    dy = torch.randint(-3, 4, (tokens, width), generator=gen).float()
    dz, dw = dg.combine_tokens_grad(dy.cuda(), z.cuda(), got[2], w.cuda(), dz=torch.zeros(rows.shape).cuda())
    ref_dz = torch.zeros(rows.shape)
    ref_dz[place[place >= 0]] = (w[..., None] * dy[:, None])[place >= 0]
    ref_dw = torch.where(place >= 0, (z[place.clamp(min=0)] * dy[:, None]).sum(-1), 0.0)
    assert torch.equal(dz.cpu(), ref_dz) and torch.equal(dw.cpu(), ref_dw)
    q, s = dg.quantize_rows(x.cuda(), got[2], torch.zeros(rows.shape, dtype=torch.int8).cuda(),
                            torch.zeros(rows.shape[0]).cuda())
    q1, s1 = (t.cpu() for t in dg.quantize_rows(x.cuda()))
    t = want[1][kept].long() // top_k
    assert torch.equal(q.cpu()[kept], q1[t]) and torch.equal(s.cpu()[kept], s1[t])
