"""stream= of the torch entry points: the null stream (0, what
torch.cuda.current_stream().cuda_stream is by default) is the null stream, not
another one that does not wait for it; what a call allocates belongs to the
stream it names, so that no block is reused while work of another stream still
reads it."""
import contextlib
import types

import pytest
import torch

import dense_gemm_10_amd as dg
from dense_gemm_10_amd import grouped, scaled, tokens


class _Streams:
    """torch.cuda's streams and the launch, replaced on the CPU: `now` is the
    handle of the current stream, `calls` what was launched where."""

    def __init__(self, monkeypatch):
        self.now, self.calls = 0x5000, []

        class Handle(int):
            pass

        def external(handle, device=None):
            return Handle(handle if handle else 0x7777)          # 0: one of the pool

        @contextlib.contextmanager
        def current(stream):
            before, self.now = self.now, int(stream)
            yield
            self.now = before

        def launch(entry, name, device, stream, *args):
            self.calls.append((name, self.now if stream is None else stream))

        monkeypatch.setattr(torch.cuda, "ExternalStream", external)
        monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Handle(0))
        monkeypatch.setattr(torch.cuda, "stream", current)
        for module in (grouped, tokens, scaled):
            monkeypatch.setattr(module, "_launch", launch)
            monkeypatch.setattr(module, "_same_device", lambda *a, **k: None)
        monkeypatch.setattr(tokens, "_on_device", lambda *a, **k: None)
        # gemm() and every allocation
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=self.now))
        monkeypatch.setattr(dg, "dg_gemm", lambda *a: self.calls.append(("dg_gemm", a[-1])))
        self.allocated, empty = [], torch.empty

        def counted(*args, **kw):
            self.allocated.append(self.now)
            return empty(*args, **kw)

        monkeypatch.setattr(torch, "empty", counted)


def _calls():
    """(name, call with the given keywords) of every entry point that takes a stream."""
    x, index = torch.zeros(6, 8), torch.zeros(6, 2, dtype=torch.int64)
    place, w, z = torch.zeros(6, 2, dtype=torch.int32), torch.zeros(6, 2), torch.zeros(12, 8)
    A, B = torch.zeros(6, 8, dtype=torch.int8), torch.zeros(4, 8, dtype=torch.int8)
    off = torch.zeros(4, dtype=torch.int32)
    W, Q, scales = torch.zeros(3, 8, 4), torch.zeros(4, 4, dtype=torch.uint8), torch.zeros(4, 1)
    long = torch.zeros(64, 16384)                      # split over K: a workspace
    return [
        ("dg_dispatch", lambda **k: dg.sort_tokens(index, 3, **k)),
        ("dg_dispatch", lambda **k: dg.dispatch_tokens(x, index, 3, **k)),
        ("dg_spread", lambda **k: dg.spread_tokens(x, place, **k)),
        ("dg_combine", lambda **k: dg.combine_tokens(z, place, w, **k)),
        ("dg_combine_grad", lambda **k: dg.combine_tokens_grad(x, z, place, w, **k)),
        ("dg_quantize", lambda **k: dg.quantize_rows(x, **k)),
        ("dg_gemm_scaled", lambda **k: dg.gemm_scaled(A, B, **k)),
        ("dg_gemm_scaled", lambda **k: dg.gemm_scaled(x, B, **k)),
        ("dg_gemm_grouped", lambda **k: dg.gemm_grouped(x, W, off, **k)),
        ("dg_gemm_grouped", lambda **k: dg.gemm_grouped_k(x.t(), x, off, **k)),
        ("dg_gemm_qweight", lambda **k: dg.gemm_qweight(x, Q, scales, group_size=8, **k)),
        ("dg_gemm_grouped", lambda **k: dg.gemm_grouped(x, W, off, torch.zeros(6, 4), **k)),
        ("dg_gemm", lambda **k: dg.gemm(x, W[0], **k)),
        ("dg_gemm", lambda **k: dg.gemm(long, long.t(), **k)),
        ("dg_gemm", lambda **k: dg.gemm(long, long.t(), torch.zeros(64, 64), **k)),
    ]


@pytest.mark.parametrize("at", range(len(_calls())))
@pytest.mark.parametrize("stream,want", [(None, 0x5000), (0, 0), (0x9000, 0x9000)])
def test_call_runs_on_the_stream_it_names(stream, want, at, monkeypatch):
    s = _Streams(monkeypatch)
    name, call = _calls()[at]
    call(stream=stream)
    assert s.calls == [(name, want)] and s.now == 0x5000
    assert all(where == want for where in s.allocated)


def test_a_workspace_is_among_the_allocations(monkeypatch):
    """The last case above would show nothing otherwise."""
    s = _Streams(monkeypatch)
    _calls()[-1][1](stream=0x9000)
    assert s.allocated == [0x9000]


@pytest.mark.gpu
def test_null_stream_waits_for_its_own_work():
    """Inputs written on the null stream behind a long kernel; every call that
    names that stream has to see them."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gen = torch.Generator(device="cuda").manual_seed(3)
    tokens_, k, groups, width = 600, 2, 8, 256
    x = torch.randn(tokens_, width, device="cuda", generator=gen).bfloat16()
    index = torch.randint(0, groups, (tokens_, k), device="cuda", generator=gen)
    w = torch.rand(tokens_, k, device="cuda", generator=gen)
    B = torch.randint(-127, 128, (96, width), device="cuda", generator=gen, dtype=torch.int8)
    _, _, _, place = dg.dispatch_tokens(x, index, groups)
    z = torch.randn(tokens_ * k, width, device="cuda", generator=gen).bfloat16()

    def calls(**kw):
        return [*dg.sort_tokens(index, groups, **kw), *dg.dispatch_tokens(x, index, groups, **kw),
                dg.spread_tokens(x, place, **kw), dg.combine_tokens(z, place, w, **kw),
                *dg.combine_tokens_grad(x, z, place, w, **kw), *dg.quantize_rows(x, **kw),
                dg.gemm_scaled(x, B, **kw)]

    want = [t.clone() for t in calls()]
    new_x, new_z = x.clone(), z.clone()
    x.zero_(), z.zero_()
    torch.cuda.synchronize()
    assert torch.cuda.current_stream().cuda_stream == 0
    torch.cuda._sleep(20_000_000)
    x.copy_(new_x), z.copy_(new_z)
    got = calls(stream=torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_products_leave_the_current_streams_memory_alone():
    """C and workspace of a call with stream= are no blocks that the current
    stream freed while its work on them is still pending."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gen = torch.Generator(device="cuda").manual_seed(5)
    rows, K, N, groups = 384, 512, 256, 4
    x = torch.randn(rows, K, device="cuda", generator=gen).bfloat16()
    W = torch.randn(groups, K, N, device="cuda", generator=gen).bfloat16()
    dy = torch.randn(rows, N, device="cuda", generator=gen).bfloat16()
    off = torch.tensor([0, 100, 100, 250, rows], dtype=torch.int32, device="cuda")
    Q = torch.randint(0, 256, (N, K // 2), device="cuda", generator=gen, dtype=torch.uint8)
    scales = torch.rand(N, K // 128, device="cuda", generator=gen).bfloat16()
    long = torch.randn(128, 16384, device="cuda", generator=gen).bfloat16()
    need = dg.dg_gemm_workspace_size(dg.make_desc(128, 128, 16384, a_type="bf16", b_order="col"))
    assert need > 0

    def calls(**kw):
        return [dg.gemm_grouped(x, W, off, **kw), dg.gemm_grouped_k(x.t(), dy, off, **kw),
                dg.gemm_qweight(x, Q, scales, group_size=128, **kw), dg.gemm(x, W[0], **kw),
                dg.gemm(long, long.t(), **kw)]

    want = [t.clone() for t in calls()]
    sizes = [t.numel() * t.element_size() for t in want] + [need]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.full((n,), 85, dtype=torch.uint8, device="cuda") for n in sizes]
    spans = [(f.data_ptr(), f.data_ptr() + n) for f, n in zip(freed, sizes)]
    kept = [torch.empty_like(f) for f in freed]
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(20_000_000)
    for k, f in zip(kept, freed):
        k.copy_(f)
    freed = f = None
    got = calls(stream=side.cuda_stream)
    for t in got:
        assert not any(lo <= t.data_ptr() < hi for lo, hi in spans)
    torch.cuda.synchronize()
    for k in kept:
        assert bool((k == 85).all())
    for a, b in zip(got, want):
        assert torch.equal(a, b)
