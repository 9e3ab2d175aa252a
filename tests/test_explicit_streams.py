"""stream= of the torch entry points: the null stream (0, what
torch.cuda.current_stream().cuda_stream is by default) is the null stream, not
another one that does not wait for it."""
import contextlib

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


def _calls():
    """(name, call with the given keywords) of every entry point that takes a stream."""
    x, index = torch.zeros(6, 8), torch.zeros(6, 2, dtype=torch.int64)
    place, w, z = torch.zeros(6, 2, dtype=torch.int32), torch.zeros(6, 2), torch.zeros(12, 8)
    A, B = torch.zeros(6, 8, dtype=torch.int8), torch.zeros(4, 8, dtype=torch.int8)
    return [
        ("dg_dispatch", lambda **k: dg.sort_tokens(index, 3, **k)),
        ("dg_dispatch", lambda **k: dg.dispatch_tokens(x, index, 3, **k)),
        ("dg_spread", lambda **k: dg.spread_tokens(x, place, **k)),
        ("dg_combine", lambda **k: dg.combine_tokens(z, place, w, **k)),
        ("dg_combine_grad", lambda **k: dg.combine_tokens_grad(x, z, place, w, **k)),
        ("dg_quantize", lambda **k: dg.quantize_rows(x, **k)),
        ("dg_gemm_scaled", lambda **k: dg.gemm_scaled(A, B, **k)),
        ("dg_gemm_scaled", lambda **k: dg.gemm_scaled(x, B, **k)),
    ]


@pytest.mark.parametrize("at", range(len(_calls())))
@pytest.mark.parametrize("stream,want", [(None, 0x5000), (0, 0), (0x9000, 0x9000)])
def test_call_runs_on_the_stream_it_names(stream, want, at, monkeypatch):
    s = _Streams(monkeypatch)
    name, call = _calls()[at]
    call(stream=stream)
    assert s.calls == [(name, want)] and s.now == 0x5000


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
