"""Whose memory a call uses when it is given a stream, on the CPU with stand-ins: every tensor that an entry point makes
comes from the given stream, and the ones it returns are recorded for the current stream."""
import contextlib

import pytest
import torch

import exact_io_aware_76_b200 as fa
from test_binding_checks import FakeLib, T

BF16, F32, E4, I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32
made = []


class S(T):
    """A stand-in that notes the stream under which it makes tensors."""

    def new_empty(self, shape, dtype=None):
        t = S((shape,) if isinstance(shape, int) else shape, dtype or self.dtype, self.device)
        t.stream, t.recorded = torch.cuda.current_stream(self.device), []
        made.append(t)
        return t

    def record_stream(self, stream):
        self.recorded.append(stream)


@pytest.fixture
def streams(monkeypatch):
    current = ["current"]
    monkeypatch.setattr(torch.cuda, "set_stream", lambda stream: current.append(stream))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: current[-1])
    monkeypatch.setattr(torch, "empty_like", lambda x: x.new_empty(x.shape))
    monkeypatch.setattr(fa, "lib", lambda: FakeLib([]))
    monkeypatch.setattr(fa, "_device", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(fa, "_stream", lambda stream, dev: None)
    for size in ("workspace_size", "sink_workspace_size", "cache_workspace_size"):
        monkeypatch.setattr(fa, size, lambda *a: 1024)
    made.clear()
    yield
    assert current[-1] == "current"


def qkv(dtype=BF16, Hkv=4):
    return S((2, 100, 4, 64), dtype), S((2, 120, Hkv, 64), dtype), S((2, 120, Hkv, 64), dtype)


def bwd(call, **kw):
    return call(*qkv(), S((2, 100, 4, 64)), S((2, 4, 100), F32), S((2, 100, 4, 64)), **kw)


def cache():
    return dict(k_pages=S((10, 2, 16, 64), E4), v_pages=S((10, 2, 16, 64), E4), k_scale=S((10, 2), F32),
                v_scale=S((10, 2), F32), table=S((3, 5), I32), lens=S((3,), I32))


CALLS = {
    "fwd": (lambda **kw: fa.fwd(*qkv(), **kw), 2, 0),
    "fwd with sinks": (lambda **kw: fa.fwd(*qkv(), window=(9, 0), sinks=2, **kw), 2, 0),
    "fwd_fp8": (lambda **kw: fa.fwd_fp8(*qkv(E4), **kw), 2, 0),
    "bwd": (lambda **kw: bwd(fa.bwd, **kw), 3, 1),
    "bwd with sinks": (lambda **kw: bwd(fa.bwd, window=(9, 0), sinks=2, **kw), 3, 1),
    "bwd_noalloc": (lambda **kw: bwd(fa.bwd_noalloc, **kw), 3, 0),
    "fwd_cache": (lambda **kw: fa.fwd_cache(S((3, 1, 4, 64)), **cache(), **kw), 2, 1),
}


@pytest.mark.parametrize("name", CALLS)
def test_made_tensors_belong_to_the_given_stream(streams, name):
    call, returned, internal = CALLS[name]
    result = call(stream="given")
    assert len(result) == returned and len(made) == returned + internal
    assert all(t.stream == "given" for t in made)
    assert all(t.recorded == ["current"] for t in result)
    assert all(t.recorded == [] for t in made if not any(t is r for r in result))


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_they_are_the_current_ones(streams, name):
    call, returned, internal = CALLS[name]
    call()
    assert len(made) == returned + internal and all(t.stream == "current" and not t.recorded for t in made)
