"""Host-side checks of the paged cache's entry points, without a GPU: the C ABI refuses bad arguments before anything is
launched, and the binding refuses operands that do not fit together."""
import contextlib

import pytest
import torch

import exact_io_aware_76_b200 as fa
from test_binding_checks import FakeLib, T

FAKE = 0x10000
E4, I32, F32, BF16 = torch.float8_e4m3fn, torch.int32, torch.float32, torch.bfloat16


def append(k=FAKE, kp=FAKE, ks=FAKE, table=FAKE, counts=None, B=2, T=3, Hkv=2, D=64, num=10, page=16, width=5, dtype=1):
    return fa.lib().fa_cache_append(k, FAKE, kp, FAKE, ks, FAKE, table, FAKE, counts, B, T, Hkv, D, num, page, width,
                                    dtype, None)


def attend(q=FAKE, kp=FAKE, ks=FAKE, table=FAKE, B=2, Sq=3, H=4, Hkv=2, D=64, num=10, page=16, width=5, left=-1,
           sinks=0, scale=0.0, dtype=1, ws=FAKE, ws_bytes=1 << 40):
    return fa.lib().fa_cache_fwd(q, kp, FAKE, ks, FAKE, table, FAKE, FAKE, FAKE, B, Sq, H, Hkv, D, num, page, width,
                                 left, sinks, scale, dtype, ws, ws_bytes, None)


BOTH = [dict(kp=None), dict(kp=FAKE + 8), dict(ks=None), dict(ks=FAKE + 2), dict(table=None), dict(table=FAKE + 1),
        dict(B=0), dict(Hkv=0), dict(D=0), dict(num=0), dict(page=48), dict(page=256), dict(page=0), dict(width=0),
        dict(num=2 ** 27, page=128), dict(width=2 ** 27), dict(dtype=3)]


@pytest.mark.parametrize("kw", BOTH + [dict(k=None), dict(k=FAKE + 8), dict(T=0), dict(counts=FAKE + 2)])
def test_append_refusals(kw):
    assert append(**kw) == -1


@pytest.mark.parametrize("kw", BOTH + [dict(q=None), dict(q=FAKE + 8), dict(Sq=0), dict(H=3), dict(sinks=-1),
                                       dict(scale=float("inf"))])
def test_attention_refusals(kw):
    assert attend(**kw) == -1


def test_head_dims_and_workspace():
    assert append(D=96) == -2 and attend(D=96) == -2
    need = fa.cache_workspace_size(2, 3, 4, 2, 64)
    assert need > 0
    for kw in (dict(ws=None), dict(ws=FAKE + 16), dict(ws_bytes=need - 1)):
        assert attend(**kw) == -5
    assert fa.cache_workspace_size(2, 400, 4, 2, 64) > need
    for bad in ((0, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 1, 3, 2, 64), (1, 1, 1, 1, 96), (1, 1, 0, 1, 64)):
        assert fa.cache_workspace_size(*bad) == 0


@pytest.fixture
def fake_lib(monkeypatch):
    current = []

    @contextlib.contextmanager
    def device_ctx(dev):
        current.append(dev)
        try:
            yield
        finally:
            current.pop()

    lib = FakeLib(current)
    monkeypatch.setattr(fa, "lib", lambda: lib)
    monkeypatch.setattr(fa, "_device", device_ctx)
    monkeypatch.setattr(fa, "_stream", lambda stream, dev: None)
    monkeypatch.setattr(fa, "cache_workspace_size", lambda *a: 1024)
    return lib


def cache(**over):
    c = dict(k_pages=T((10, 2, 16, 64), E4), v_pages=T((10, 2, 16, 64), E4), k_scale=T((10, 2), F32),
             v_scale=T((10, 2), F32), table=T((3, 5), I32), lens=T((3,), I32))
    c.update(over)
    return c


def test_well_formed_calls_reach_the_library(fake_lib):
    fa.cache_append(T((3, 7, 2, 64)), T((3, 7, 2, 64)), **cache(), counts=T((3,), I32))
    fa.fwd_cache(T((3, 1, 4, 64)), **cache(), out=T((3, 1, 4, 64)), lse=T((3, 4, 1), F32),
                 workspace=T((1024,), torch.uint8))
    assert [c[0] for c in fake_lib.calls] == ["fa_cache_append", "fa_cache_fwd"]


BAD = [dict(k_pages=T((10, 2, 16, 64), torch.uint8)), dict(v_pages=T((9, 2, 16, 64), E4)),
       dict(k_pages=T((10, 2, 16, 128), E4)), dict(k_pages=T((10, 3, 16, 64), E4)),
       dict(k_pages=T((10, 2, 20, 64), E4), v_pages=T((10, 2, 20, 64), E4)), dict(k_scale=T((10,), F32)),
       dict(v_scale=T((10, 2), BF16)), dict(table=T((2, 5), I32)), dict(table=T((3, 5), torch.int64)),
       dict(table=T((3, 5), I32, contiguous=False)), dict(lens=T((3, 1), I32)), dict(lens=T((3,), torch.int64)),
       dict(lens=T((3,), I32, device="cuda:1")), dict(k_pages=T((10, 2, 16, 64), E4, device="cpu"))]


@pytest.mark.parametrize("over", BAD)
def test_binding_refuses_bad_caches(fake_lib, over):
    with pytest.raises((ValueError, TypeError)):
        fa.cache_append(T((3, 7, 2, 64)), T((3, 7, 2, 64)), **cache(**over))
    with pytest.raises((ValueError, TypeError)):
        fa.fwd_cache(T((3, 1, 4, 64)), **cache(**over), out=T((3, 1, 4, 64)), lse=T((3, 4, 1), F32),
                     workspace=T((1024,), torch.uint8))
    assert fake_lib.calls == []


@pytest.mark.parametrize("over", [dict(q=T((3, 1, 4, 64), F32)), dict(q=T((3, 1, 3, 64))), dict(q=T((3, 4, 64))),
                                  dict(q=T((3, 1, 4, 64), device="cpu")), dict(sinks=-1), dict(sinks=0.5),
                                  dict(out=T((3, 1, 4, 64), torch.float16)), dict(lse=T((3, 1, 4), F32)),
                                  dict(workspace=T((1000,), torch.uint8))])
def test_binding_refuses_bad_queries(fake_lib, over):
    a = dict(q=T((3, 1, 4, 64)), out=T((3, 1, 4, 64)), lse=T((3, 4, 1), F32), workspace=T((1024,), torch.uint8))
    a.update(over)
    with pytest.raises((ValueError, TypeError)):
        fa.fwd_cache(a.pop("q"), **cache(), **a)
    assert fake_lib.calls == []


@pytest.mark.parametrize("over", [dict(k=T((3, 7, 2, 64), F32)), dict(v=T((3, 7, 2, 64), torch.float16)),
                                  dict(v=T((3, 6, 2, 64))), dict(counts=T((2,), I32)), dict(counts=T((3,), F32)),
                                  dict(k=T((3, 7, 2, 64), contiguous=False))])
def test_binding_refuses_bad_tokens(fake_lib, over):
    a = dict(k=T((3, 7, 2, 64)), v=T((3, 7, 2, 64)), counts=None)
    a.update(over)
    with pytest.raises((ValueError, TypeError)):
        fa.cache_append(a["k"], a["v"], **cache(), counts=a["counts"])
    assert fake_lib.calls == []


@pytest.mark.parametrize("left,passed", [(130, 130), (2 ** 32 + 130, 2 ** 31 - 1), (-1, -1), (-2 ** 32 + 130, -1)])
def test_windows_past_32_bits_stay_open(fake_lib, monkeypatch, left, passed):
    seen = []
    monkeypatch.setattr(fake_lib, "fa_cache_fwd", lambda *a: seen.append(a) or 0, raising=False)
    fa.fwd_cache(T((3, 1, 4, 64)), **cache(), window_left=left, sinks=5, out=T((3, 1, 4, 64)), lse=T((3, 4, 1), F32),
                 workspace=T((1024,), torch.uint8))
    assert seen[0][17:19] == (passed, 5)
