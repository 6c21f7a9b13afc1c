"""Host-side checks of the entry points with sinks: refusals before anything is launched, and workspace sizes."""
import pytest

import exact_io_aware_76_b200 as fa

FAKE = 0x10000


def fwd(sinks=4, left=64, B=1, Sq=128, Sk=128, H=2, Hkv=1, D=64, scale=0.0, dtype=1, q=FAKE):
    return fa.lib().fa_fwd_sink(q, FAKE, FAKE, FAKE, FAKE, B, Sq, Sk, H, Hkv, D, 1, left, 0, sinks, scale, dtype, None)


def bwd(sinks=4, left=64, B=1, Sq=128, Sk=128, H=2, Hkv=1, D=64, scale=0.0, dtype=1, q=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return fa.lib().fa_bwd_sink(q, *[FAKE] * 8, B, Sq, Sk, H, Hkv, D, 1, left, 0, sinks, scale, dtype, ws, ws_bytes,
                                None)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("kw,rc", [(dict(sinks=-1), -1), (dict(B=0), -1), (dict(Hkv=3), -1), (dict(q=None), -1),
                                   (dict(q=FAKE + 8), -1), (dict(scale=float("nan")), -1), (dict(dtype=7), -1),
                                   (dict(D=96), -2)])
def test_refusals(call, kw, rc):
    assert call(**kw) == rc


def size(B=1, Sq=4200, Sk=4200, H=1, Hkv=1, D=128, causal=1, left=130, right=0, sinks=3):
    return fa.lib().fa_bwd_sink_workspace_size(B, Sq, Sk, H, Hkv, D, causal, left, right, sinks)


def test_workspace_sizes():
    plain = fa.workspace_size(1, 4200, 1, 128)
    assert size() > plain  # few CTAs, a long sequence: the sinks' queries are split
    assert bwd(Sq=4200, Sk=4200, H=1, D=128, left=130, sinks=3, ws_bytes=size() - 1) == -5
    assert size(sinks=0) == plain and size(left=-1) == plain and size(sinks=4200) == plain and size(left=5000) == plain
    assert size(B=8, H=32, Hkv=32) == fa.workspace_size(8, 4200, 32, 128)  # enough work in every SM: no split
    for bad in (dict(sinks=-1), dict(B=0), dict(Hkv=0), dict(H=3, Hkv=2), dict(D=96)):
        assert size(**bad) == 0


@pytest.mark.parametrize("sinks", [-1, 1.5, 2 ** 31])
def test_binding_refuses_bad_counts(sinks):
    with pytest.raises(ValueError):
        fa.check_sinks(sinks, 0.0)


def test_binding_refuses_sinks_with_dropout():
    fa.check_sinks(4, 0.0)
    with pytest.raises(ValueError):
        fa.check_sinks(4, 0.1)


@pytest.mark.parametrize("left", [4199, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 130, -1, -2 ** 32 + 130])
def test_bounds_past_32_bits_hide_nothing(left):
    plain = fa.workspace_size(1, 4200, 1, 128)
    assert fa.sink_workspace_size(1, 4200, 4200, 1, 1, 128, True, (left, 0), 3) == plain
