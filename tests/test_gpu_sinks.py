"""Sliding window with sinks (fa_fwd_sink / fa_bwd_sink) on the GPU against the plain 64-bit definition, with the
bounds of parity_util: O within 1e-2 (bf16) or 2e-3 (fp16) of unit-scale inputs, LSE within 1e-3, each gradient
within 2e-2 in the Frobenius norm of every head."""
import pytest
import torch

import exact_io_aware_76_b200 as fa
import masked_reference as ref
from exact_io_aware_76_b200.inputs import draw
from parity_util import all_heads, check_grad, check_lse, check_out, gather_lse, gather_rows, heads_f64

pytestmark = pytest.mark.gpu

CASES = [
    # B, Sq, Sk, H, Hkv, D, causal, window, sinks, dtype
    (1, 1, 1, 1, 1, 64, True, (0, 0), 1, "f16"),              # one token
    (1, 1, 900, 2, 1, 128, True, (100, 0), 4, "bf16"),        # one query, sinks in a tile of their own
    (1, 333, 333, 4, 2, 64, True, (64, 0), 4, "f16"),
    (2, 700, 700, 4, 2, 128, True, (0, 0), 1, "bf16"),        # only itself and the first key
    (1, 1000, 1501, 2, 2, 64, True, (255, 0), 16, "bf16"),    # Sq != Sk
    (1, 1501, 1000, 2, 2, 128, True, (255, 0), 16, "f16"),    # rows without keys
    (1, 1200, 1200, 2, 1, 128, True, (200, -1), 127, "f16"),  # sinks end inside, at and behind a tile's edge
    (1, 1200, 1200, 2, 1, 128, True, (200, 0), 128, "bf16"),
    (1, 1200, 1200, 2, 1, 64, True, (200, 0), 129, "bf16"),
    (1, 1300, 1300, 2, 2, 128, True, (128, 0), 700, "bf16"),  # sinks reach into the early windows
    (2, 640, 900, 6, 3, 64, False, (300, 50), 40, "f16"),     # not causal, right bound
    (1, 500, 800, 2, 2, 128, False, (60, -1), 5, "bf16"),     # unbounded to the right
    (1, 2048, 2048, 2, 2, 128, True, (5000, 0), 4, "bf16"),   # the window hides nothing
    (1, 300, 300, 2, 2, 64, True, (20, 0), 300, "f16"),       # every key is a sink
    (1, 4200, 4200, 1, 1, 128, True, (130, 0), 3, "bf16"),    # the sinks' queries are split over CTAs
    (1, 4200, 4200, 2, 1, 64, True, (130, 0), 200, "f16"),
]


def make(B, Sq, Sk, H, Hkv, D, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    return tuple(draw(s, dt, g, "cuda") for s in ((B, Sq, H, D), (B, Sk, Hkv, D), (B, Sk, Hkv, D), (B, Sq, H, D)))


@pytest.mark.parametrize("B,Sq,Sk,H,Hkv,D,causal,window,sinks,dtype", CASES)
def test_forward_and_backward(B, Sq, Sk, H, Hkv, D, causal, window, sinks, dtype):
    q, k, v, do = make(B, Sq, Sk, H, Hkv, D, dtype, 7000 + Sq + sinks)
    out, lse = fa.fwd(q, k, v, causal=causal, window=window, sinks=sinks)
    dq, dk, dv = fa.bwd(q, k, v, out, lse, do, causal=causal, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    mask = ref.visible(Sq, Sk, causal, window, sinks, "cuda")
    o_r, l_r, dq_r, dk_r, dv_r = ref.attention(q, k, v, lambda b: mask, do=do)
    heads, kv = all_heads(B, H), all_heads(B, Hkv)
    check_out(gather_rows(out, heads), gather_rows(o_r, heads), q.dtype)
    check_lse(gather_lse(lse, heads), gather_lse(l_r, heads))
    if Sq > 1 or Sk > 1:  # one visible key: dQ and dK are exactly 0, and rounding is all a kernel can return
        check_grad(heads_f64(dq, heads), heads_f64(dq_r, heads), "dQ", elementwise=True)
        check_grad(heads_f64(dk, kv), heads_f64(dk_r, kv), "dK", elementwise=True)
    check_grad(heads_f64(dv, kv), heads_f64(dv_r, kv), "dV", elementwise=True)
    unseen = ~mask.any(0)
    assert not dk[:, unseen].any() and not dv[:, unseen].any()
    blind = ~mask.any(1)
    assert not out[:, blind].any() and not dq[:, blind].any()


def test_scale_of_either_sign():
    q, k, v, do = make(1, 600, 600, 2, 2, 128, "bf16", 71)
    for scale in (-0.05, 0.3):
        out, lse = fa.fwd(q, k, v, causal=True, window=(100, 0), sinks=5, scale=scale)
        dq, dk, dv = fa.bwd(q, k, v, out, lse, do, causal=True, window=(100, 0), sinks=5, scale=scale)
        mask = ref.visible(600, 600, True, (100, 0), 5, "cuda")
        o_r, l_r, dq_r, dk_r, dv_r = ref.attention(q, k, v, lambda b: mask, scale=scale, do=do)
        heads = all_heads(1, 2)
        check_out(gather_rows(out, heads), gather_rows(o_r, heads), q.dtype)
        check_lse(gather_lse(lse, heads), gather_lse(l_r, heads))
        for g, r, n in ((dq, dq_r, "dQ"), (dk, dk_r, "dK"), (dv, dv_r, "dV")):
            check_grad(heads_f64(g, heads), heads_f64(r, heads), n)


def test_no_sinks_and_all_sinks_are_the_plain_kernels():
    q, k, v, do = make(1, 700, 700, 2, 2, 128, "bf16", 72)
    a = fa.fwd(q, k, v, causal=True, window=(100, 0))
    b = fa.fwd(q, k, v, causal=True, window=(100, 0), sinks=0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = fa.fwd(q, k, v, causal=True)
    b = fa.fwd(q, k, v, causal=True, window=(100, 0), sinks=700)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    b = fa.fwd(q, k, v, causal=True, sinks=9)  # no left bound: sinks change nothing
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_gradients_repeat_and_match_differences():
    """dK and dV repeat bit for bit although several CTAs share the sinks; the derivative of sum(O * dO) along a
    random direction agrees with central differences of the 64-bit forward (step 1e-4: their own error is ~1e-7)."""
    Sq, window, sinks = 4200, (130, 0), 3
    q, k, v, do = make(1, Sq, Sq, 1, 1, 128, "bf16", 73)
    out, lse = fa.fwd(q, k, v, causal=True, window=window, sinks=sinks)
    dq, dk, dv = fa.bwd(q, k, v, out, lse, do, causal=True, window=window, sinks=sinks)
    _, dk2, dv2 = fa.bwd(q, k, v, out, lse, do, causal=True, window=window, sinks=sinks)
    assert torch.equal(dk, dk2) and torch.equal(dv, dv2)
    mask = ref.visible(Sq, Sq, True, window, sinks, "cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    for which, grad in ((0, dq), (1, dk), (2, dv)):
        # a direction along the gradient itself, so that the derivative is its norm and not a cancelling sum; the
        # sinks' rows alone for k and v, where the split sums land
        u = torch.randn(q.shape, generator=g, device="cuda", dtype=torch.float64) * grad.double().abs().mean()
        u = u + grad.double()
        if which:
            u[:, sinks:] = 0
        x = [q.double(), k.double(), v.double()]

        def loss(step):
            y = list(x)
            y[which] = x[which] + step * u
            return (ref.attention(*y, lambda b: mask)[0] * do.double()).sum()

        h = 1e-4 / float(u.abs().max())
        want = float((loss(h) - loss(-h)) / (2 * h))
        got = float((grad.double() * u).sum())
        assert abs(got - want) <= 2e-2 * abs(want), (which, got, want)


def test_captured_backward_replays_with_its_own_workspace():
    q, k, v, do = make(1, 2100, 2100, 2, 1, 128, "bf16", 74)
    kw = dict(causal=True, window=(130, 0), sinks=4)
    out, lse = fa.fwd(q, k, v, **kw)
    want = fa.bwd(q, k, v, out, lse, do, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        fa.bwd(q, k, v, out, lse, do, **kw)
    s.synchronize()
    with torch.cuda.graph(graph):
        o2, l2 = fa.fwd(q, k, v, **kw)
        grads = fa.bwd(q, k, v, o2, l2, do, **kw)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, out) and torch.equal(grads[1], want[1]) and torch.equal(grads[2], want[2])
        check_grad(heads_f64(grads[0], all_heads(1, 2)), heads_f64(want[0], all_heads(1, 2)), "dQ", rtol=1e-3)


@pytest.mark.parametrize("D", [64, 128])
def test_bounds_beyond_every_key(D):
    """Window bounds up to the largest integer hide nothing, with and without sinks, forward and backward."""
    q, k, v, do = make(1, 500, 400, 2, 1, D, "bf16", 75)
    big = 2 ** 31 - 1
    for causal, window in ((True, (big, big)), (False, (big, big)), (False, (30, big))):
        plain = (-1, -1) if window[0] == big else (30, -1)
        for sinks in (0, 5):
            a = fa.fwd(q, k, v, causal=causal, window=window, sinks=sinks)
            b = fa.fwd(q, k, v, causal=causal, window=plain, sinks=sinks)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            ga = fa.bwd(q, k, v, *a, do, causal=causal, window=window, sinks=sinks)
            gb = fa.bwd(q, k, v, *a, do, causal=causal, window=plain, sinks=sinks)
            assert torch.equal(ga[1], gb[1]) and torch.equal(ga[2], gb[2])
            assert ga[1].any()


def test_given_outputs_on_another_stream():
    q, k, v, do = make(1, 900, 900, 2, 1, 128, "f16", 76)
    kw = dict(causal=True, window=(100, 0), sinks=6)
    want = fa.fwd(q, k, v, **kw)
    gwant = fa.bwd(q, k, v, *want, do, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fa.fwd(q, k, v, stream=s, **kw)
    ggot = fa.bwd(q, k, v, *got, do, stream=s, **kw)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(ggot[1], gwant[1]) and torch.equal(ggot[2], gwant[2])
