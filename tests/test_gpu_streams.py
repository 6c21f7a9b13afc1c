"""Calls on a given stream while the current one is behind: memory that the current stream has given back, but whose last
use there has not run yet, is not written by the call."""
import pytest
import torch

import exact_io_aware_76_b200 as fa
from test_gpu_cache import gen, make_cache

pytestmark = pytest.mark.gpu


def calls():
    g = gen(90)
    q, k, v, do = (torch.randn((1, 256, 2, 64), generator=g, device="cuda").to(torch.bfloat16) for _ in range(4))
    out, lse = fa.fwd(q, k, v, causal=True)
    e = [x.to(torch.float8_e4m3fn) for x in (q, k, v)]
    c = make_cache([900, 300], 2, 64, 32, g)
    q1 = torch.randn((2, 1, 8, 64), generator=g, device="cuda").to(torch.bfloat16)
    win = dict(causal=True, window=(50, 0), sinks=3)
    return {"fwd": lambda **kw: fa.fwd(q, k, v, causal=True, **kw),
            "fwd with sinks": lambda **kw: fa.fwd(q, k, v, **win, **kw),
            "fwd_fp8": lambda **kw: fa.fwd_fp8(*e, **kw),
            "bwd": lambda **kw: fa.bwd(q, k, v, out, lse, do, causal=True, **kw)[1:],  # (dQ's sums have no fixed order)
            "bwd_noalloc": lambda **kw: fa.bwd_noalloc(q, k, v, out, lse, do, causal=True, **kw)[1:],
            "fwd_cache": lambda **kw: fa.fwd_cache(q1, **c, **kw)}


@pytest.mark.parametrize("name", ["fwd", "fwd with sinks", "fwd_fp8", "bwd", "bwd_noalloc", "fwd_cache"])
def test_memory_the_current_stream_still_uses(name):
    call = calls()[name]
    want = call()
    sizes = [x.nbytes for x in want] + [1 << 20]
    s = torch.cuda.Stream()
    busy = torch.randn((8192, 8192), device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    for _ in range(10):
        busy = busy @ busy * 1e-2
    for n in sizes * 3:  # written by the current stream after all that, and given back before
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
    got = call(stream=s)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["fwd", "fwd with sinks", "fwd_fp8", "bwd", "fwd_cache"])
def test_captured_on_a_side_stream(name):
    """Two calls on two branches of one captured graph, each with tensors and workspaces of its own; replays agree."""
    call = calls()[name]
    want = call()
    side = [torch.cuda.Stream() for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        for s in side:
            s.wait_stream(here)
        got = [call(stream=s) for s in side]
        for s in side:
            here.wait_stream(s)
    for _ in range(3):
        for r in got:
            for x in r:
                x.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))
    assert fa.device_status() == 0
