"""The paged e4m3 cache where its kernels could go wrong without a sign: runs of short units in one CTA, factors that
leave the fp32 range, query rows that see nothing, light weights beside heavy ones, lengths past the table."""
import math

import pytest
import torch

import exact_io_aware_76_b200 as fa
from test_gpu_cache import DT, E4M3, check, gen, make_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hkv,Sq,D,dtype", [(16, 8, 1, 128, "bf16"), (16, 8, 1, 64, "f16"), (16, 4, 3, 128, "f16"),
                                              (16, 2, 4, 64, "bf16")])
def test_short_units_whose_rows_differ_by_large_factors(H, Hkv, Sq, D, dtype):
    """Many units of one to three tiles per CTA, the query rows of neighbouring units 2^12 apart: a row factor of the
    wrong unit changes every score of a row. Equal bits in every run."""
    g = gen(86)
    B = 200
    lens = torch.randint(1, 385, (B,), generator=g, device="cuda").tolist()
    c = make_cache(lens, Hkv, D, 64, g)
    q = torch.randn((B, Sq, Hkv, H // Hkv, D), generator=g, device="cuda")
    unit = torch.arange(B * Hkv, device="cuda").view(B, 1, Hkv, 1, 1)
    q = (q * torch.where(unit % 2 == 0, 2.0 ** -8, 2.0 ** 4)).view(B, Sq, H, D).to(DT[dtype])
    out, lse = fa.fwd_cache(q, **c)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    check(q, c, out, lse, -1, 0, only=range(0, B, 8))
    for _ in range(20):
        again = fa.fwd_cache(q, **c)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("Sq,H,Hkv", [(4, 2, 1), (4, 4, 1), (4, 8, 1), (90, 2, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_query_rows_that_are_not_finite(Sq, H, Hkv, dtype, bad):
    """A padded batch with NaNs or infinities in its padding: a row that sees no key (shorter sequence, no page) is 0 and
    -inf whatever its q holds; one that sees a key is NaN; the other rows have the bits that they have beside rows of
    zeros. One sequence is long enough to be cut between CTAs."""
    g = gen(87)
    lens = [3, 0, 20000, 700, 150]
    c = make_cache(lens, Hkv, 128, 32, g)
    c["table"][4] = -1
    q = torch.randn((len(lens), Sq, H, 128), generator=g, device="cuda").to(DT[dtype])
    rows = torch.zeros((len(lens), Sq, H), dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        rows[b, :max(0, Sq - n), 0] = True  # the padding of one head
    rows[4, :, 1] = True                    # no pages
    rows[2, 1, 1] = rows[3, Sq - 1, 0] = True
    q[rows] = 0
    want = fa.fwd_cache(q, **c)
    q[rows] = bad
    blind = torch.isneginf(want[1]).transpose(1, 2)
    out, lse = fa.fwd_cache(q, **c)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    lse, clean = lse.transpose(1, 2), want[1].transpose(1, 2)
    assert blind[0, :Sq - 3].all() and blind[1].all() and blind[4].all() and not blind[2:4].any()
    assert not out[blind].any() and torch.isneginf(lse[blind]).all()
    assert torch.isnan(out[rows & ~blind]).all() and torch.isnan(lse[rows & ~blind]).all()
    assert torch.equal(out[~rows], want[0][~rows]) and torch.equal(lse[~rows], clean[~rows])


@pytest.mark.parametrize("Sq,H", [(4, 2), (4, 4), (8, 4), (90, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [None, 1e-38, -1e-38])
def test_zeros_in_queries_and_keys(Sq, H, dtype, scale):
    """A row of zeros over pages of zeros, as an append leaves them (scale 2^-50): the product of the two smallest factors
    is not to turn masked scores into NaNs. Every visible key counts the same."""
    n, D, page = 200, 64, 32
    g = gen(88)
    m = -(-n // page)
    c = {x: torch.zeros((m, 1, page, D), device="cuda").to(E4M3) for x in ("k_pages", "v_pages")}
    c.update({x: torch.ones((m, 1), device="cuda") for x in ("k_scale", "v_scale")})
    c["table"] = torch.arange(m, device="cuda", dtype=torch.int32)[None].contiguous()
    c["lens"] = torch.tensor([n], dtype=torch.int32, device="cuda")
    k = torch.zeros((1, n, 1, D), device="cuda", dtype=DT[dtype])
    fa.cache_append(k, torch.randn(k.shape, generator=g, device="cuda").to(k.dtype), **c)
    assert (c["k_scale"] == 2.0 ** -50).all()
    q = torch.randn((1, Sq, H, D), generator=g, device="cuda").to(DT[dtype])
    q[:, :, 0] = 0
    out, lse = fa.fwd_cache(q, **c, scale=scale)
    check(q, c, out, lse, -1, 0, scale)
    seen = torch.arange(n - Sq + 1, n + 1, device="cuda").double()
    assert (lse[0, 0].double() - seen.log()).abs().max() <= 1e-5


@pytest.mark.parametrize("Sq,H", [(1, 8), (1, 16), (1, 32), (40, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heavy", [0, 9999])
def test_light_weights_beside_a_heavy_one(Sq, H, dtype, heavy):
    """One key d (in the exponent of e) above 20000 equal ones, which all round the same way. Their weights' relative error:
    2^-11 from fp16, 2^-30 e^d from the last part's smallest step, 2^-13 for up to 640 sums in fp32 (2^-23 each) and the
    exponentials; then the output's own rounding. As many sequences (over the same pages) as CTAs, so that few are cut and the
    heavy key's maximum is the light ones' too."""
    n, D, page, B = 20001, 64, 64, 150
    m = -(-n // page)
    kp, vp = (torch.zeros((m, 1, page, D), device="cuda") for _ in range(2))
    kp[heavy // page, 0, heavy % page, 0] = 1.0
    vp[..., 1] = 1.0
    vp[heavy // page, 0, heavy % page, 1] = 0.0
    c = {"k_pages": kp.to(E4M3), "v_pages": vp.to(E4M3), "k_scale": torch.ones((m, 1), device="cuda"),
         "v_scale": torch.ones((m, 1), device="cuda"),
         "table": torch.arange(m, device="cuda", dtype=torch.int32).repeat(B, 1),
         "lens": torch.full((B,), n, dtype=torch.int32, device="cuda")}
    for d in (8.0, 11.0, 12.0, 13.0, 14.0, 16.0, 18.0):
        q = torch.zeros((B, Sq, H, D), device="cuda", dtype=DT[dtype])
        q[..., 0] = d
        out, lse = fa.fwd_cache(q, **c, scale=1.0)
        light = (n - Sq + torch.arange(Sq, device="cuda")).double() * math.exp(-d)
        want = (light / (1 + light))[None, :, None].expand(B, Sq, H)
        tol = torch.finfo(DT[dtype]).eps / 2 + 2.0 ** -11 + 2.0 ** -13 + 2.0 ** -30 * math.exp(d)
        off = (out[..., 1].double() / want - 1).abs().max()
        assert off <= tol, (d, float(off), tol)
        assert (lse.double() - (d + torch.log1p(light))).abs().max() <= 1e-4


@pytest.mark.parametrize("Sq,H", [(1, 8), (3, 8), (4, 8), (90, 2)])
@pytest.mark.parametrize("left,sinks", [(-1, 0), (200, 5)])
def test_lengths_past_the_table(Sq, H, left, sinks):
    """A length beyond max_pages * page counts as that many tokens in the attention; an append drops what lies beyond, in a
    cache whose other pages and slots keep their bytes."""
    g = gen(89)
    page, Hkv, D = 32, 1, 64
    c = make_cache([1504, 1504], Hkv, D, page, g, width=47)  # as many tokens as the table has places for
    c["lens"][1] = 300
    q = torch.randn((2, Sq, H, D), generator=g, device="cuda").to(torch.bfloat16)
    want = fa.fwd_cache(q, **c, window_left=left, sinks=sinks)
    check(q, c, *want, left, sinks)
    for n in (1505, 10 ** 6, 2 ** 31 - 1):
        c["lens"][0] = n
        got = fa.fwd_cache(q, **c, window_left=left, sinks=sinks)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c["lens"][0], c["lens"][1] = 1510, 0
    k, v = (torch.randn((2, 10, Hkv, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    before = {x: c[x].clone() for x in ("k_pages", "v_pages", "k_scale", "v_scale")}
    once = {**c, **{x: t.clone() for x, t in before.items()}, "lens": torch.tensor([1504, 0], dtype=torch.int32, device="cuda")}
    fa.cache_append(k[:, :4].contiguous(), v[:, :4].contiguous(), **once)  # the four that have a place
    fa.cache_append(k, v, **c)
    for x in ("k_pages", "v_pages", "k_scale", "v_scale"):
        assert torch.equal(c[x].view(torch.uint8), once[x].view(torch.uint8))
    last = int(c["table"][0, 46])
    assert not torch.equal(c["k_pages"][last].view(torch.uint8), before["k_pages"][last].view(torch.uint8))
    for n in (1600, 2 ** 31 - 1):
        c["lens"][0] = n
        fa.cache_append(k, v, **c)  # none has a place
        assert torch.equal(c["k_pages"].view(torch.uint8), once["k_pages"].view(torch.uint8))
    assert fa.device_status() == 0
