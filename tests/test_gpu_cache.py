"""The paged e4m3 cache on the GPU: fa_cache_append against a rounding written out in 64 bits (bit for bit), and
fa_cache_fwd against the plain 64-bit definition on the values the cache holds.

Bounds of the attention, from what the kernel rounds: with p the exact probabilities and v the values,
  |O - O_ref| <= tol * sum_j p_j |v_j| + 4 floor * max_j p_j * ||v||_2 + half a step of the output type,
tol = 2^-7 (bf16) or 2^-9 (fp16): the weights' own rounding (2^-8, 2^-11) and as much or more for the scores' fp32
sums and what q's parts drop; floor: half the last part's smallest step against a largest weight of at least 2^2
(bf16: 2^-10 / 2^2; fp16: 2^-17 / 2^2), independent for the keys, so four standard deviations of at most that each."""
import math

import pytest
import torch

import exact_io_aware_76_b200 as fa
import masked_reference as ref

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make_cache(lens, Hkv, D, page, g, spread=0, spare=3, pow2=True, width=None):
    """Pages in random order with unit-normal values for lens tokens, under scales that differ by page and head
    (2^-spread .. 2^spread around what the values need); NaN codes in every slot no token has; page numbers nobody may
    use behind the last page."""
    B = len(lens)
    need = [-(-n // page) for n in lens]
    width = max(1, max(need) + 2) if width is None else width
    n = sum(need) + spare
    order = torch.randperm(n, generator=g, device="cuda").tolist()
    table = torch.full((B, width), -7, dtype=torch.int32)
    table[:, 1::2] = 10 ** 9
    for b in range(B):
        for i in range(need[b]):
            table[b, i] = order.pop()
    c = {"table": table.cuda(), "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    for x in "kv":
        e = torch.randint(-spread, spread + 1, (n, Hkv), generator=g, device="cuda").float()
        scale = torch.exp2(e - 6) * (1.0 if pow2 else 1.37)
        codes = (torch.randn((n, Hkv, page, D), generator=g, device="cuda") * 64).clamp(-448, 448).to(E4M3)
        raw = codes.view(torch.uint8)
        used = torch.zeros((n, page), dtype=torch.bool, device="cuda")
        for b in range(B):
            for i in range(need[b]):
                used[table[b, i], :min(page, lens[b] - i * page)] = True
        raw[~used[:, None, :, None].expand_as(raw)] = 0x7F
        c[x + "_pages"], c[x + "_scale"] = codes, scale
    return c


def values(c, x, b, h, n):
    """float64 [n, D] of K or V of head h, and which of the n tokens have a page."""
    pages, scale = c[x + "_pages"], c[x + "_scale"]
    page = pages.shape[2]
    out = torch.zeros((n, pages.shape[3]), dtype=torch.float64, device="cuda")
    has = torch.zeros(n, dtype=torch.bool, device="cuda")
    for i in range(-(-n // page)):
        pid = int(c["table"][b, i])
        lo, hi = i * page, min(n, (i + 1) * page)
        if 0 <= pid < pages.shape[0]:
            out[lo:hi] = pages[pid, h, :hi - lo].double() * scale[pid, h].double()
            has[lo:hi] = True
    return out, has


def check(q, c, out, lse, left, sinks, scale=None, only=None):
    B, Sq, H, D = q.shape
    Hkv = c["k_pages"].shape[1]
    tol, floor = (2.0 ** -7, 2.0 ** -12) if q.dtype == torch.bfloat16 else (2.0 ** -9, 2.0 ** -19)
    for b in range(B) if only is None else only:
        n = int(c["lens"][b])
        mask = ref.visible(Sq, n, True, (left, -1), sinks, "cuda", shift=n - Sq)
        for g in range(Hkv):
            k, has = values(c, "k", b, g, n)
            v, _ = values(c, "v", b, g, n)
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                o, ls = out[b, :, h].double(), lse[b, h].double()
                if n == 0:
                    assert not o.any() and torch.isneginf(ls).all()
                    continue
                m = mask & has
                p, o_r, l_r = ref.forward(q[b, :, h].double(), k, v, m, scale)
                blind = ~m.any(1)
                assert not o[blind].any() and torch.isneginf(ls[blind]).all()
                if (~blind).any():
                    assert torch.isfinite(ls[~blind]).all() and (ls - l_r)[~blind].abs().max() <= 1e-3
                seen = v * m.any(0)[:, None]
                exponent = torch.floor(torch.log2(o_r.abs().clamp(min=2.0 ** -14)))
                ulp = 2.0 ** (exponent - (8 if q.dtype == torch.bfloat16 else 11))
                bound = tol * (p @ v.abs()) + 4 * floor * p.amax(-1, keepdim=True) * seen.norm(dim=0)[None] + ulp
                bad = ~((o - o_r).abs() <= bound)
                assert not bad.any(), (b, h, int(bad.sum()), float(((o - o_r).abs() / bound).max()))


CASES = [
    # H, Hkv, Sq, D, page, lens, left, sinks, dtype
    (1, 1, 1, 128, 16, [1], -1, 0, "bf16"),
    (8, 2, 1, 64, 16, [200, 0, 1, 127, 128, 129], -1, 0, "bf16"),
    (8, 1, 1, 128, 32, [5000], -1, 0, "f16"),                  # one sequence over many CTAs
    (32, 1, 1, 128, 64, [700, 20000, 3], -1, 0, "bf16"),       # 32 query heads on one K/V head, ragged
    (10, 2, 3, 64, 128, [1000, 2, 131], -1, 0, "f16"),         # three tokens, one sequence shorter than that
    (8, 8, 4, 128, 64, [640, 333], 100, 4, "bf16"),            # window and sinks
    (8, 2, 1, 128, 16, [3000, 90, 1500], 255, 20, "f16"),
    (4, 1, 8, 64, 32, [3000, 4], 64, 200, "bf16"),             # sinks in two tiles
    (4, 4, 1, 128, 64, [900], 0, 1, "bf16"),                   # itself and the first token
    (8, 8, 1, 128, 64, [100 + 331 * i for i in range(24)], -1, 0, "bf16"),  # many tiles and units per CTA
    (8, 8, 1, 64, 16, [100 + 97 * i for i in range(40)], 700, 4, "f16"),
    (4, 4, 70, 128, 32, [40 + 211 * i for i in range(24)], -1, 0, "bf16"),
    (33, 1, 1, 128, 64, [500, 129], -1, 0, "bf16"),            # one row too many for the small kernel
    (8, 2, 40, 64, 16, [300, 40, 17, 0], -1, 0, "f16"),
    (8, 2, 300, 128, 64, [300, 1000, 301], -1, 0, "bf16"),     # a whole prompt, and chunks of two
    (4, 1, 257, 128, 128, [3000], -1, 0, "f16"),
    (4, 2, 500, 64, 32, [2500, 400], 300, 10, "bf16"),
    (2, 1, 700, 128, 64, [700, 5000], 50, 130, "f16"),
]


@pytest.mark.parametrize("H,Hkv,Sq,D,page,lens,left,sinks,dtype", CASES)
def test_attention(H, Hkv, Sq, D, page, lens, left, sinks, dtype):
    g = gen(900 + Sq + H)
    c = make_cache(lens, Hkv, D, page, g)
    q = torch.randn((len(lens), Sq, H, D), generator=g, device="cuda").to(DT[dtype])
    out, lse = fa.fwd_cache(q, **c, window_left=left, sinks=sinks)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    check(q, c, out, lse, left, sinks)
    again = fa.fwd_cache(q, **c, window_left=left, sinks=sinks)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("Sq,H,Hkv", [(1, 8, 2), (90, 4, 1)])
@pytest.mark.parametrize("pow2", [True, False])
def test_scales_far_apart(Sq, H, Hkv, pow2):
    """Scales of the pages from 2^-26 to 2^14: the ones that matter are the large ones, whatever comes first."""
    g = gen(31)
    c = make_cache([1500, 700], Hkv, 128, 32, g, pow2=pow2)
    e = torch.randint(-20, 21, c["v_scale"].shape, generator=g, device="cuda").float()
    c["v_scale"] = c["v_scale"] * torch.exp2(e)
    q = torch.randn((2, Sq, H, 128), generator=g, device="cuda").to(torch.bfloat16)
    out, lse = fa.fwd_cache(q, **c)
    check(q, c, out, lse, -1, 0)


@pytest.mark.parametrize("Sq,H,Hkv", [(1, 8, 2), (90, 4, 1)])
def test_tokens_without_a_page(Sq, H, Hkv):
    """Pages given back (numbers outside the cache): their tokens are not seen, wherever they lie."""
    g = gen(32)
    c = make_cache([1500, 700], Hkv, 128, 32, g)
    c["table"][0, 3:30] = -1
    c["table"][0, 40] = c["k_pages"].shape[0]
    c["table"][1, 0] = 2 ** 31 - 1
    c["table"][1, 5:] = -2 ** 31
    q = torch.randn((2, Sq, H, 128), generator=g, device="cuda").to(torch.bfloat16)
    out, lse = fa.fwd_cache(q, **c)
    check(q, c, out, lse, -1, 0)
    c["table"][:] = -1
    out, lse = fa.fwd_cache(q, **c)
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("Sq,H,Hkv", [(1, 8, 2), (90, 4, 1)])
def test_stale_tokens_outside_window_and_sinks(Sq, H, Hkv):
    """NaN codes in tokens that the window hides from every query change nothing."""
    g = gen(33)
    c = make_cache([1500], Hkv, 64, 32, g, width=47)
    q = torch.randn((1, Sq, H, 64), generator=g, device="cuda").to(torch.bfloat16)
    left, sinks = 200, 5
    want = fa.fwd_cache(q, **c, window_left=left, sinks=sinks)
    for x in "kv":
        raw = c[x + "_pages"].view(torch.uint8)
        for t in range(sinks, 1500 - Sq - left):
            raw[int(c["table"][0, t // 32]), :, t % 32] = 0x7F
    got = fa.fwd_cache(q, **c, window_left=left, sinks=sinks)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    c["lens"][:] = 10 ** 6  # more than the table holds: the tokens it holds count
    assert torch.isfinite(fa.fwd_cache(q, **c, window_left=-1)[1]).sum() >= 0
    assert fa.device_status() == 0


@pytest.mark.parametrize("Sq,H,Hkv", [(1, 2, 1), (90, 2, 1)])
@pytest.mark.parametrize("scale", [-0.1, 0.02, 4.0])
def test_scale_and_odd_queries(Sq, H, Hkv, scale):
    """Softmax scales of either sign, query rows of zeros, tiny and huge rows; a NaN stays in its row."""
    g = gen(34)
    c = make_cache([600], Hkv, 128, 64, g)
    q = torch.randn((1, Sq, H, 128), generator=g, device="cuda").to(torch.float16)
    q[0, 0, 0] = 0
    out, lse = fa.fwd_cache(q, **c, scale=scale)
    check(q, c, out, lse, -1, 0, scale)
    q[0, -1, 1] *= 2.0 ** -12
    out, lse = fa.fwd_cache(q, **c, scale=scale)
    check(q, c, out, lse, -1, 0, scale)
    for bad in (math.nan, math.inf):
        q2 = q.clone()
        q2[0, 0, 0, 5] = bad
        o2, l2 = fa.fwd_cache(q2, **c, scale=scale)
        assert torch.isnan(o2[0, 0, 0]).all() and torch.isnan(l2[0, 0, 0])
        keep = torch.ones((1, Sq, H), dtype=torch.bool, device="cuda")
        keep[0, 0, 0] = False
        assert torch.equal(o2[keep], out[keep])


# --------------------------------------------------------------------------------------------------- append
def round_e4m3(x):
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return (torch.round(x / step) * step).clamp(-448, 448)


def append_reference(c, k, v, counts):
    """The appended cache in float64 codes and scales, token by token."""
    out = {}
    B, T, Hkv, D = k.shape
    page = c["k_pages"].shape[2]
    num = c["k_pages"].shape[0]
    for x, new in (("k", k), ("v", v)):
        codes, scale = c[x + "_pages"].double().cpu(), c[x + "_scale"].double().cpu()
        for b in range(B):
            n = int(c["lens"][b])
            cnt = max(0, min(counts[b], T, n))
            p = n - cnt
            while p < n:
                i = p // page
                hi = min(n, (i + 1) * page)
                pid = int(c["table"][b, i]) if i < c["table"].shape[1] else -1
                if 0 <= pid < num:
                    rows = new[b, T - n + p:T - n + hi].double().cpu().transpose(0, 1)  # [Hkv, tokens, D]
                    a = p % page
                    for h in range(Hkv):
                        fin = rows[h][torch.isfinite(rows[h])].abs()
                        big = float(fin.max()) if fin.numel() else 0.0
                        s = 2.0 ** -50
                        while s * 448 < big and s < 2.0 ** 50:
                            s *= 2
                        if a:
                            old = float(scale[pid, h])
                            s = max(s, old)
                            codes[pid, h, :a] = round_e4m3(codes[pid, h, :a] * (old / s))
                        codes[pid, h, a:a + hi - p] = torch.where(torch.isnan(rows[h]), math.nan,
                                                                  round_e4m3((rows[h] / s).clamp(-448, 448)))
                        scale[pid, h] = s
                p = hi
        out[x + "_pages"], out[x + "_scale"] = codes, scale
    return out


def same(a, b):
    a, b = a.double().cpu(), b.double()
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))


@pytest.mark.parametrize("Hkv,D,page,T,lens,counts,dtype", [
    (1, 128, 16, 1, [1], None, "bf16"),
    (3, 64, 16, 1, [16, 17, 5, 0], None, "f16"),               # last of a page, first of one, inside, nothing there
    (2, 128, 64, 1, [100, 65, 64, 1], [1, 1, 0, 1], "bf16"),
    (2, 64, 32, 40, [40, 100, 41, 39], [40, 33, 1, 39], "f16"),  # padded rows
    (1, 128, 128, 300, [300, 1000], [300, 300], "bf16"),
    (2, 128, 16, 50, [50, 50], [99, -3], "f16"),               # counts out of range are clamped
])
def test_append(Hkv, D, page, T, lens, counts, dtype):
    g = gen(50 + T)
    c = make_cache(lens, Hkv, D, page, g, spread=2)
    for x in "kv":  # what is there before has finite codes in its slots, others hold NaN codes that must stay
        c[x + "_scale"] = c[x + "_scale"].clone()
    B = len(lens)
    k, v = (torch.randn((B, T, Hkv, D), generator=g, device="cuda").mul_(2.0 ** m).to(DT[dtype]) for m in (3, -4))
    k[0, -1, 0, 3] = math.inf
    k[0, -1, 0, 4] = -math.inf
    v[-1, -1, 0, 5] = math.nan
    for b in range(B):  # rows of padding are not read
        n = T if counts is None else max(0, min(counts[b], T))
        k[b, :T - n], v[b, :T - n] = math.nan, math.nan
    want = append_reference(c, k, v, [T] * B if counts is None else counts)
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    fa.cache_append(k, v, **c, counts=cnt)
    torch.cuda.synchronize()
    for x in ("k_pages", "v_pages", "k_scale", "v_scale"):
        assert same(c[x], want[x]), x


def test_append_extreme_magnitudes_and_no_pages():
    g = gen(60)
    c = make_cache([20, 20, 20], 1, 64, 16, g)
    c["table"][2, :] = -1
    k = torch.zeros((3, 20, 1, 64), device="cuda", dtype=torch.bfloat16)
    v = torch.full_like(k, 3e38)
    v[1] = 1e-30
    want = append_reference(c, k, v, [20] * 3)
    fa.cache_append(k, v, **c)
    for x in ("k_pages", "v_pages", "k_scale", "v_scale"):
        assert same(c[x], want[x]), x


# ------------------------------------------------------------------------------------------------- together
def test_prompt_then_tokens_as_a_model_runs_them():
    """A layer of a streaming decoder: prompts appended and attended in one chunk, then tokens one at a time with the
    lengths advanced on the device; every step against 64 bits on what the cache holds, and the first chunk against the
    forward with sinks on the unrounded values (e4m3 K and V: relative error 2^-4 of each, so a loose bound)."""
    B, H, Hkv, D, page, left, sinks = 2, 8, 2, 128, 32, 150, 4
    g = gen(70)
    lens = [333, 250]
    c = make_cache([n + 40 for n in lens], Hkv, D, page, g)
    T = max(lens)
    c["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn((B, T, n, D), generator=g, device="cuda").to(torch.bfloat16) for n in (H, Hkv, Hkv))
    fa.cache_append(k, v, **c, counts=c["lens"])
    out, lse = fa.fwd_cache(q, **c, window_left=left, sinks=sinks)
    check(q, c, out, lse, left, sinks)
    plain, _ = fa.fwd(q[:1], k[:1], v[:1], causal=True, window=(left, 0), sinks=sinks)
    assert (out[:1].float() - plain.float()).norm() <= 0.1 * plain.float().norm()
    for _ in range(35):
        c["lens"] += 1
        q, k, v = (torch.randn((B, 1, n, D), generator=g, device="cuda").to(torch.bfloat16) for n in (H, Hkv, Hkv))
        fa.cache_append(k, v, **c)
        out, lse = fa.fwd_cache(q, **c, window_left=left, sinks=sinks)
    check(q, c, out, lse, left, sinks)
    assert fa.device_status() == 0


def test_captured_step_follows_the_lengths():
    """A captured decoding step replays with the lengths and tokens of then; two captured steps with workspaces of
    their own do not disturb each other."""
    H, Hkv, D, page = 8, 2, 128, 64
    g = gen(80)
    c = make_cache([900, 1200], Hkv, D, page, g)
    final = c["lens"].clone()
    c["lens"] -= 5
    q, k, v = (torch.randn((2, 1, n, D), generator=g, device="cuda").to(torch.bfloat16) for n in (H, Hkv, Hkv))
    s = torch.cuda.Stream()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fa.cache_append(k, v, **c)
            outs.append(fa.fwd_cache(q, **c))
        graphs.append(graph)
    while True:
        c["lens"] += 1
        q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
        k.copy_(torch.randn(k.shape, generator=g, device="cuda"))
        torch.cuda.synchronize()
        graphs[0].replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0][0], outs[1][0])
        check(q, c, *outs[0], -1, 0)
        if torch.equal(c["lens"], final):
            break


def test_another_stream():
    g = gen(81)
    c = make_cache([900, 1200], 2, 128, 64, g)
    q = torch.randn((2, 1, 8, 128), generator=g, device="cuda").to(torch.bfloat16)
    want = fa.fwd_cache(q, **c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fa.fwd_cache(q, **c, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_more_than_32_bits_of_bytes():
    """A cache of over 4 GiB of K: the last pages are read and written right."""
    page, Hkv, D = 128, 8, 128
    n = (1 << 32) // (page * Hkv * D) + 40
    g = gen(82)
    c = {"k_pages": torch.zeros((n, Hkv, page, D), dtype=torch.uint8, device="cuda").view(E4M3),
         "v_pages": torch.zeros((n, Hkv, page, D), dtype=torch.uint8, device="cuda").view(E4M3),
         "k_scale": torch.ones((n, Hkv), device="cuda"), "v_scale": torch.ones((n, Hkv), device="cuda"),
         "table": torch.arange(n - 4, n, device="cuda", dtype=torch.int32)[None].contiguous(),
         "lens": torch.tensor([500], dtype=torch.int32, device="cuda")}
    k, v = (torch.randn((1, 500, Hkv, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    fa.cache_append(k, v, **c)
    q = torch.randn((1, 1, 8, D), generator=g, device="cuda").to(torch.bfloat16)
    out, lse = fa.fwd_cache(q, **c)
    check(q, c, out, lse, -1, 0)
    assert not c["k_pages"].view(torch.uint8)[:n - 4].any()


@pytest.mark.parametrize("longest", [300, 6000])
def test_more_sequences_than_threads(longest):
    """The split of the work searches the sequences in blocks: many short ones, without and with long ones between."""
    g = gen(83)
    lens = torch.randint(0, 301, (1000,), generator=g, device="cuda").tolist()
    for b in (0, 383, 384, 767, 768, 999):
        lens[b] = longest
    c = make_cache(lens, 1, 64, 16, g)
    q = torch.randn((1000, 1, 2, 64), generator=g, device="cuda").to(torch.bfloat16)
    out, lse = fa.fwd_cache(q, **c)
    check(q, c, out, lse, -1, 0, only=[0, 1, 2, 100, 382, 383, 384, 385, 500, 767, 768, 769, 998, 999])
    seen = c["lens"] > 0
    assert torch.isfinite(lse[seen]).all() and torch.isneginf(lse[~seen]).all()
    alone = fa.fwd_cache(q[500:501], **{**c, "table": c["table"][500:501].contiguous(), "lens": c["lens"][500:501]})
    assert (out[500] - alone[0][0]).abs().max() <= 2.0 ** -6


def test_more_row_blocks_than_threads():
    g = gen(84)
    c = make_cache([1100, 1500, 1101], 1, 128, 64, g)
    q = torch.randn((3, 1100, 32, 128), generator=g, device="cuda").to(torch.float16)
    out, lse = fa.fwd_cache(q, **c)
    check(q, c, out, lse, -1, 0)


def test_shared_pages_and_two_calls_at_once():
    """Sequences that share a prefix's pages (and one that has a page twice), and two calls on two streams."""
    g = gen(85)
    c = make_cache([1280, 1300, 1500], 2, 128, 64, g)
    c["table"][1, :18] = c["table"][0, :18]
    c["table"][2, 3] = c["table"][2, 2]
    q = torch.randn((3, 2, 8, 128), generator=g, device="cuda").to(torch.bfloat16)
    want = fa.fwd_cache(q, **c)
    check(q, c, *want, -1, 0)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append([fa.fwd_cache(q, **c) for _ in range(3)])
    torch.cuda.synchronize()
    for r in got[0] + got[1]:
        assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1])


def test_one_heavy_token_among_many_light_ones():
    """An attention sink: one key 11 (in the exponent of e) above 20000 equal ones, whose weights together are what
    counts: sum 20000 e^-11 = 0.33 against 1. Both kernels keep weights that small."""
    n, D = 20001, 64
    for Sq, H in ((1, 8), (1, 16), (1, 32), (40, 4)):
        for dtype in (torch.bfloat16, torch.float16):
            page = 64
            m = -(-n // page)
            kp = torch.zeros((m, 1, page, D), device="cuda")
            kp[0, 0, 0, 0] = 1.0
            vp = torch.zeros((m, 1, page, D), device="cuda")
            vp[..., 1] = 1.0
            vp[0, 0, 0, 1] = 0.0
            c = {"k_pages": kp.to(E4M3), "v_pages": vp.to(E4M3), "k_scale": torch.ones((m, 1), device="cuda"),
                 "v_scale": torch.ones((m, 1), device="cuda"),
                 "table": torch.arange(m, device="cuda", dtype=torch.int32)[None].contiguous(),
                 "lens": torch.tensor([n], dtype=torch.int32, device="cuda")}
            q = torch.zeros((1, Sq, H, D), device="cuda", dtype=dtype)
            q[..., 0] = 11.0
            out, lse = fa.fwd_cache(q, **c, scale=1.0)
            light = (n - Sq + torch.arange(Sq, device="cuda")).double() * math.exp(-11.0)
            want = (light / (1 + light))[None, :, None].expand(1, Sq, H)
            # the light weights share one rounding: a step of the last part (2^-9 / 2^4 of a largest weight of at least
            # 2^6) against e^-11 = 2^-15.9 of it is 2^-3.1, half of it 6%; the others' parts are finer
            tol = 0.07 if dtype == torch.bfloat16 and Sq == 1 and H < 32 else 0.03
            assert ((out[..., 1].double() - want).abs() <= tol * want).all(), (Sq, H, dtype)
            assert (lse.double() - (11.0 + torch.log1p(light))).abs().max() <= 1e-3
