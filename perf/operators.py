"""What the newest operators of the library are measured by: their cases, inputs, plain forms and exact values.

Three operators that a decoder-only model with bounded memory uses together:

  sink_fwd, sink_train   attention with a sliding window and a few first tokens that stay visible ("sinks"):
                         the forward alone, and a training step's forward and backward.
                         Key j is visible to query i, with c = i + Sk - Sq its aligned key, iff j <= c and
                         (j >= c - left or j < sinks).
  cache_append           new keys and values of a batch of sequences, rounded to e4m3 with one power-of-two scale per
                         page (block of tokens) and head, and written into a paged cache. Sequence b's last
                         counts[b] of T new tokens land at positions lens[b] - counts[b] .. lens[b] - 1. A page's scale
                         is the smallest power of two that brings the largest finite magnitude of the page's
                         tokens to at most 448; a page that holds earlier tokens keeps the larger of its old scale
                         and the new tokens' and its codes move to that scale.
  cache_fwd              attention of Sq new tokens' queries per sequence over that cache (one token: a decoding
                         step; many: a chunk of a prompt), with the same window and sinks; the queries are
                         the last Sq tokens of the sequence.

``own`` chooses between elementary torch operations (False) and the library's kernels (True).
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------------------------ cases
def _sink(name, op, dtype, B, H, Hkv, Sq, Sk, D, left, sinks):
    return dict(name=name, op=op, dtype=dtype, B=B, H=H, Hkv=Hkv, Sq=Sq, Sk=Sk, D=D, left=left, sinks=sinks)


def _cache(name, dtype, B, H, Hkv, Sq, D, page, shortest, longest, left, sinks):
    return dict(name=name, op="cache_fwd", dtype=dtype, B=B, H=H, Hkv=Hkv, Sq=Sq, D=D, page=page, shortest=shortest,
                longest=longest, left=left, sinks=sinks)


def _append(name, dtype, B, Hkv, T, D, page, shortest, longest):
    return dict(name=name, op="cache_append", dtype=dtype, B=B, Hkv=Hkv, T=T, D=D, page=page, shortest=shortest,
                longest=longest)


def listed():
    return [
        # a short, odd-sized document: latency counts
        _sink("sink fwd short", "sink_fwd", "f16", 1, 4, 2, 333, 333, 64, 64, 4),
        # one long document with a window of 2048 and grouped heads: the prompt pass of a streaming model
        _sink("sink fwd long", "sink_fwd", "bf16", 1, 16, 4, 16384, 16384, 128, 2047, 4),
        # fine-tuning on ragged samples, more keys than queries (an earlier chunk is kept), head dim 64
        _sink("sink train odd", "sink_train", "f16", 2, 8, 8, 1000, 1501, 64, 255, 16),
        # pre-training step of a windowed layer
        _sink("sink train large", "sink_train", "bf16", 2, 16, 4, 8192, 8192, 128, 1023, 4),
        # one user, one token, a short conversation: the smallest call
        _cache("decode one short", "bf16", 1, 8, 2, 1, 64, 16, 200, 200, -1, 0),
        # a serving batch with conversations of very different lengths
        _cache("decode ragged", "bf16", 32, 32, 8, 1, 128, 64, 100, 8000, -1, 0),
        # streaming decoding far past the window: only the window and the first tokens are read
        _cache("decode streaming", "f16", 48, 32, 8, 1, 128, 32, 5000, 30000, 4095, 64),
        # a full batch of long contexts: the cache's bandwidth
        _cache("decode large", "bf16", 32, 64, 8, 1, 128, 128, 30000, 32768, -1, 0),
        # a chunk of each prompt against what is cached of it
        _cache("chunk of prompts", "bf16", 2, 32, 8, 512, 128, 64, 3500, 8192, -1, 0),
        # one new token of every sequence of a batch
        _append("append tokens", "bf16", 64, 8, 1, 128, 64, 20, 250),
        # whole prompts of different lengths, padded to the longest
        _append("append prompts", "f16", 8, 8, 1900, 128, 32, 1200, 1900),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sink_fwd", "sink_train", "cache_fwd", "cache_fwd", "cache_append"])
    dtype = rng.choice(["f16", "bf16"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    if op.startswith("sink"):
        group = rng.choice([1, 1, 2, 4])
        B = rng.randint(1, 3)
        H = Hkv * group
        most = 16 * 16384 ** 2 if op == "sink_fwd" else 2 * 16 * 8192 ** 2
        Sk = _log_int(rng, 64, min(16384, int(math.sqrt(most / (B * H)))))
        Sq = Sk if rng.random() < 0.7 else max(1, rng.randint(Sk // 2, Sk))
        c = _sink("", op, dtype, B, H, Hkv, Sq, Sk, D, _log_int(rng, 16, 4096), rng.choice([1, 4, 7, 64, 130]))
    elif op == "cache_fwd":
        H = Hkv * rng.choice([1, 2, 4, 5, 8])
        Sq = 1 if rng.random() < 0.6 else _log_int(rng, 2, 512)
        longest = max(Sq, _log_int(rng, 100, 32768))
        most = min(32 * 8 * 32768 // (Hkv * longest), 2 * 32 * 512 * 8192 // (H * Sq * longest) if Sq > 1 else 64)
        B = _log_int(rng, 1, max(1, min(64, most)))
        window = rng.random() < 0.4
        c = _cache("", dtype, B, H, Hkv, Sq, D, rng.choice([16, 32, 64, 128]), rng.randint(1, longest), longest,
                   _log_int(rng, 16, 4096) if window else -1, rng.choice([0, 4, 50]) if window else 0)
    else:
        T = rng.choice([1, 1, _log_int(rng, 2, 1900)])
        longest = T + _log_int(rng, 1, 300)
        B = _log_int(rng, 1, max(1, min(96, 8 * 8 * 1900 // (Hkv * longest))))
        c = _append("", dtype, B, Hkv, T, D, rng.choice([16, 32, 64, 128]), rng.randint(1, longest), longest)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------------ inputs
def _lengths(case, g):
    """Lengths in tokens, spread over [shortest, longest] with the longest among them."""
    lens = torch.randint(case["shortest"], case["longest"] + 1, (case["B"],), generator=g, device="cuda",
                         dtype=torch.int32)
    lens[0] = case["longest"]
    return lens


def _pages(case, lens, g):
    """A page table with the pages in random order (-1 behind a sequence's last page) and the number of pages."""
    page = case["page"]
    need = (lens.to(torch.int64) + page - 1) // page
    width = (case["longest"] + page - 1) // page
    n = case["B"] * width
    ids = torch.randperm(n, generator=g, device="cuda").to(torch.int32).view(case["B"], width)
    return torch.where(torch.arange(width, device="cuda")[None] < need[:, None], ids, -1).contiguous(), n


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt, op, D = DTYPES[case["dtype"]], case["op"], case["D"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dt)

    s = {"case": case}
    if op.startswith("sink"):
        B, H, Hkv, Sq, Sk = (case[x] for x in ("B", "H", "Hkv", "Sq", "Sk"))
        s.update(q=normal(B, Sq, H, D), k=normal(B, Sk, Hkv, D), v=normal(B, Sk, Hkv, D))
        if op == "sink_train":
            s["do"] = normal(B, Sq, H, D)
        return s
    Hkv, page = case["Hkv"], case["page"]
    lens = _lengths(case, g)
    table, n = _pages(case, lens, g)

    def pool():
        # codes of unit-normal tokens under per-page scales like those an append leaves: amax 2.5 .. 5 of a page
        # times a magnitude of the page and head (outlier heads and tokens), as a power of two
        codes = (torch.randn((n, Hkv, page, D), generator=g, device="cuda") * 64).clamp_(-448, 448).to(E4M3)
        e = torch.randint(-8, -4, (n, Hkv), generator=g, device="cuda")
        return codes, torch.exp2(e.float())

    s["k_pages"], s["k_scale"] = pool()
    s["v_pages"], s["v_scale"] = pool()
    s.update(table=table, lens=lens)
    if op == "cache_fwd":
        s["q"] = normal(case["B"], case["Sq"], case["H"], D)
    else:
        s["k"], s["v"] = normal(case["B"], case["T"], Hkv, D), normal(case["B"], case["T"], Hkv, D)
        s["counts"] = torch.minimum(lens, torch.full_like(lens, case["T"]))
    return s


# -------------------------------------------------------------------------------------------------- plain forms
def _visible(c, keys, left, sinks):
    """Boolean mask from aligned keys c [..., Sq, 1] and key indices [Sk]."""
    m = keys <= c
    return m & ((keys >= c - left) | (keys < sinks)) if left >= 0 else m


def _grouped(x, Hkv):
    """[B, Sq, H, D] -> fp32 [B, Hkv, group * Sq, D] (query head h = hkv * group + its place in the group)."""
    B, Sq, H, D = x.shape
    return x.float().view(B, Sq, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)


def _ungrouped(x, Sq):
    B, Hkv, R, D = x.shape
    return x.view(B, Hkv, R // Sq, Sq, D).permute(0, 3, 1, 2, 4).reshape(B, Sq, Hkv * (R // Sq), D)


def _softmax(s, mask):
    """Masked softmax and log-sum-exp over the last axis; rows without a visible key give zeros and -inf."""
    s = s.masked_fill_(~mask, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = (m + l.log()).squeeze(-1)
    return p.div_(torch.where(l > 0, l, 1.0)), lse


def _plain_sink(s):
    c = s["case"]
    B, Sq, Sk, Hkv, D, group = c["B"], c["Sq"], c["Sk"], c["Hkv"], c["D"], c["H"] // c["Hkv"]
    scale = 1.0 / math.sqrt(D)
    q, k, v = _grouped(s["q"], Hkv), s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)
    keys = torch.arange(Sk, device="cuda")
    mask = _visible((torch.arange(Sq, device="cuda") + Sk - Sq)[:, None], keys, c["left"], c["sinks"])
    mask = mask[None, None, None].expand(B, Hkv, group, Sq, Sk).reshape(B, Hkv, group * Sq, Sk)
    p, lse = _softmax((q @ k.transpose(-1, -2)).mul_(scale), mask)
    del mask
    o = p @ v
    dt = s["q"].dtype
    out = (_ungrouped(o, Sq).to(dt), lse.view(B, c["H"], Sq))
    if c["op"] == "sink_fwd":
        return out
    do = _grouped(s["do"], Hkv)
    dv = p.transpose(-1, -2) @ do
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq, dk = (ds @ k).mul_(scale), (ds.transpose(-1, -2) @ q).mul_(scale)
    return out + (_ungrouped(dq, Sq).to(dt), dk.transpose(1, 2).to(dt).contiguous(),
                  dv.transpose(1, 2).to(dt).contiguous())


def _gathered(pages, scale, table):
    """The cache's values in token order: fp32 [B, Hkv, width * page, D] (zeros where the table has no page)."""
    ids = table.clamp(min=0).long()
    x = pages.view(torch.uint8)[ids].view(E4M3).float() * scale[ids][..., None, None]
    x = torch.where((table >= 0)[:, :, None, None, None], x, 0.0)
    B, W, Hkv, P, D = x.shape
    return x.transpose(1, 2).reshape(B, Hkv, W * P, D)


def _plain_cache_fwd(s):
    c = s["case"]
    B, Sq, Hkv, D, group = c["B"], c["Sq"], c["Hkv"], c["D"], c["H"] // c["Hkv"]
    q = _grouped(s["q"], Hkv)
    k = _gathered(s["k_pages"], s["k_scale"], s["table"])
    aligned = s["lens"].long()[:, None] - Sq + torch.arange(Sq, device="cuda")  # [B, Sq]
    keys = torch.arange(k.shape[2], device="cuda")
    mask = _visible(aligned[:, :, None], keys, c["left"], c["sinks"])  # [B, Sq, keys]
    mask = mask[:, None, None].expand(B, Hkv, group, Sq, len(keys)).reshape(B, Hkv, group * Sq, -1)
    p, lse = _softmax((q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D)), mask)
    del k, mask
    o = p @ _gathered(s["v_pages"], s["v_scale"], s["table"])
    return _ungrouped(o, Sq).to(s["q"].dtype), lse.view(B, c["H"], Sq)


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s, exponent within [-50, 50]."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875), -50).clamp(-50, 50)
    return torch.ldexp(torch.ones_like(amax), e)


def _plain_append(s):
    c = s["case"]
    T, page = c["T"], c["page"]
    lens, counts, table = s["lens"].long(), s["counts"].long(), s["table"].long()
    pos = lens[:, None] - T + torch.arange(T, device="cuda")  # [B, T]
    b, t = torch.nonzero(pos >= (lens - counts)[:, None], as_tuple=True)
    p = pos[b, t]
    pid, slot = table[b, p // page], p % page
    first = lens - counts  # position of the first new token; its page may hold earlier ones
    has = (counts > 0) & (first % page > 0)
    fb = torch.nonzero(has, as_tuple=True)[0]
    old_pid, old_n = table[fb, first[fb] // page], first[fb] % page
    for new, pages, scale in ((s["k"], s["k_pages"], s["k_scale"]), (s["v"], s["v_pages"], s["v_scale"])):
        x = new.float()[b, t]  # [N, Hkv, D]
        amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
        need = torch.zeros_like(scale).index_reduce_(0, pid, amax, "amax")
        want = _pow2_scale(need)
        touched = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda")
        touched[pid] = True
        old = scale.clone()
        want[old_pid] = torch.maximum(want[old_pid], old[old_pid])
        scale.copy_(torch.where(touched[:, None], want, old))
        kept = torch.arange(page, device="cuda")[None, None, :, None] < old_n[:, None, None, None]
        codes = pages.view(torch.uint8)[old_pid].view(E4M3)
        moved = (codes.float() * (old[old_pid] / want[old_pid])[..., None, None]).to(E4M3)
        pages.view(torch.uint8)[old_pid] = torch.where(kept, moved.view(torch.uint8), codes.view(torch.uint8))
        y = (x / want[pid][..., None]).clamp(-448.0, 448.0).to(E4M3)
        pages.view(torch.uint8)[pid, :, slot] = y.view(torch.uint8)
    return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]


# ----------------------------------------------------------------------------------------------------------- run
def run(s):
    c = s["case"]
    if not own:
        return {"sink_fwd": _plain_sink, "sink_train": _plain_sink, "cache_fwd": _plain_cache_fwd,
                "cache_append": _plain_append}[c["op"]](s)
    import exact_io_aware_76_b200 as fa

    if c["op"].startswith("sink"):
        out, lse = fa.fwd(s["q"], s["k"], s["v"], causal=True, window=(c["left"], 0), sinks=c["sinks"])
        if c["op"] == "sink_fwd":
            return out, lse
        grads = fa.bwd(s["q"], s["k"], s["v"], out, lse, s["do"], causal=True, window=(c["left"], 0),
                       sinks=c["sinks"])
        return (out, lse) + tuple(grads)
    cache = (s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
    if c["op"] == "cache_fwd":
        return fa.fwd_cache(s["q"], *cache, s["table"], s["lens"], window_left=c["left"], sinks=c["sinks"])
    fa.cache_append(s["k"], s["v"], *cache, s["table"], s["lens"], counts=s["counts"])
    return cache


# ---------------------------------------------------------------------------------------------------------- work
def _pairs(Sq, Sk, left, sinks):
    """Visible (query, key) pairs of one head."""
    n = 0
    for i in range(Sq):
        c = i + Sk - Sq
        if c >= 0:
            lo = max(0, c - left) if left >= 0 else 0
            n += c + 1 - lo + min(lo, sinks)
    return n


def _mean_len(case):
    return (case["shortest"] + case["longest"]) / 2 + (case["longest"] - case["shortest"]) / (2 * case["B"])


def work(case):
    D, op = case["D"], case["op"]
    if op.startswith("sink"):
        B, H, Hkv, Sq, Sk = (case[x] for x in ("B", "H", "Hkv", "Sq", "Sk"))
        flops = 4.0 * B * H * D * _pairs(Sq, Sk, case["left"], case["sinks"])
        qs, ks, lse = 2.0 * B * Sq * H * D, 2.0 * B * Sk * Hkv * D, 4.0 * B * H * Sq
        if op == "sink_fwd":
            return {"bytes": 2 * qs + 2 * ks + lse, "flops": flops}
        # forward, then q, k, v, out, lse, dout in and dq, dk, dv out; five more products
        return {"bytes": 2 * qs + 2 * ks + lse + 4 * qs + 4 * ks + lse, "flops": 3.5 * flops}
    B, Hkv, page, n = case["B"], case["Hkv"], case["page"], _mean_len(case)
    if op == "cache_append":
        tokens = B * min(n, case["T"])
        return {"bytes": tokens * Hkv * D * 2 * (2.0 + 1.0) + 2 * 4.0 * Hkv * (tokens / page + B), "flops": 0.0}
    H, Sq, left, sinks = case["H"], case["Sq"], case["left"], case["sinks"]
    seen = min(n, left + Sq + sinks) if left >= 0 else n
    per = min(n, left + 1 + sinks) if left >= 0 else max(1.0, n - Sq / 2)
    return {"bytes": B * Hkv * seen * (2.0 * D + 8.0 / page) + 4.0 * B * Sq * H * D + 4.0 * B * H * Sq + 4.0 * B * seen / page,
            "flops": 4.0 * B * H * D * Sq * per}


# --------------------------------------------------------------------------------------------------------- exact
def _exact_head(q, k, v, c0, left, sinks, scale):
    """One head in 64 bits: q [Sq, D], k, v [Sk, D]; query i is aligned with key i + c0."""
    i = torch.arange(q.shape[0], device=q.device)[:, None] + c0
    j = torch.arange(k.shape[0], device=q.device)[None]
    hidden = j > i
    if left >= 0:
        hidden |= (j < i - left) & (j >= sinks)
    w = torch.softmax((scale * q @ k.T).masked_fill(hidden, -1e300), -1).masked_fill(hidden, 0.0)
    lse = torch.logsumexp((scale * q @ k.T).masked_fill(hidden, -math.inf), -1)
    return w, w @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    op, D = case["op"], case["D"]
    if op.startswith("sink"):
        B, H, Hkv, Sq, Sk = (case[x] for x in ("B", "H", "Hkv", "Sq", "Sk"))
        q, k, v = (s[x].double() for x in "qkv")
        scale = D ** -0.5
        out, lse = torch.empty_like(q), torch.empty((B, H, Sq), dtype=torch.float64, device="cuda")
        dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
        for b in range(B):
            for h in range(H):
                g = h // (H // Hkv)
                w, o, ls = _exact_head(q[b, :, h], k[b, :, g], v[b, :, g], Sk - Sq, case["left"], case["sinks"], scale)
                out[b, :, h], lse[b, h] = o, ls
                if op == "sink_train":
                    do = s["do"][b, :, h].double()
                    dw = do @ v[b, :, g].T
                    dz = w * (dw - (w * dw).sum(-1, keepdim=True))
                    dq[b, :, h] = scale * dz @ k[b, :, g]
                    dk[b, :, g] += scale * dz.T @ q[b, :, h]
                    dv[b, :, g] += w.T @ do
        return (out, lse) if op == "sink_fwd" else (out, lse, dq, dk, dv)
    B, Hkv, page = case["B"], case["Hkv"], case["page"]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    if op == "cache_fwd":
        q = s["q"].double()
        Sq, H = case["Sq"], case["H"]
        group = H // Hkv
        out, lse = torch.empty_like(q), torch.empty((B, H, Sq), dtype=torch.float64, device="cuda")
        for b in range(B):
            n = -(-lens[b] // page)
            ids = torch.tensor(table[b][:n], device="cuda")
            for g in range(Hkv):
                k, v = (torch.cat(list((s[x + "_pages"].view(torch.uint8)[ids, g].view(E4M3).double()
                                        * s[x + "_scale"][ids, g].double()[:, None, None])))[:lens[b]] for x in "kv")
                for h in range(g * group, (g + 1) * group):
                    _, o, ls = _exact_head(q[b, :, h], k, v, lens[b] - Sq, case["left"], case["sinks"], D ** -0.5)
                    out[b, :, h], lse[b, h] = o, ls
        return out, lse
    found = []
    for x in "kv":
        pages, scales = s[x + "_pages"].double().cpu(), s[x + "_scale"].double().cpu()
        new, counts = s[x].double().cpu(), s["counts"].tolist()
        for b in range(B):
            start = lens[b] - counts[b]
            for n in range(start // page, -(-lens[b] // page)):
                lo, hi = max(start, n * page), min(lens[b], (n + 1) * page)
                pid, a, z = table[b][n], lo % page, lo % page + hi - lo
                tokens = new[b, case["T"] - lens[b] + lo:case["T"] - lens[b] + hi].transpose(0, 1)  # [Hkv, n, D]
                for h in range(Hkv):
                    biggest = float(tokens[h].abs().max())
                    sc = 2.0 ** -50
                    while sc * 448.0 < biggest:
                        sc *= 2.0
                    if a > 0:
                        sc = max(sc, float(scales[pid, h]))
                        pages[pid, h, :a] = _round_e4m3(pages[pid, h, :a] * (float(scales[pid, h]) / sc))
                    pages[pid, h, a:z] = _round_e4m3(tokens[h] / sc)
                    scales[pid, h] = sc
        found.append((pages, scales))
    return found[0][0], found[1][0], found[0][1], found[1][1]


def _round_e4m3(x):
    """The nearest values of 4 significant bits, exponents -6 .. 8 and steps of 2^-9 below (ties to even)."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(x / step) * step
