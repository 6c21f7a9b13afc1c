"""Plain 64-bit attention with a window, sinks and grouped heads, written from the definition, and its gradients by
the chain rule. Test infrastructure for the operators the fp64 oracle's mask does not cover."""
import math

import torch


def visible(Sq, Sk, causal, window, sinks, device, shift=None):
    """Boolean [Sq, Sk]: key j is visible to query i iff, with c = i + shift (default Sk - Sq) its aligned key,
    (left < 0 or j >= c - left or j < sinks) and (right < 0 or j <= c + right) and (not causal or j <= c)."""
    c = torch.arange(Sq, device=device)[:, None] + (Sk - Sq if shift is None else shift)
    j = torch.arange(Sk, device=device)[None]
    left, right = window
    m = torch.ones((Sq, Sk), dtype=torch.bool, device=device)
    if left >= 0:
        m &= (j >= c - left) | (j < sinks)
    if right >= 0:
        m &= j <= c + right
    if causal:
        m &= j <= c
    return m


def forward(q, k, v, mask, scale=None):
    """One head in float64: q [Sq, D], k, v [Sk, D], mask [Sq, Sk] -> (probabilities, O, LSE)."""
    scale = 1 / math.sqrt(q.shape[1]) if scale is None else scale
    s = (scale * (q @ k.T)).masked_fill(~mask, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(mask, torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None]), 0.0)
    return p, p @ v, lse


def attention(q, k, v, mask_of, scale=None, do=None):
    """[B, Sq, H, D] / [B, Sk, Hkv, D] in float64; mask_of(b) -> [Sq, Sk]. Returns out, lse[, dq, dk, dv]."""
    B, Sq, H, D = q.shape
    group = H // k.shape[2]
    sc = 1 / math.sqrt(D) if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    out, lse = torch.zeros_like(q), torch.zeros((B, H, Sq), dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b in range(B):
        mask = mask_of(b)
        for h in range(H):
            g = h // group
            p, o, ls = forward(q[b, :, h], k[b, :, g], v[b, :, g], mask, scale)
            out[b, :, h], lse[b, h] = o, ls
            if do is not None:
                d = do[b, :, h].double()
                ds = p * (d @ v[b, :, g].T - (d * o).sum(-1, keepdim=True))
                dq[b, :, h] = sc * ds @ k[b, :, g]
                dk[b, :, g] += sc * ds.T @ q[b, :, h]
                dv[b, :, g] += p.T @ d
    return (out, lse) if do is None else (out, lse, dq, dk, dv)
