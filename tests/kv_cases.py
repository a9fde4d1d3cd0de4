"""Paged caches for the tests and a plain 64-bit attention over them.

Slots of pages that hold no token, and pages that no sequence holds, are filled
with NaN (bf16; the scales of int8 codes), so that a kernel that lets them in
shows it.
"""
import math

import torch

U = 2.0 ** -24  # unit roundoff of fp32
U16 = 2.0 ** -8  # of bf16: half a unit in the last of its 8 significant bits


def make_cache(w4, lens, heads, ps, D, kv, seed, layers=1, spare=3, W=None, device="cuda",
               pages=None):
    """(cache, table, lens tensor, K, V): K[b], V[b] float64 [len, heads, D] hold
    the cached values of layer `layers - 1`."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // ps) for n in lens]
    W = W or max(max(need), 1) + 1
    used = sum(need)
    pages = pages or used + spare
    shape = (layers, pages, heads, ps, D)
    order = torch.randperm(pages, generator=g)[:used] if pages < 1 << 20 else torch.arange(used)
    if pages > used + spare:  # a large pool: the last pages, at the largest offsets
        order = pages - 1 - torch.randperm(used, generator=g)
    table = torch.full((len(lens), W), -1, dtype=torch.int32)
    dt = torch.bfloat16 if kv == "bf16" else torch.int8
    cache = w4.KVCache.empty(layers, pages, heads, ps, D, dt, device)
    small = pages <= used + spare
    if kv == "bf16" and small:
        cache.k.fill_(math.nan)
        cache.v.fill_(math.nan)
    elif kv != "bf16" and small:
        cache.k.fill_(113)
        cache.v.fill_(-77)
        cache.k_scale.fill_(math.nan)
        cache.v_scale.fill_(math.nan)
    K, V, at = [], [], 0
    for b, n in enumerate(lens):
        ids = order[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = ids.int()
        kvd = []
        for pool, scales in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            x = torch.randn((n, heads, D), generator=g)
            if n > 2:
                x[n // 2] *= 6.0  # a token that stands out
            pad = need[b] * ps - n
            if kv == "bf16":
                c = x.bfloat16()
                kvd.append(c.double())
                full = torch.cat([c, torch.full((pad, heads, D), math.nan).bfloat16()])
                pool[layers - 1, ids.to(device)] = full.view(-1, ps, heads, D).transpose(1, 2).to(device)
            else:
                s = x.abs().amax(-1) / 127
                c = torch.round(x / s[..., None]).clamp(-128, 127)
                kvd.append((c.double() * s.double()[..., None]))
                full = torch.cat([c.to(torch.int8), torch.full((pad, heads, D), 99, dtype=torch.int8)])
                fs = torch.cat([s, torch.full((pad, heads), math.nan)])
                pool[layers - 1, ids.to(device)] = full.view(-1, ps, heads, D).transpose(1, 2).to(device)
                scales[layers - 1, ids.to(device)] = fs.view(-1, ps, heads).transpose(1, 2).to(device)
        K.append(kvd[0])
        V.append(kvd[1])
    return cache, table.to(device), torch.tensor(lens, dtype=torch.int32, device=device), K, V


def attend(q, K, V, pos, window, sinks, scale, hole=None):
    """(out, bound): float64 attention of q [n, hq, D] at positions pos [n] over
    K, V [len, heads, D], and per element the error that a kernel with fp32
    scores, softmax and sums may have:

      score error  e_j = (D + 8) U sum_d |q_d k_jd| scale + 8 U (|s_j| + |m|)
                   (D products and sums, the scale factors, the exponent's
                   argument),
      exp          4 U relative (argument's last step and the exponential),
      sums         (n + 64) U relative, in any order with rescaling,
      so |err| <= (2 max_j e_j + (2 n + 136) U) sum_j p_j |v_j| / sum_j p_j.
    hole: tokens [len] (bool) that have no page."""
    n, hq, D = q.shape
    L, heads, _ = K.shape
    q = q.double().cpu()
    out = torch.zeros((n, hq, D), dtype=torch.float64)
    mean = torch.zeros_like(out)
    rel = torch.zeros((n, hq, 1), dtype=torch.float64)
    if L == 0:
        return out, rel * 0, mean
    j = torch.arange(L)
    pos = torch.as_tensor(pos)[:, None]
    see = j <= pos
    if window:
        see = see & ((j > pos - window) | (j < sinks))
    if hole is not None:
        see = see & ~hole
    G = hq // heads
    for h in range(hq):
        k, v, qh = K[:, h // G], V[:, h // G], q[:, h]
        s = torch.where(see, qh @ k.T * scale, -math.inf)
        sa = torch.where(see, qh.abs() @ k.abs().T * abs(scale), 0.0)
        m = s.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, 0.0, m)
        p = torch.exp(s - m)
        tot = p.sum(-1, keepdim=True)
        tot = torch.where(tot == 0, 1.0, tot)
        out[:, h] = p @ v / tot
        mean[:, h] = p @ v.abs() / tot
        e = (D + 8) * U * sa + 8 * U * (torch.where(see, s, 0.0).abs() + m.abs())
        rel[:, h] = 2 * e.amax(-1, keepdim=True) + (2 * L + 136) * U
    return out, rel, mean


def close(y, out, rel, mean, p_rounded=False):
    """Whether y is within the bound: fp32 `rel` of the mean |v|; bf16 outputs
    add their own rounding, and softmax weights rounded to bf16 (their sum taken
    after the rounding) U16 of the mean |v| from the product and the rounded
    weights' normalization alike."""
    if y.numel() == 0:
        return True, (0.0, 0)
    tol = rel * mean
    if p_rounded:
        tol = tol + 2 * U16 * mean
    if y.dtype == torch.bfloat16:
        tol = tol + U16 * (out.abs() + tol)
    d = (y.double().cpu() - out).abs()
    bad = ~(d <= tol + 1e-30)
    return not bad.any(), (float((d / (tol + 1e-30)).nan_to_num(1e9).max()), int(bad.sum()))
