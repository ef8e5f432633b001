"""Plain forms, in 64 bits on the CPU, of routing from logits, of the query/key norm with
rotation and of decode attention over a paged cache (tests only; no code is shared with
the library)."""
import math

import torch

NEG = -math.inf
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def scores(logits, score):
    """(scores, usable) in 64 bits: -inf and NaN logits are not usable, +inf is the largest finite."""
    usable = logits.float() > NEG
    l = logits.float().clamp(max=torch.finfo(torch.float32).max).double()
    l = torch.where(usable, l, torch.zeros_like(l))
    if score == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        m = torch.where(usable, l, torch.full_like(l, NEG)).amax(1, keepdim=True)
        m = torch.where(m == NEG, torch.zeros_like(m), m)
        e = torch.where(usable, torch.exp(l - m), torch.zeros_like(l))
        z = e.sum(1, keepdim=True)
        s = e / torch.where(z == 0, torch.ones_like(z), z)
    return torch.where(usable, s, torch.zeros_like(s)), usable, l


def select(logits, k, bias, score, renorm, scale, groups, top_groups, group_top):
    logits = logits.cpu()
    T, E = logits.shape
    s, usable, l = scores(logits, score)
    b = torch.zeros(E) if bias is None else bias.cpu().float()
    ok = usable & (b > NEG)
    c = torch.where(ok, s + b.double(), torch.full_like(s, NEG))
    rank = c if bias is not None else torch.where(ok, l, torch.full_like(l, NEG))
    idx = torch.zeros((T, k), dtype=torch.int32)
    n = E // groups
    for t in range(T):
        cand = list(range(E))
        if groups > 1:
            gs = []
            for g in range(groups):
                best = sorted(c[t, g * n:(g + 1) * n].tolist(), reverse=True)[:group_top]
                gs.append(sum(v for v in best if v > NEG) if best[0] > NEG else NEG)
            keep = sorted(range(groups), key=lambda g: (-gs[g], g))[:top_groups]
            cand = [e for e in cand if e // n in keep]
        row = rank[t].tolist()
        idx[t] = torch.tensor(sorted(cand, key=lambda e: (-row[e], e))[:k])
    return idx, gates_of(logits, idx, bias, score, renorm, scale)


def _shift(l):
    """Largest finite value of each row (0 without one), a constant of the derivative."""
    m = l.detach().amax(1, keepdim=True)
    return torch.where(m == NEG, torch.zeros_like(m), m)


def gates_of(logits, idx, bias, score, renorm, scale):
    """Gates of given ids (differentiable in fp64 logits)."""
    i = idx.long()
    ok = (logits.gather(1, i) > NEG)
    if bias is not None:
        ok = ok & (bias.cpu()[i] > NEG)
    l = logits.double().clamp(max=torch.finfo(torch.float32).max)
    lsel = torch.where(ok, l.gather(1, i), torch.full_like(l.gather(1, i), NEG))
    if score == "sigmoid":
        ls = torch.nn.functional.logsigmoid(lsel)
    elif renorm:  # the row's denominator cancels; the shift keeps 2^128 + log 2 apart from 2^128
        ls = lsel - _shift(lsel)
    else:
        usable = logits > NEG
        u = torch.where(usable, l, torch.full_like(l, NEG))
        den = torch.logsumexp(u - _shift(u), 1, keepdim=True)
        ls = lsel - _shift(u) - torch.where(den == NEG, torch.zeros_like(den), den)
    if renorm:
        z = torch.logsumexp(ls, 1, keepdim=True)
        ls = ls - torch.where(z == NEG, torch.zeros_like(z), z)
    return scale * torch.exp(ls)


def turn(x, pos, inv_freq, interleaved, back=False):
    """Rotate rows x [R, heads, dh] (fp64) by pos [R] * inv_freq."""
    if inv_freq is None:
        return x
    t = pos.double()[:, None, None] * inv_freq.cpu().double()
    c, s = torch.cos(t), torch.sin(t) * (-1 if back else 1)
    n = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :n], x[..., n:])
    ya, yb = a * c - b * s, b * c + a * s
    return torch.stack((ya, yb), -1).flatten(-2) if interleaved else torch.cat((ya, yb), -1)


def norm_turn(x, w, pos, inv_freq, interleaved, eps, norm):
    """x [R, heads, dh] fp64 -> y."""
    u = x
    if norm:
        u = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if w is not None:
            u = u * w
    return turn(u, pos, inv_freq, interleaved)


def pair_size(y, interleaved):
    """|y_a| + |y_b| of each value's pair: what a rotation's fp32 errors go by."""
    n = y.shape[-1] // 2
    a = y.abs()
    if interleaved:
        s = a[..., 0::2] + a[..., 1::2]
        return torch.stack((s, s), -1).flatten(-2)
    s = a[..., :n] + a[..., n:]
    return torch.cat((s, s), -1)


def decode(q, k_cache, v_cache, table, lens, sorted_slot, kslots, q_heads):
    """q [B*kslots, q_heads*dh]; caches [pages, page, kvh, dh] as real values.  Returns (o, lse, sum p|v|)."""
    B, (pages, page, kvh, dh) = len(lens), k_cache.shape
    group = q_heads // kvh
    rows = B * kslots
    o = torch.zeros((rows, q_heads, dh), dtype=torch.float64)
    size = torch.zeros_like(o)
    lse = torch.full((rows, q_heads), NEG, dtype=torch.float64)
    slot = torch.arange(rows) if sorted_slot is None else sorted_slot.cpu().long()
    kd, vd, qd = k_cache.double(), v_cache.double(), q.cpu().double().view(rows, q_heads, dh)
    held = {}  # keys and values of a sequence
    for i in range(rows):
        b = int(slot[i]) // kslots
        if b not in held:
            n = min(max(int(lens[b]), 0), table.shape[1] * page)
            u = torch.arange(n)
            p_, f_ = table[b][u // page].long(), u % page
            there = (p_ >= 0) & (p_ < pages)
            held[b] = kd[p_[there], f_[there]], vd[p_[there], f_[there]]  # [n, kvh, dh]
        K, V = held[b]
        if K.shape[0] == 0:
            continue
        for h in range(q_heads):
            sc = K[:, h // group] @ qd[i, h] / math.sqrt(dh)
            z = torch.logsumexp(sc, 0)
            w = torch.exp(sc - z)
            o[i, h] = w @ V[:, h // group]
            size[i, h] = w @ V[:, h // group].abs()
            lse[i, h] = z
    return o.view(rows, -1), lse, size.view(rows, -1)
