"""What is measured of the routing, query/key norm and paged-attention operators.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges, ``prepare``
makes what a user's program has in hand before the call, ``run`` makes one call: the
framework's where ``own`` is true, else the operator's plain form in elementary torch
operations.  ``exact`` computes the same outputs in 64 bits, from the definitions.

The operators (``op``):

  select  routing from logits: scores, selection bias, groups, top-k, gates (``fwd``),
          and the gradient of the logits (``bwd``)
  qk      norm of queries and keys for each head with the position rotation, of a
          Mixture-of-Attention layer's grouped queries and shared keys (``fwd``, ``bwd``)
  append  the same for serving: queries normed and rotated, keys and values stored in a
          paged cache (bf16, or e4m3 codes with a scale per token and head)
  decode  attention of one new token for each sequence over the paged cache
"""
import math

import torch

own = False
DEV = "cuda"
EPS = 1e-6
THETA = 10000.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _select(name, way, T, E, k, score, dtype, bias=True, renorm=True, scale=1.0, groups=1,
            top_groups=1, group_top=2):
    return dict(name=name, op="select", way=way, T=T, E=E, k=k, score=score, dtype=dtype, bias=bias,
                renorm=renorm, scale=scale, groups=groups, top_groups=top_groups,
                group_top=group_top)


def _qk(name, way, T, kslots, q_heads, kv_heads, dh, dtype, interleaved=False):
    return dict(name=name, op="qk", way=way, T=T, kslots=kslots, q_heads=q_heads,
                kv_heads=kv_heads, dh=dh, dtype=dtype, interleaved=interleaved)


def _append(name, B, longest, new, page, kslots, q_heads, kv_heads, dh, cache):
    return dict(name=name, op="append", B=B, longest=longest, new=new, page=page, kslots=kslots,
                q_heads=q_heads, kv_heads=kv_heads, dh=dh, cache=cache)


def _decode(name, B, longest, page, kslots, q_heads, kv_heads, dh, cache, empty=False):
    return dict(name=name, op="decode", B=B, longest=longest, page=page, kslots=kslots,
                q_heads=q_heads, kv_heads=kv_heads, dh=dh, cache=cache, empty=empty)


def listed():
    return [
        # one token of a decode step routed over the fine-grained layer's 64 experts: latency
        _select("select_one_token", "fwd", 1, 64, 8, "sigmoid", "f32", groups=8, top_groups=4,
                scale=2.5),
        # a training batch over many experts in groups, 4 of 8 groups kept
        _select("select_train", "fwd", 16384, 256, 8, "sigmoid", "f32", groups=8, top_groups=4,
                scale=2.5),
        # the gradient of plain softmax gates: dense in the experts
        _select("select_grad", "bwd", 16384, 64, 8, "softmax", "bf16", renorm=False),
        # the Mixture-of-Attention workload's queries and keys (8192 tokens, 4 slots, 4 heads)
        _qk("qk_train", "fwd", 8192, 4, 4, 4, 128, "bf16"),
        _qk("qk_train_grad", "bwd", 8192, 4, 4, 4, 128, "bf16"),
        # odd token count, more query heads than key heads, fp32, pairs side by side
        _qk("qk_odd_grad", "bwd", 1021, 3, 6, 2, 64, "f32", interleaved=True),
        # one new token for each of 37 running sequences
        _append("append_step", 37, 2048, 1, 16, 4, 4, 4, 128, "bf16"),
        # prompts of five sequences written at once to an e4m3 cache
        _append("append_prompt", 5, 2048, 1400, 64, 4, 4, 4, 128, "e4m3"),
        # a single user, one sequence of the workload's length: latency
        _decode("decode_one", 1, 2048, 16, 4, 4, 4, 128, "bf16"),
        # an ordinary ragged batch with small pages and an unused batch row
        _decode("decode_batch", 128, 4096, 16, 4, 4, 4, 128, "bf16", empty=True),
        # long contexts, the largest
        _decode("decode_long", 64, 16384, 64, 4, 4, 4, 128, "bf16"),
        # e4m3 cache, query heads sharing key heads, pages that are no power of two
        _decode("decode_e4m3", 48, 8190, 48, 2, 8, 2, 128, "e4m3"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "qk", "append", "decode", "decode"])
    kslots = rng.choice([1, 2, 3, 4, 6, 8])
    kv_heads = rng.choice([1, 2, 3, 4])
    q_heads = kv_heads * rng.choice([1, 1, 2, 3])
    dh = rng.choice([64, 128, 128])
    if op == "select":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(2, 256 // groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, top_groups * (E // groups)))
        c = _select("", rng.choice(["fwd", "bwd"]), _log(rng, 1, 16384), E, k,
                    rng.choice(["softmax", "sigmoid"]), rng.choice(["f32", "bf16"]),
                    bias=rng.random() < 0.7, renorm=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), groups=groups, top_groups=top_groups,
                    group_top=rng.choice([1, 2]))
    elif op == "qk":
        most = 8192 * 20 * 128 // (dh * (kslots * q_heads + kv_heads))
        c = _qk("", rng.choice(["fwd", "bwd"]), _log(rng, 1, min(8192, most)), kslots, q_heads,
                kv_heads, dh, rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.4)
    else:
        page = rng.choice([1, 7, 16, 16, 32, 48, 64, 100, 256])
        cache = rng.choice(["bf16", "bf16", "e4m3"])
        if op == "append":
            B = _log(rng, 1, 128)
            new = 1 if rng.random() < 0.5 else _log(rng, 1, 8192 // B)
            c = _append("", B, new + rng.randint(0, 500), new, page, kslots, q_heads, kv_heads, dh,
                        cache)
        else:
            B = _log(rng, 1, 256)
            c = _decode("", B, _log(rng, 1, min(65536, 1000000 // B)), page, kslots, q_heads,
                        kv_heads, dh, cache, empty=B > 1 and rng.random() < 0.3)
    del c["name"]
    return c


def _lengths(case):
    """Cached tokens of each sequence, the same for every seed: the longest, then a spread
    over the whole range; an unused batch row (length 0) at the end if the case has one."""
    B, longest = case["B"], case["longest"]
    if case["op"] == "append":
        n = _new(case)
        return [n[b] + int((longest - case["new"]) * ((b * 0.618034) % 1.0)) for b in range(B)]
    out = [longest] + [1 + int((longest - 1) * ((b * 0.618034) % 1.0)) for b in range(1, B)]
    if case["empty"]:
        out[-1] = 0
    return out


def _new(case):
    """New tokens of each sequence of an append: one each, or prompts of several lengths."""
    if case["new"] == 1:
        return [1] * case["B"]
    return [max(1, int(case["new"] * (1.0 - 0.5 * ((b * 0.618034) % 1.0))))
            for b in range(case["B"])]


# ---------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "select":
        T, E, k, es = case["T"], case["E"], case["k"], 4 if case["dtype"] == "f32" else 2
        if case["way"] == "fwd":
            return {"bytes": T * E * es + T * k * 8, "flops": 0}
        scores = not (case["score"] == "softmax" and case["renorm"])
        return {"bytes": T * E * es * (2 if scores else 1) + T * k * 12, "flops": 0}
    width = (case["kslots"] * case["q_heads"] + case["kv_heads"]) * case["dh"]
    if op == "qk":
        es = 4 if case["dtype"] == "f32" else 2
        moved = 2 if case["way"] == "fwd" else 3
        return {"bytes": case["T"] * (moved * width * es + 4 * case["kslots"] + 4), "flops": 0}
    row = case["kv_heads"] * (case["dh"] + 4 if case["cache"] == "e4m3" else 2 * case["dh"])
    G = case["kslots"] * case["q_heads"]
    if op == "append":
        T = sum(_new(case))
        return {"bytes": T * (2 * G * case["dh"] * 2 + 2 * case["kv_heads"] * case["dh"] * 2 + 2 * row),
                "flops": 0}
    keys = sum(_lengths(case))
    rows = case["B"] * G
    return {"bytes": keys * 2 * row + rows * (2 * case["dh"] * 2 + 4),
            "flops": 4.0 * keys * G * case["dh"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dt(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


class _Rand:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)

    def normal(self, shape, dtype=torch.float32, std=1.0, mean=0.0):
        t = torch.randn(shape, generator=self.g, device=DEV)
        return (t * std + mean).to(dtype)

    def perm(self, n):
        return torch.randperm(n, generator=self.g, device=DEV)


def _grouped(r, T, kslots, experts=16):
    """Slots sorted by a random top-k choice of experts: slot t*kslots + j of each grouped row."""
    n = max(experts, kslots)
    pick = torch.rand((T, n), generator=r.g, device=DEV).argsort(1)[:, :kslots]
    return torch.sort(pick.reshape(-1), stable=True).indices.to(torch.int32)


def _inv_freq(dh):
    i = torch.arange(dh // 2, dtype=torch.float64, device=DEV)
    return (THETA ** (-2.0 * i / dh)).float()


def _codes(vals):
    amax = vals.abs().amax(-1)
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / 448.0)
    return (vals / scale[..., None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    r, op = _Rand(seed * 7919 + 13), case["op"]
    s = dict(case=case)
    if op == "select":
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = r.normal((T, E), _dt(case["dtype"]))
        s["bias"] = r.normal((E,), std=0.05) if case["bias"] else None
        if case["way"] == "bwd":  # a training step has these from its forward
            s["idx"], s["gates"] = _select_plain(s)
            s["dgates"] = r.normal((T, k))
        return s
    kslots, q_heads, kv_heads, dh = (case[n] for n in ("kslots", "q_heads", "kv_heads", "dh"))
    s["inv_freq"] = _inv_freq(dh)
    if op != "decode":
        s["wq"], s["wk"] = (r.normal((dh,), std=0.1, mean=1.0) for _ in range(2))
    if op == "qk":
        T, dt = case["T"], _dt(case["dtype"])
        s["slots"] = _grouped(r, T, kslots)
        s["positions"] = (torch.arange(T, device=DEV) % 2048).to(torch.int32)
        s["q"] = r.normal((T * kslots, q_heads * dh), dt)
        s["k"] = r.normal((T, kv_heads * dh), dt)
        if case["way"] == "bwd":
            s["dq"] = r.normal((T * kslots, q_heads * dh), dt)
            s["dk"] = r.normal((T, kv_heads * dh), dt)
        return s
    # paged cache: the pages of the sequences in random order, a few unused ones among them
    B, page = case["B"], case["page"]
    lens = [_lengths(case)[i] for i in r.perm(B).tolist()] if op == "decode" else _lengths(case)
    need = [-(-n // page) for n in lens]
    total = sum(need) + 3
    order = r.perm(total).to(torch.int32)
    table = torch.full((B, max(max(need), 1)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    shape = (total, page, kv_heads, dh)
    for n in ("k_cache", "v_cache"):
        vals = r.normal(shape, torch.bfloat16)
        if case["cache"] == "e4m3":
            spread = 0.5 + torch.rand(shape[:3], generator=r.g, device=DEV)
            codes, s[n[0] + "_scale"] = _codes(vals.float() * spread[..., None])
            vals = codes.view(torch.uint8)
        s[n] = vals
    T = B
    if op == "append":
        new = _new(case)
        T = sum(new)
        if case["new"] > 1:
            s["starts"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32,
                                       device=DEV)
        s["k"] = r.normal((T, kv_heads * dh), torch.bfloat16)
        s["v"] = r.normal((T, kv_heads * dh), torch.bfloat16)
    s["slots"] = _grouped(r, T, kslots)
    s["q"] = r.normal((T * kslots, q_heads * dh), torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import sparse_mixture_experts_smoe_b200 as smoe
    c = s["case"]
    if c["op"] == "select":
        if c["way"] == "fwd":
            return smoe.smoe_route_select(s["logits"], c["k"], s["bias"], score=c["score"],
                                          renorm=c["renorm"], scale=c["scale"], groups=c["groups"],
                                          top_groups=c["top_groups"], group_top=c["group_top"])
        return smoe.smoe_route_select_bwd(s["logits"], s["idx"], s["gates"], s["dgates"],
                                          score=c["score"], renorm=c["renorm"], scale=c["scale"])
    heads = dict(q_heads=c["q_heads"], kv_heads=c["kv_heads"])
    if c["op"] == "qk":
        args = dict(heads, positions=s["positions"], inv_freq=s["inv_freq"], wq=s["wq"], wk=s["wk"],
                    eps=EPS, interleaved=c["interleaved"])
        if c["way"] == "fwd":
            return smoe.smoe_moa_qk_norm_rope_fwd(s["q"], s["k"], s["slots"], c["kslots"], **args)
        return smoe.smoe_moa_qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["slots"],
                                              c["kslots"], **args)
    scales = dict(k_scale=s.get("k_scale"), v_scale=s.get("v_scale"))
    if c["op"] == "append":
        q = smoe.smoe_moa_cache_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"],
                                       s["lens"], s["slots"], c["kslots"], c["q_heads"],
                                       starts=s.get("starts"), inv_freq=s["inv_freq"], wq=s["wq"],
                                       wk=s["wk"], eps=EPS, **scales)
        return _append_out(s, q)
    return smoe.smoe_moa_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                s["slots"], c["kslots"], c["q_heads"], **scales)


def _append_out(s, q):
    if s["case"]["cache"] == "bf16":
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return {"q": q, "k_codes": s["k_cache"].view(torch.float8_e4m3fn),
            "v_codes": s["v_cache"].view(torch.float8_e4m3fn), "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


# ---- plain forms -----------------------------------------------------------
def _plain(s):
    c = s["case"]
    if c["op"] == "select":
        return _select_plain(s) if c["way"] == "fwd" else _select_plain_bwd(s)
    if c["op"] == "qk":
        return _qk_plain(s) if c["way"] == "fwd" else _qk_plain_bwd(s)
    return _append_plain(s) if c["op"] == "append" else _decode_plain(s)


def _select_plain(s):
    # in 64 bits: the choice compares scores that may lie next to one another
    c, l = s["case"], s["logits"].double()
    T, E = l.shape
    p = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
    rank = p if s["bias"] is None else p + s["bias"].double()
    if c["groups"] > 1:
        n = E // c["groups"]
        by = rank.view(T, c["groups"], n)
        best = by.sort(dim=2, descending=True).values[:, :, :c["group_top"]].sum(2)
        keep = best.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        ok = torch.zeros((T, c["groups"]), dtype=torch.bool, device=l.device).scatter_(1, keep, True)
        rank = by.masked_fill(~ok[:, :, None], -math.inf).view(T, E)
    idx = rank.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    g = p.gather(1, idx)
    if c["renorm"]:
        g = g / g.sum(1, keepdim=True)
    return idx.to(torch.int32), (c["scale"] * g).float()


def _select_plain_bwd(s):
    c, l, idx = s["case"], s["logits"].float(), s["idx"].long()
    g, dg = s["gates"], s["dgates"]
    if c["score"] == "softmax" and not c["renorm"]:
        own_part = torch.zeros_like(l).scatter_(1, idx, g * dg)
        dl = own_part - torch.softmax(l, 1) * (g * dg).sum(1, keepdim=True)
    else:
        d = g * (dg - (g * dg).sum(1, keepdim=True) / c["scale"]) if c["renorm"] else g * dg
        if c["score"] == "sigmoid":
            d = d * torch.sigmoid(-l.gather(1, idx))
        dl = torch.zeros_like(l).scatter_(1, idx, d)
    return dl.to(s["logits"].dtype)


def _angles(positions, inv_freq):
    # in 64 bits: the angles of far positions
    a = positions.double()[:, None] * inv_freq.double()
    return a.cos().float()[:, None, :], a.sin().float()[:, None, :]


def _halves(x, interleaved):
    n = x.shape[-1] // 2
    return (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :n], x[..., n:])


def _join(a, b, interleaved):
    return torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)


def _turn(x, cos, sin, interleaved):
    a, b = _halves(x, interleaved)
    return _join(a * cos - b * sin, b * cos + a * sin, interleaved)


def _norm_turn(x, heads, w, positions, inv_freq, interleaved):
    h = x.float().view(x.shape[0], heads, -1)
    u = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * w
    return _turn(u, *_angles(positions, inv_freq), interleaved)


def _norm_turn_bwd(dy, x, heads, w, positions, inv_freq, interleaved):
    h = x.float().view(x.shape[0], heads, -1)
    rstd = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    cos, sin = _angles(positions, inv_freq)
    du = _turn(dy.float().view(h.shape), cos, -sin, interleaved)
    hat = h * rstd
    dw = (du * hat).sum((0, 1))
    dx = rstd * (du * w - hat * (du * w * hat).mean(-1, keepdim=True))
    return dx.reshape(x.shape).to(x.dtype), dw


def _qk_plain(s):
    c = s["case"]
    pos = s["positions"]
    qpos = pos[(s["slots"] // c["kslots"]).long()]
    q = _norm_turn(s["q"], c["q_heads"], s["wq"], qpos, s["inv_freq"], c["interleaved"])
    k = _norm_turn(s["k"], c["kv_heads"], s["wk"], pos, s["inv_freq"], c["interleaved"])
    return q.reshape(s["q"].shape).to(s["q"].dtype), k.reshape(s["k"].shape).to(s["k"].dtype)


def _qk_plain_bwd(s):
    c = s["case"]
    pos = s["positions"]
    qpos = pos[(s["slots"] // c["kslots"]).long()]
    dq, dwq = _norm_turn_bwd(s["dq"], s["q"], c["q_heads"], s["wq"], qpos, s["inv_freq"],
                             c["interleaved"])
    dk, dwk = _norm_turn_bwd(s["dk"], s["k"], c["kv_heads"], s["wk"], pos, s["inv_freq"],
                             c["interleaved"])
    return dq, dk, dwq, dwk


def _append_plain(s):
    c = s["case"]
    T, page = s["k"].shape[0], c["page"]
    row = torch.arange(T, device=DEV)
    if "starts" in s:
        starts = s["starts"].long()
        seq = torch.searchsorted(starts, row, right=True) - 1
        pos = s["lens"].long()[seq] - starts[seq + 1] + row
    else:
        seq, pos = row, s["lens"].long() - 1
    qpos = pos[(s["slots"] // c["kslots"]).long()]
    q = _norm_turn(s["q"], c["q_heads"], s["wq"], qpos, s["inv_freq"], False)
    k = _norm_turn(s["k"], c["kv_heads"], s["wk"], pos, s["inv_freq"], False)
    v = s["v"].float().view(k.shape)
    at = (s["table"][seq, pos // page].long(), pos % page)
    if c["cache"] == "bf16":
        s["k_cache"][at] = k.to(torch.bfloat16)
        s["v_cache"][at] = v.to(torch.bfloat16)
    else:
        kc, ks = _codes(k)
        vc, vs = _codes(v)
        s["k_cache"][at], s["k_scale"][at] = kc.view(torch.uint8), ks
        s["v_cache"][at], s["v_scale"][at] = vc.view(torch.uint8), vs
    return _append_out(s, q.reshape(s["q"].shape).to(torch.bfloat16))


def _rows(s, n, at):
    x = s[n][at]
    if s["case"]["cache"] == "e4m3":
        return x.view(torch.float8_e4m3fn).float() * s[n[0] + "_scale"][at][..., None]
    return x.float()


def _decode_plain(s):
    c = s["case"]
    B, page, ks, qh, kvh, dh = (c[n] for n in ("B", "page", "kslots", "q_heads", "kv_heads", "dh"))
    place = torch.arange(c["longest"], device=DEV)
    at = (s["table"][:, place // page].clamp(min=0).long(), (place % page).expand(B, -1))
    K, V = _rows(s, "k_cache", at), _rows(s, "v_cache", at)  # [B, L, kvh, dh]
    q = torch.empty_like(s["q"])
    q[s["slots"].long()] = s["q"]  # to token order
    q = q.float().view(B, ks, kvh, qh // kvh, dh).permute(0, 2, 1, 3, 4).reshape(B, kvh, -1, dh)
    sc = torch.matmul(q, K.permute(0, 2, 3, 1)) / math.sqrt(dh)  # [B, kvh, G, L]
    seen = place < s["lens"][:, None]
    sc.masked_fill_(~seen[:, None, None, :], -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(sc - top)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, V.permute(0, 2, 1, 3)) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (torch.log(total) + top)[..., 0]

    def out(x, *tail):
        x = x.view(B, kvh, ks, qh // kvh, *tail).transpose(1, 2).reshape(B * ks, -1)
        return x[s["slots"].long()]

    return out(o, dh).to(torch.bfloat16), out(lse)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "select":
        return _select_exact(s)
    if case["op"] == "qk":
        return _qk_exact(s)
    return _append_exact(s) if case["op"] == "append" else _decode_exact(s)


def _gates_exact(c, l, idx):
    """Gates of the chosen experts as a function of the logits, for autograd as well."""
    p = 1.0 / (1.0 + torch.exp(-l)) if c["score"] == "sigmoid" else torch.exp(
        l - torch.logsumexp(l, 1, keepdim=True))
    g = torch.stack([p[torch.arange(l.shape[0], device=l.device), idx[:, j]]
                     for j in range(idx.shape[1])], 1)
    return c["scale"] * (g / g.sum(1, keepdim=True) if c["renorm"] else g)


def _select_exact(s):
    c, l = s["case"], s["logits"].double()
    if c["way"] == "bwd":
        l.requires_grad_(True)
        (_gates_exact(c, l, s["idx"].long()) * s["dgates"].double()).sum().backward()
        return l.grad
    T, E = l.shape
    p = 1.0 / (1.0 + torch.exp(-l)) if c["score"] == "sigmoid" else torch.exp(
        l - torch.logsumexp(l, 1, keepdim=True))
    rank = p + (0.0 if s["bias"] is None else s["bias"].double())
    lane = torch.arange(T, device=l.device)
    if c["groups"] > 1:
        by = rank.view(T, c["groups"], -1)
        m = by.amax(2)
        score = m
        if c["group_top"] == 2:
            rest = by.scatter(2, by.argmax(2, keepdim=True), -math.inf)
            score = m + rest.amax(2)
        open_ = torch.zeros_like(score, dtype=torch.bool)
        for _ in range(c["top_groups"]):
            best = (score == score.amax(1, keepdim=True)).int().argmax(1)
            open_[lane, best] = True
            score[lane, best] = -math.inf
        rank = torch.where(open_[:, :, None], by, torch.full_like(by, -math.inf)).view(T, E)
    rank = rank.clone()
    idx = []
    for _ in range(c["k"]):
        best = (rank == rank.amax(1, keepdim=True)).int().argmax(1)  # the lowest of equals
        idx.append(best)
        rank[lane, best] = -math.inf
    idx = torch.stack(idx, 1)
    return idx.to(torch.int32), _gates_exact(c, l, idx)


def _head_exact(x, w, pos, inv_freq, interleaved):
    """One head's rows [R, dh] in 64 bits, as complex numbers turned by their angles."""
    u = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w
    n = x.shape[-1] // 2
    z = torch.complex(u[:, 0::2], u[:, 1::2]) if interleaved else torch.complex(u[:, :n], u[:, n:])
    z = z * torch.polar(torch.ones_like(z.real), pos.double()[:, None] * inv_freq.double())
    if interleaved:
        return torch.view_as_real(z).reshape(x.shape)
    return torch.cat((z.real, z.imag), -1)


def _rows_exact(x, heads, w, pos, inv_freq, interleaved):
    dh = w.numel()
    return torch.cat([_head_exact(x[:, h * dh:(h + 1) * dh], w, pos, inv_freq, interleaved)
                      for h in range(heads)], 1)


def _qk_exact(s):
    c = s["case"]
    leaves = [s[n].double().requires_grad_(True) for n in ("q", "k", "wq", "wk")]
    q, k, wq, wk = leaves
    qpos = s["positions"][torch.div(s["slots"], c["kslots"], rounding_mode="floor").long()]
    yq = _rows_exact(q, c["q_heads"], wq, qpos, s["inv_freq"], c["interleaved"])
    yk = _rows_exact(k, c["kv_heads"], wk, s["positions"], s["inv_freq"], c["interleaved"])
    if c["way"] == "fwd":
        return yq, yk
    return list(torch.autograd.grad([yq, yk], leaves, [s["dq"].double(), s["dk"].double()]))


def _append_exact(s):
    c = s["case"]
    lens, new = s["lens"].tolist(), _new(c)
    pos = torch.cat([torch.arange(n - m, n, device=DEV) for n, m in zip(lens, new)])
    seq = torch.cat([torch.full((m,), b, device=DEV) for b, m in enumerate(new)])
    qpos = pos[torch.div(s["slots"], c["kslots"], rounding_mode="floor").long()]
    q = _rows_exact(s["q"].double(), c["q_heads"], s["wq"].double(), qpos, s["inv_freq"], False)
    k = _rows_exact(s["k"].double(), c["kv_heads"], s["wk"].double(), pos, s["inv_freq"], False)
    k = k.view(-1, c["kv_heads"], c["dh"])
    v = s["v"].double().view(k.shape)
    flat = s["table"].long()[seq, pos // c["page"]] * c["page"] + pos % c["page"]

    def stored(old, rows):
        out = old.double().flatten(0, 1)
        out[flat] = rows
        return out.view(old.shape)

    if c["cache"] == "bf16":
        return {"q": q, "k_cache": stored(s["k_cache"], k), "v_cache": stored(s["v_cache"], v)}
    return {"q": q, "k_codes": None, "v_codes": None,
            "k_scale": stored(s["k_scale"], k.abs().amax(-1) / 448.0),
            "v_scale": stored(s["v_scale"], v.abs().amax(-1) / 448.0)}


def _decode_exact(s):
    c = s["case"]
    B, page, ks, qh, kvh, dh = (c[n] for n in ("B", "page", "kslots", "q_heads", "kv_heads", "dh"))
    row_of = torch.empty(B * ks, dtype=torch.long, device=DEV)
    row_of[s["slots"].long()] = torch.arange(B * ks, device=DEV)
    o = torch.zeros((B * ks, qh, dh), dtype=torch.float64, device=DEV)
    lse = torch.full((B * ks, qh), -math.inf, dtype=torch.float64, device=DEV)
    head = torch.arange(qh, device=DEV) // (qh // kvh)
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        u = torch.arange(n, device=DEV)
        at = (s["table"][b].long()[u // page], u % page)

        def rows(name):
            x = s[name][at]
            if c["cache"] == "e4m3":
                return x.view(torch.float8_e4m3fn).double() * s[name[0] + "_scale"][at].double()[..., None]
            return x.double()

        K, V = rows("k_cache")[:, head], rows("v_cache")[:, head]  # [n, qh, dh]
        mine = row_of[b * ks:(b + 1) * ks]
        q = s["q"][mine].double().view(ks, qh, dh)
        sc = torch.einsum("jhd,uhd->jhu", q, K) / dh ** 0.5
        z = torch.logsumexp(sc, -1, keepdim=True)
        o[mine] = torch.einsum("jhu,uhd->jhd", torch.exp(sc - z), V)
        lse[mine] = z[..., 0]
    return o.view(B * ks, qh * dh), lse
