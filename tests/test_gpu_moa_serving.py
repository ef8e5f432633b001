"""The operators together, as a Mixture-of-Attention layer uses them: routing from logits,
expert sort, per-expert projections, query/key norm with rotation, and attention, token by
token over a paged cache and as the training form over whole sequences."""
import math

import pytest
import torch

import sparse_mixture_experts_smoe_b200 as smoe

from . import _plain_ops as plain

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
E, KS, H, DH, D = 6, 2, 2, 128, 64  # experts, slots, heads, head size, model width
W = H * DH


def _layer(seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: (std * torch.randn(*s, generator=g))  # noqa: E731
    p = dict(wr=r(D, E, std=0.3).cuda(), bias=r(E, std=0.05).cuda(),
             wq=r(E, D, W, std=D ** -0.5).to(BF).cuda(), wk=r(D, W, std=D ** -0.5).to(BF).cuda(),
             wv=r(D, W, std=D ** -0.5).to(BF).cuda(), wo=r(E, W, D, std=W ** -0.5).to(BF).cuda(),
             nq=(1 + r(DH, std=0.1)).cuda(), nk=(1 + r(DH, std=0.1)).cuda())
    p["freq"] = (10000.0 ** (-2.0 * torch.arange(DH // 2, dtype=torch.float64) / DH)).float().cuda()
    return p


def _project(p, x):
    idx, gates = smoe.smoe_route_select(x.float() @ p["wr"], KS, p["bias"], score="sigmoid", scale=1.5)
    ss, off = smoe.smoe_sort(idx, E)
    q = smoe.parallel_linear_fwd(x, p["wq"], ss, off, KS, 0, 1)
    return gates, ss, off, q, x @ p["wk"], x @ p["wv"]


def _output(p, o, gates, ss, off):
    return smoe.parallel_linear_fwd(o, p["wo"], ss, off, 1, 1, 0, gates=gates.reshape(-1), combine_k=KS)


def _cache(pages, page, f8):
    mk = lambda: torch.zeros(pages, page, H, DH, dtype=torch.uint8 if f8 else BF, device="cuda")  # noqa: E731
    sc = [torch.ones(pages, page, H, device="cuda") for _ in range(2)] if f8 else [None, None]
    return mk(), mk(), dict(k_scale=sc[0], v_scale=sc[1])


@pytest.mark.parametrize("f8", [False, True])
def test_prompt_then_tokens(f8):
    """Prompts written at once, then three tokens one at a time, against the training form
    over the whole sequences.  Queries and bf16 keys are the same bits; the two attentions
    round their weights and outputs to bf16 each (e4m3 keys and values are 2^-4 off)."""
    B, L, new, page = 3, 45, 3, 16
    p = _layer(1)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(B, L, D, generator=g).to(BF).cuda()
    # training form: whole sequences
    gates, ss, off, q, k, v = _project(p, x.view(B * L, D))
    pos = torch.arange(L, device="cuda").repeat(B).int()
    qn, kn = smoe.smoe_moa_qk_norm_rope_fwd(q, k, ss, KS, q_heads=H, kv_heads=H, positions=pos,
                                            inv_freq=p["freq"], wq=p["nq"], wk=p["nk"])
    o, lse = smoe.smoe_moa_attn_fwd(qn, kn, v, ss, KS, L, H)
    y = _output(p, o, gates, ss, off).view(B, L, D)
    inv = torch.empty(B * L * KS, dtype=torch.long, device="cuda")
    inv[ss.long()] = torch.arange(B * L * KS, device="cuda")
    # serving form
    kc, vc, sc = _cache(B * 4, page, f8)
    table = torch.randperm(B * 4, generator=g).int().view(B, 4).cuda()
    kw = dict(inv_freq=p["freq"], wq=p["nq"], wk=p["nk"], **sc)
    n0 = L - new
    xp = x[:, :n0].reshape(B * n0, D)
    starts = torch.arange(0, B * n0 + 1, n0, device="cuda").int()
    lens = torch.full((B,), n0, dtype=torch.int32, device="cuda")
    _, ss1, _, q1, k1, v1 = _project(p, xp)
    smoe.smoe_moa_cache_append(q1, k1, v1, kc, vc, table, lens, ss1, KS, H, starts=starts, **kw)
    for t in range(n0, L):
        lens += 1
        g1, ss1, off1, q1, k1, v1 = _project(p, x[:, t].contiguous())
        q1 = smoe.smoe_moa_cache_append(q1, k1, v1, kc, vc, table, lens, ss1, KS, H, **kw)
        o1, lse1 = smoe.smoe_moa_decode(q1, kc, vc, table, lens, ss1, KS, H, **sc)
        y1 = _output(p, o1, g1, ss1, off1)
        assert smoe.smoe_check() == 0
        for i in range(B * KS):
            s = int(ss1[i])
            j = int(inv[(s // KS * L + t) * KS + s % KS])  # the row of the training form
            if not f8:
                assert torch.equal(q1[i], qn[j])
            a, b = o1[i].double(), o[j].double()
            vmax = v.view(B, L, W)[s // KS, :t + 1].double().abs().amax()
            # both: weights and outputs rounded by 2^-8; e4m3: values by 2^-4, and scores by
            # 2^-4 of sum |q k| / sqrt(dh), which bounds the weights' change
            size = vmax * (4 * 2.0 ** -8 if not f8 else 2.0 ** -1)
            assert ((a - b).abs() <= size).all()
            if not f8:
                assert ((lse1[i] - lse[j]).abs() <= 2.0 ** -13 * (1 + lse[j].abs())).all()
        assert (y1 - y[:, t]).abs().max() <= (0.05 if not f8 else 0.5) * y.abs().max()


def test_layer_in_one_graph():
    """A decode step captured once and replayed with new inputs, as a server runs it."""
    B, page = 5, 16
    p = _layer(3)
    g = torch.Generator().manual_seed(4)
    kc, vc, sc = _cache(B * 3, page, True)
    table = torch.arange(B * 3, dtype=torch.int32, device="cuda").view(B, 3)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    x = torch.zeros(B, D, dtype=BF, device="cuda")

    def step(caches, n):
        gates, ss, off, q, k, v = _project(p, x)
        q = smoe.smoe_moa_cache_append(q, k, v, caches[0], caches[1], table, n, ss, KS, H,
                                       inv_freq=p["freq"], wq=p["nq"], wk=p["nk"], **caches[2])
        o, lse = smoe.smoe_moa_decode(q, caches[0], caches[1], table, n, ss, KS, H, **caches[2])
        return _output(p, o, gates, ss, off), lse

    lens += 1
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step((kc.clone(), vc.clone(), {n: t.clone() for n, t in sc.items()}), lens)
    torch.cuda.current_stream().wait_stream(st)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        y, lse = step((kc, vc, sc), lens)
    mine = (kc.clone(), vc.clone(), {n: t.clone() for n, t in sc.items()})
    lens.zero_()
    for _ in range(20):
        lens += 1
        x.copy_(torch.randn(B, D, generator=g).to(BF))
        gr.replay()
        y2, lse2 = step(mine, lens)
        assert torch.equal(y, y2) and torch.equal(lse, lse2)
    assert smoe.smoe_check() == 0 and torch.equal(kc, mine[0]) and torch.equal(vc, mine[1])


def test_gradients_of_the_layer():
    """Routing, norm, attention and projections backward in fp32 and bf16 steps, against
    autograd of the plain forms in 64 bits, from the same upstream gradients: each step's
    gradients within that step's roundings."""
    B, L = 2, 33
    T = B * L
    p = _layer(5)
    g = torch.Generator().manual_seed(6)
    x = torch.randn(T, D, generator=g).to(BF).cuda()
    logits = x.float() @ p["wr"]
    idx, gates = smoe.smoe_route_select(logits, KS, p["bias"], score="sigmoid", scale=1.5)
    ss, off = smoe.smoe_sort(idx, E)
    o = torch.randn(T * KS, W, generator=g).to(BF).cuda()  # grouped rows of an attention
    dy = torch.randn(T, D, generator=g).to(BF).cuda()
    do, dwo, dgates = smoe.parallel_linear_bwd(dy, o, p["wo"], ss, off, 1, 1, 0, gates=gates.reshape(-1),
                                               combine_k=KS, want_dgates=True)
    dl = smoe.smoe_route_select_bwd(logits, idx, gates, dgates.view(T, KS), score="sigmoid", scale=1.5)
    assert smoe.smoe_check() == 0
    l64 = logits.cpu().double().requires_grad_(True)
    gates64 = plain.gates_of(l64, idx.cpu(), p["bias"].cpu(), "sigmoid", True, 1.5)
    slot = ss.cpu().long()
    token = slot // KS
    prod = torch.einsum("sw,swd->sd", o.cpu().double(), p["wo"].cpu().double()[idx.cpu().flatten()[slot].long()])
    rows = gates64.flatten()[slot][:, None] * prod
    y = torch.zeros(T, D, dtype=torch.float64).index_add(0, token, rows)
    ref, = torch.autograd.grad((y * dy.cpu().double()).sum(), l64)
    # dgate is a sum of D products of dy and the expert product, which is rounded to bf16
    gd = torch.zeros(T * KS, dtype=torch.float64)
    gd[slot] = (prod.abs() * dy.cpu().double()[token].abs()).sum(1)
    gd = gd.view(T, KS)
    g64 = gates64.detach()
    size = torch.zeros(T, E, dtype=torch.float64).scatter_(
        1, idx.cpu().long(), g64 * (gd + (g64 * gd).sum(1, keepdim=True) / 1.5))
    assert ((dl.cpu().double() - ref).abs() <= 2.0 ** -7 * size).all()
    # queries and keys: norm and rotation backward after the attention's own backward
    pos = torch.arange(L, device="cuda").repeat(B).int()
    q = torch.randn(T * KS, W, generator=g).to(BF).cuda()
    k, v = (torch.randn(T, W, generator=g).to(BF).cuda() for _ in range(2))
    kw = dict(q_heads=H, kv_heads=H, positions=pos, inv_freq=p["freq"], wq=p["nq"], wk=p["nk"])
    qn, kn = smoe.smoe_moa_qk_norm_rope_fwd(q, k, ss, KS, **kw)
    att, lse = smoe.smoe_moa_attn_fwd(qn, kn, v, ss, KS, L, H)
    dqn, dkn, dv = smoe.smoe_moa_attn_bwd(qn, kn, v, att, lse, o, ss, KS, L, H)
    dq, dk, dwq, dwk = smoe.smoe_moa_qk_norm_rope_bwd(dqn, dkn, q, k, ss, KS, **kw)
    leaves = [t.cpu().double().requires_grad_(True) for t in (q, k, p["nq"], p["nk"], v)]
    q64, k64, nq, nk, v64 = leaves
    posc, freq = pos.cpu(), p["freq"].cpu()
    a = plain.norm_turn(q64.view(T * KS, H, DH), nq, posc[token], freq, False, 1e-6, True)
    b = plain.norm_turn(k64.view(T, H, DH), nk, posc, freq, False, 1e-6, True)
    sc = torch.einsum("shd,thd->hst", a, b) / math.sqrt(DH)
    t = torch.arange(T)
    seen = (t[None] <= token[:, None]) & (t[None] // L == token[:, None] // L)
    w = torch.softmax(sc.masked_fill(~seen[None], -math.inf), -1)
    out = torch.einsum("hst,thd->shd", w, v64.view(T, H, DH)).reshape(T * KS, W)
    grads = torch.autograd.grad((out * o.cpu().double()).sum(), leaves)
    for name, got, ref in zip(("dq", "dk", "dwq", "dwk", "dv"), (dq, dk, dwq, dwk, dv), grads):
        err = (got.cpu().double() - ref).norm() / ref.norm()
        # bf16 queries, keys, weights, scores' gradients and outputs: five roundings of 2^-8
        assert err <= 5 * 2.0 ** -8, (name, float(err))
