"""Query/key norm with rotation (smoe_moa_qk_norm_rope_fwd / _bwd) and its serving form
(smoe_moa_cache_append) against a plain form in 64 bits."""
import math

import pytest
import torch

import sparse_mixture_experts_smoe_b200 as smoe

from . import _plain_ops as plain

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
EPS = 1e-6
# fp32 errors of y relative to its pair |y_a| + |y_b|: the norm's factor (a sum of 128
# squares in a tree of at most 19 additions, a root, a quotient, two products: under
# 2^-19), the angle (2^-22 of a radian) and sine and cosine (2 ulp), two products and a sum.
TURN = 2.0 ** -17

CASES = {
    # T, kslots, q_heads, kv_heads, dh, dtype, interleaved, norm, rotate
    "one_token": (1, 1, 1, 1, 128, BF, False, True, True),
    "slots": (67, 4, 4, 4, 128, BF, False, True, True),
    "shared_heads": (45, 3, 6, 2, 64, BF, True, True, True),
    "fp32": (33, 2, 3, 1, 128, F32, False, True, True),
    "fp32_interleaved": (50, 1, 4, 4, 64, F32, True, True, True),
    "norm_only": (31, 2, 2, 2, 64, BF, False, True, False),
    "rotation_only": (31, 2, 2, 1, 128, F32, False, False, True),
    "many": (2500, 4, 2, 1, 128, BF, False, True, True),
}


def _freq(dh, theta=10000.0):
    return (theta ** (-2.0 * torch.arange(dh // 2, dtype=torch.float64) / dh)).float()


def _problem(name, seed=0):
    T, ks, qh, kvh, dh, dtype, inter, norm, rotate = CASES[name]
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = dict(T=T, ks=ks, qh=qh, kvh=kvh, dh=dh, dtype=dtype, inter=inter, norm=norm)
    p["q"], p["k"] = r(T * ks, qh * dh).to(dtype), r(T, kvh * dh).to(dtype)
    p["dq"], p["dk"] = r(T * ks, qh * dh).to(dtype), r(T, kvh * dh).to(dtype)
    p["wq"], p["wk"] = (1 + 0.2 * r(dh), 1 + 0.2 * r(dh)) if norm else (None, None)
    p["slots"] = torch.randperm(T * ks, generator=g).int()
    p["pos"] = torch.randint(0, 200000, (T,), generator=g).int()
    p["pos"][0] = 0
    p["freq"] = _freq(dh) if rotate else None
    return p


def _gpu(p, *names):
    return [None if p[n] is None else p[n].cuda() for n in names]


def _kw(p):
    pos, freq, wq, wk = _gpu(p, "pos", "freq", "wq", "wk")
    return dict(q_heads=p["qh"], kv_heads=p["kvh"], positions=pos, inv_freq=freq, wq=wq, wk=wk,
                eps=EPS, norm=p["norm"], interleaved=p["inter"])


def _ref(p, x, heads, w, pos):
    x = x.double().view(x.shape[0], heads, p["dh"])
    return plain.norm_turn(x, None if w is None else w.double(), pos, p["freq"], p["inter"], EPS,
                           p["norm"])


@pytest.mark.parametrize("name", list(CASES))
def test_forward(name):
    p = _problem(name)
    q, k, slots = _gpu(p, "q", "k", "slots")
    yq, yk = smoe.smoe_moa_qk_norm_rope_fwd(q, k, slots, p["ks"], **_kw(p))
    assert smoe.smoe_check() == 0
    qpos = p["pos"][(p["slots"] // p["ks"]).long()]
    for got, x, heads, w, pos in ((yq, p["q"], p["qh"], p["wq"], qpos),
                                  (yk, p["k"], p["kvh"], p["wk"], p["pos"])):
        ref = _ref(p, x, heads, w, pos)
        tol = plain.HALF[p["dtype"]] * ref.abs() + TURN * plain.pair_size(ref, p["inter"])
        assert got.dtype == p["dtype"] and got.shape == x.shape
        assert ((got.cpu().double().view(ref.shape) - ref).abs() <= tol).all()


@pytest.mark.parametrize("name", list(CASES))
def test_backward(name):
    p = _problem(name, 1)
    q, k, slots, dq, dk = _gpu(p, "q", "k", "slots", "dq", "dk")
    got = smoe.smoe_moa_qk_norm_rope_bwd(dq, dk, q, k, slots, p["ks"], **_kw(p))
    again = smoe.smoe_moa_qk_norm_rope_bwd(dq, dk, q, k, slots, p["ks"], **_kw(p))
    assert smoe.smoe_check() == 0
    qpos = p["pos"][(p["slots"] // p["ks"]).long()]
    for i, (x, dy, heads, w, pos) in enumerate(((p["q"], p["dq"], p["qh"], p["wq"], qpos),
                                                (p["k"], p["dk"], p["kvh"], p["wk"], p["pos"]))):
        xd = x.double().requires_grad_(True)
        wd = None if w is None else w.double().requires_grad_(True)
        y = plain.norm_turn(xd.view(x.shape[0], heads, p["dh"]), wd, pos, p["freq"], p["inter"], EPS,
                            p["norm"])
        dyd = dy.double().view(y.shape)
        grads = torch.autograd.grad((y * dyd).sum(), [xd] + ([wd] if w is not None else []))
        # sizes that the errors go by: the turned-back gradient by its pairs, the norm's two terms
        du = plain.pair_size(plain.turn(dyd, pos, p["freq"], p["inter"], back=True), p["inter"])
        size = du
        if p["norm"]:
            xh = x.double().view(y.shape)
            r = 1 / torch.sqrt((xh * xh).mean(-1, keepdim=True) + EPS)
            hat = (xh * r).abs()
            wabs = w.double().abs()
            size = r * (wabs * du + hat * (wabs * du * hat).mean(-1, keepdim=True))
        ref = grads[0].view(y.shape)
        tol = plain.HALF[p["dtype"]] * ref.abs() + 2 * TURN * size
        assert ((got[i].cpu().double().view(y.shape) - ref).abs() <= tol).all()
        assert torch.equal(got[i], again[i])
        if w is None:
            assert got[2 + i] is None
            continue
        # a sum of fp32 products: each within 2 TURN, the tree of sums under 2^-17 of the sum of sizes
        tol = 3 * TURN * (du * hat).sum((0, 1))
        assert ((got[2 + i].cpu().double() - grads[1]).abs() <= tol).all()
        assert torch.equal(got[2 + i], again[2 + i])


def test_backward_against_differences():
    p = _problem("shared_heads", 2)
    p = {**p, "dtype": F32, **{n: p[n].float() for n in ("q", "k", "dq", "dk")}}
    q, k, slots, dq, dk = _gpu(p, "q", "k", "slots", "dq", "dk")
    got = smoe.smoe_moa_qk_norm_rope_bwd(dq, dk, q, k, slots, p["ks"], **_kw(p))
    pos = p["pos"]

    def loss(x, w):
        y = plain.norm_turn(x.view(-1, p["kvh"], p["dh"]), w, pos, p["freq"], p["inter"], EPS, True)
        return (y * p["dk"].double().view(y.shape)).sum()

    x, w, h = p["k"].double(), p["wk"].double(), 1e-5
    g = torch.Generator().manual_seed(3)
    for _ in range(3):
        vx = torch.randn(x.shape, generator=g, dtype=torch.float64)
        vw = torch.randn(w.shape, generator=g, dtype=torch.float64)
        num = (loss(x + h * vx, w + h * vw) - loss(x - h * vx, w - h * vw)) / (2 * h)
        a = (got[1].cpu().double() * vx).sum() + (got[3].cpu().double() * vw).sum()
        scale = (got[1].cpu().double() * vx).abs().sum() + (got[3].cpu().double() * vw).abs().sum()
        assert abs(float(a - num)) <= 1e-5 * float(scale)


def test_far_positions_negative_and_zero_frequencies():
    """Positions up to 2^31 - 1, and pairs of frequency 0, which stay as they are."""
    dh, T = 64, 6
    pos = torch.tensor([0, 1, 2 ** 20 + 1, 2 ** 30 + 7, 2 ** 31 - 1, -5], dtype=torch.int32)
    freq = _freq(dh, 5e5)
    freq[20:] = 0.0
    k = torch.randn(T, dh, generator=torch.Generator().manual_seed(4))
    _, y = smoe.smoe_moa_qk_norm_rope_fwd(None, k.cuda(), None, 1, q_heads=1, kv_heads=1,
                                          positions=pos.cuda(), inv_freq=freq.cuda(), norm=False)
    # position * frequency reaches 2^31 radians: in 64 bits the reference itself is off by 2^-22
    ref = plain.turn(k.double().view(T, 1, dh), pos, freq, False)
    tol = TURN * plain.pair_size(ref, False)
    assert ((y.cpu().double().view(ref.shape) - ref).abs() <= tol).all()
    y = y.cpu()
    assert torch.equal(y[:, 20:32], k[:, 20:32]) and torch.equal(y[:, 52:], k[:, 52:])


def test_rows_apart_in_place_and_parts():
    p = _problem("slots", 5)
    q, k, slots = _gpu(p, "q", "k", "slots")
    kw = _kw(p)
    yq, yk = smoe.smoe_moa_qk_norm_rope_fwd(q, k, slots, p["ks"], **kw)
    wide = torch.full((q.shape[0], q.shape[1] + 64), 7.0, dtype=BF, device="cuda")
    wide[:, 32:32 + q.shape[1]] = q
    zq, none = smoe.smoe_moa_qk_norm_rope_fwd(wide[:, 32:32 + q.shape[1]], None, slots, p["ks"], **kw)
    assert none is None and torch.equal(zq, yq)
    dq, _, dwq, dwk = smoe.smoe_moa_qk_norm_rope_bwd(wide[:, 32:32 + q.shape[1]], None, q, None, slots,
                                                     p["ks"], **kw)
    assert dwk is None
    full = smoe.smoe_moa_qk_norm_rope_bwd(q, k, q, k, slots, p["ks"], **kw)
    assert torch.equal(dq, full[0]) and torch.equal(dwq, full[2])
    q2, k2 = q.clone(), k.clone()
    smoe.smoe_moa_qk_norm_rope_fwd(q2, k2, slots, p["ks"], q_out=q2, k_out=k2, **kw)
    assert torch.equal(q2, yq) and torch.equal(k2, yk)


def test_zero_rows_and_bad_slots():
    p = _problem("slots", 6)
    q, k, slots = _gpu(p, "q", "k", "slots")
    q[3] = 0
    yq, _ = smoe.smoe_moa_qk_norm_rope_fwd(q, k, slots, p["ks"], **_kw(p))
    assert (yq[3] == 0).all() and smoe.smoe_check() == 0
    bad = slots.clone()
    bad[5], bad[6] = -1, slots.numel()
    out = torch.full_like(q, 9.0)
    smoe.smoe_moa_qk_norm_rope_fwd(q, k, bad, p["ks"], q_out=out, **_kw(p))
    assert smoe.smoe_check() == -4
    assert (out[5] == 9).all() and (out[6] == 9).all()
    keep = [i for i in range(q.shape[0]) if i not in (5, 6)]
    assert torch.equal(out[keep], yq[keep])


# ---- the paged cache ------------------------------------------------------------
def _cache(pages, page, kvh, dh, f8, order="token"):
    """Caches full of a marker value, in one of the layouts that strides allow."""
    dt = torch.uint8 if f8 else BF
    if order == "head":  # heads outermost inside a page
        mk = lambda: torch.full((pages, kvh, page, dh), 3, dtype=dt, device="cuda").permute(0, 2, 1, 3)  # noqa: E731
    elif order == "both":  # keys and values of a page side by side
        both = torch.full((pages, 2, page, kvh, dh), 3, dtype=dt, device="cuda")
        return both[:, 0], both[:, 1]
    else:
        mk = lambda: torch.full((pages, page, kvh, dh), 3, dtype=dt, device="cuda")  # noqa: E731
    return mk(), mk()


APPEND = {
    # lens, new (None: one each), page, kslots, q_heads, kv_heads, dh, e4m3, interleaved, order
    "one_each": ([5, 1, 0, 40], None, 16, 4, 4, 4, 128, False, False, "token"),
    "one_each_e4m3": ([5, 17, 0, 40], None, 7, 2, 2, 1, 64, True, True, "head"),
    "prompts": ([9, 30, 4], [9, 11, 0], 8, 3, 6, 2, 128, False, True, "both"),
    "prompts_e4m3": ([100, 3, 64], [70, 3, 1], 64, 1, 4, 4, 128, True, False, "token"),
    # more sequences than a block lists; a few without new tokens
    "many_prompts": ([3 + b % 7 for b in range(600)], [(b * 5) % 3 for b in range(600)], 4, 1, 1, 1, 64, False, False,
                     "token"),
    "page_of_one": ([6, 2], [3, 2], 1, 2, 1, 1, 64, False, False, "head"),
}


@pytest.mark.parametrize("name", list(APPEND))
@pytest.mark.parametrize("norm", [True, False])
def test_append(name, norm):
    lens, new, page, ks, qh, kvh, dh, f8, inter, order = APPEND[name]
    B = len(lens)
    g = torch.Generator().manual_seed(7)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    perm = torch.randperm(pages, generator=g).int()
    table = torch.full((B, max(need) + 1), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    n_new = new or [1] * B
    T = sum(n_new) + (2 if new else 0)  # two rows behind the last sequence
    starts = torch.tensor([sum(n_new[:b]) for b in range(B + 1)], dtype=torch.int32) if new else None
    q = torch.randn(T * ks, qh * dh, generator=g).to(BF)
    k = torch.randn(T, kvh * dh, generator=g).to(BF)
    v = torch.randn(T, kvh * dh, generator=g).to(BF)
    v[0] = 0
    wq, wk = (1 + 0.1 * torch.randn(dh, generator=g) for _ in range(2))
    slots = torch.randperm(T * ks, generator=g).int()
    freq = _freq(dh)
    kc, vc = _cache(pages, page, kvh, dh, f8, order)
    sc = [torch.full((pages, page, kvh), 3.0, device="cuda") for _ in range(2)] if f8 else [None, None]
    q_out = torch.full((T * ks, qh * dh), 5.0, dtype=BF, device="cuda")
    kw = dict(inv_freq=freq.cuda(), eps=EPS, interleaved=inter, norm=norm)
    if norm:
        kw.update(wq=wq.cuda(), wk=wk.cuda())
    smoe.smoe_moa_cache_append(q.cuda(), k.cuda(), v.cuda(), kc, vc, table.cuda(),
                               torch.tensor(lens, dtype=torch.int32, device="cuda"), slots.cuda(), ks,
                               qh, starts=None if starts is None else starts.cuda(), k_scale=sc[0],
                               v_scale=sc[1], q_out=q_out, **kw)
    assert smoe.smoe_check() == 0
    pos = torch.full((T,), -1)
    seq = torch.zeros(T, dtype=torch.long)
    t = 0
    for b in range(B):
        for i in range(n_new[b]):
            pos[t], seq[t] = lens[b] - n_new[b] + i, b
            t += 1
    live = pos >= 0
    qpos = pos[(slots // ks).long()]
    ref = plain.norm_turn(q.double().view(T * ks, qh, dh), wq.double(), qpos.clamp(min=0), freq, inter,
                          EPS, norm)
    got = q_out.cpu().double().view(ref.shape)
    tol = plain.HALF[BF] * ref.abs() + TURN * plain.pair_size(ref, inter)
    on = qpos >= 0
    assert ((got - ref).abs() <= tol)[on].all()
    assert (got[~on] == 5).all()
    rk = plain.norm_turn(k.double().view(T, kvh, dh), wk.double(), pos.clamp(min=0), freq, inter, EPS,
                         norm)
    rv = v.double().view(T, kvh, dh)
    touched = torch.zeros(pages, page, dtype=torch.bool)
    for x, ref, cache, scale in (("k", rk, kc, sc[0]), ("v", rv, vc, sc[1])):
        c = cache.cpu()
        for i in torch.nonzero(live).flatten().tolist():
            p_, f_ = int(table[seq[i], pos[i] // page]), int(pos[i] % page)
            touched[p_, f_] = True
            r = ref[i]
            err = TURN * plain.pair_size(r, inter) if x == "k" else torch.zeros_like(r)
            if not f8:
                assert ((c[p_, f_].double() - r).abs() <= plain.HALF[BF] * r.abs() + err).all()
                continue
            s = scale[p_, f_].cpu().double()
            amax = r.abs().amax(-1)
            want = torch.where(amax == 0, torch.ones_like(amax), amax / 448)
            assert ((s - want).abs() <= 4 * TURN * want).all()
            code = c[p_, f_].view(torch.float8_e4m3fn).double()
            # e4m3: half a step is 2^-4 of the value, 2^-10 below the smallest normal
            dec = code * s[:, None]
            tol = (2.0 ** -4 * r.abs() + 2.0 ** -10 * s[:, None]) * (1 + 2.0 ** -10) + 2 * err
            assert ((dec - r).abs() <= tol).all()
        assert (c[~touched].float() == 3).all()  # nothing else is written
        if f8:
            assert (scale.cpu()[~touched] == 3).all()


def test_append_reports_and_skips_bad_places():
    B, page, kvh, dh = 4, 4, 1, 64
    kc, vc = _cache(3, page, kvh, dh, False)
    table = torch.tensor([[0, 1], [7, 7], [-1, 2], [2, 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([3, 2, 1, 9], dtype=torch.int32, device="cuda")  # 9 is beyond 2 pages of 4
    k = torch.randn(B, dh, device="cuda").to(BF)
    smoe.smoe_moa_cache_append(None, k, k, kc, vc, table, lens, None, 1, 1, norm=False)
    assert smoe.smoe_check() == -4
    assert torch.equal(kc[0, 2, 0], k[0]) and torch.equal(vc[0, 2, 0], k[0])
    kc[0, 2] = 3
    assert (kc == 3).all()
    # more new tokens than the sequence has
    starts = torch.tensor([0, 3, 3, 3, 4], dtype=torch.int32, device="cuda")
    lens = torch.tensor([2, 0, 0, 1], dtype=torch.int32, device="cuda")
    smoe.smoe_moa_cache_append(None, k, k, kc, vc, table, lens, None, 1, 1, starts=starts, norm=False)
    assert smoe.smoe_check() == -4
    assert torch.equal(kc[0, 0, 0], k[1]) and torch.equal(kc[0, 1, 0], k[2])


def test_append_e4m3_of_tiny_and_large_rows():
    """Rows down to the smallest bf16 number: codes stay finite and within half a step."""
    kc, vc = _cache(1, 8, 1, 64, True)
    sc = [torch.ones(1, 8, 1, device="cuda") for _ in range(2)]
    table = torch.zeros(6, 1, dtype=torch.int32, device="cuda")
    lens = torch.arange(1, 7, dtype=torch.int32, device="cuda")
    size = torch.tensor([2.0 ** -133, 1e-38, 1e-30, 1.0, 1e30, 3e38])
    g = torch.Generator().manual_seed(21)
    k = (size[:, None] * (0.25 + 0.75 * torch.rand(6, 64, generator=g))).to(BF)
    smoe.smoe_moa_cache_append(None, k.cuda(), k.cuda(), kc, vc, table, lens, None, 1, 1, norm=False,
                               k_scale=sc[0], v_scale=sc[1])
    assert smoe.smoe_check() == 0
    for c, s in ((kc, sc[0]), (vc, sc[1])):
        s = s[0, :6].cpu().double()
        got = c[0, :6, 0].cpu().view(torch.float8_e4m3fn).double() * s
        want = k.double()
        # e4m3's half steps, and the fp32 roundings of the scale and its reciprocal
        tol = (2.0 ** -4 * want + 2.0 ** -10 * s) * (1 + 2.0 ** -20)
        assert torch.isfinite(got).all() and ((got - want).abs() <= tol).all()


def test_graph_and_stream():
    p = _problem("slots", 8)
    q, k, slots = _gpu(p, "q", "k", "slots")
    kw = _kw(p)
    want = smoe.smoe_moa_qk_norm_rope_bwd(q, k, q, k, slots, p["ks"], **kw)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = smoe.smoe_moa_qk_norm_rope_bwd(q, k, q, k, slots, p["ks"], stream=st, **kw)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = smoe.smoe_moa_qk_norm_rope_bwd(q, k, q, k, slots, p["ks"], **kw)
    for _ in range(2):
        gr.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_empty():
    e = torch.empty(0, 128, dtype=BF, device="cuda")
    w = torch.ones(128, device="cuda")
    yq, yk = smoe.smoe_moa_qk_norm_rope_fwd(e, e, None, 2, q_heads=1, kv_heads=1, wq=w, wk=w)
    assert yq.shape == (0, 128) and yk.shape == (0, 128)
    _, _, dwq, dwk = smoe.smoe_moa_qk_norm_rope_bwd(e, e, e, e, None, 2, q_heads=1, kv_heads=1, wq=w,
                                                    wk=w)
    assert (dwq == 0).all() and (dwk == 0).all()


@pytest.mark.parametrize("dh", [64, 128])
def test_append_e4m3_codes_are_the_quotients(dh):
    """Scale amax / 448 and code e4m3(v / scale), each operation rounded in fp32 as
    smoe_quantize_weights_fp8 does, to the bit: bf16 rows have many quotients half way
    between two codes, which a product with the scale's reciprocal moves off the middle."""
    B, kvh = 700, 3
    g = torch.Generator().manual_seed(31)
    size = torch.exp2(torch.randint(-110, 110, (B, 1), generator=g).float())
    size[:B // 2] = 1.0
    k, v = ((size * torch.randn(B, kvh * dh, generator=g)).to(BF) for _ in range(2))
    kc, vc = _cache(B, 1, kvh, dh, True)
    sc = [torch.zeros(B, 1, kvh, device="cuda") for _ in range(2)]
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    smoe.smoe_moa_cache_append(None, k.cuda(), v.cuda(), kc, vc, table, lens, None, 1, kvh, norm=False,
                               k_scale=sc[0], v_scale=sc[1])
    assert smoe.smoe_check() == 0
    for x, codes, scale in ((k, kc, sc[0]), (v, vc, sc[1])):
        x = x.float().view(B, kvh, dh)
        s = x.abs().amax(-1) / 448.0
        assert torch.equal(scale.cpu()[:, 0], s)
        want = (x / s[..., None]).to(torch.float8_e4m3fn)
        assert torch.equal(codes.cpu()[:, 0].view(torch.float8_e4m3fn).float(), want.float())


def test_backward_leaves_skipped_rows_out_of_the_weights():
    """A row whose slot is out of range adds nothing to dwq: the bits of a run in which the
    row's upstream gradient is 0, whatever the row holds."""
    for name in ("slots", "fp32", "many"):
        p = _problem(name, 9)
        q, k, slots, dq, dk = _gpu(p, "q", "k", "slots", "dq", "dk")
        rows = [0, 5, q.shape[0] - 1]
        none = dq.clone()
        none[rows] = 0
        want = smoe.smoe_moa_qk_norm_rope_bwd(none, dk, q, k, slots, p["ks"], **_kw(p))
        bad, x, dy = slots.clone(), q.clone(), dq.clone()
        bad[rows] = torch.tensor([-1, slots.numel(), 2 ** 31 - 1], dtype=torch.int32, device="cuda")
        x[rows[0]], dy[rows[1]] = math.nan, math.inf
        got = smoe.smoe_moa_qk_norm_rope_bwd(dy, dk, x, k, bad, p["ks"], **_kw(p))
        assert smoe.smoe_check() == -4 and smoe.smoe_check() == 0
        assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])
        keep = [i for i in range(q.shape[0]) if i not in rows]
        assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1], want[1])
