"""Attention of one new token over a paged cache (smoe_moa_decode) against a plain form in
64 bits: ragged and empty batches, pages that end anywhere, both cache types, shared key
heads, layouts, far offsets, bad tables, graphs and streams."""
import math

import pytest
import torch

import sparse_mixture_experts_smoe_b200 as smoe

from . import _plain_ops as plain

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
# Relative error of a weight.  The score is an fp32 sum of 128 products of size at most 40
# (2^-24 times a tree and a chain of under 16 roundings, 2^-15 of an exponent), ex2 2 ulp;
# then the weight is held as two bf16 numbers for a bf16 cache, as fp16 with its scale for e4m3.
SCORE = 2.0 ** -14
WEIGHT = {False: 2.0 ** -16 + SCORE, True: 2.0 ** -11 + SCORE}

CASES = {
    # lens, page, kslots, q_heads, kv_heads, dh, e4m3, layout
    "one_token": ([1], 16, 1, 1, 1, 128, False, "token"),
    "one_sequence": ([2048], 16, 4, 4, 4, 128, False, "token"),
    "ragged_and_empty": ([0, 5, 64, 0, 65, 1, 300, 0], 16, 4, 2, 2, 128, False, "token"),
    "all_empty": ([0, 0, 0], 16, 2, 2, 1, 128, False, "token"),
    "odd_pages": ([100, 33, 207], 7, 3, 3, 1, 64, False, "head"),
    "page_of_one": ([50, 3], 1, 1, 2, 2, 64, False, "both"),
    "page_of_100": ([1000, 99, 100, 101], 100, 2, 6, 2, 128, False, "head"),
    "sixteen_queries": ([513, 40], 48, 8, 4, 2, 128, False, "both"),
    "thirty_two_queries": ([700, 129], 64, 8, 4, 1, 128, False, "token"),
    "forty_one_queries": ([130, 17], 16, 41, 2, 2, 128, True, "token"),
    "ninety_queries": ([300, 64, 17], 32, 15, 12, 2, 128, False, "token"),
    "many_sequences": ([(37 * b) % 91 for b in range(300)], 16, 2, 1, 1, 64, False, "token"),
    # so much work for each warp that a part of it is fetched
    "fetched": ([12000, 9000, 11000, 10500, 10, 0], 16, 128, 4, 1, 64, False, "token"),
    "fetched_e4m3": ([12000, 9000, 11000, 10500, 10], 48, 128, 8, 2, 64, True, "head"),
    # sequences that are not split
    "short_sequences": ([(7 * b) % 90 for b in range(100)], 16, 2, 2, 2, 128, False, "token"),
    "short_e4m3": ([(11 * b) % 60 for b in range(250)], 7, 1, 2, 1, 64, True, "head"),
    "short_empty": ([0] * 77 + [33, 1], 32, 1, 1, 1, 64, False, "token"),
    # more key heads and query tiles than warps
    "many_items": ([40], 16, 128, 320, 320, 64, False, "token"),
    "e4m3": ([300, 0, 64, 63], 48, 2, 8, 2, 128, True, "token"),
    "e4m3_one": ([1], 7, 1, 1, 1, 64, True, "head"),
    "e4m3_sixteen": ([400, 31], 16, 4, 4, 1, 64, True, "both"),
    "e4m3_forty": ([260, 5], 100, 5, 8, 1, 128, True, "token"),
    "e4m3_long": ([4099], 256, 4, 1, 1, 128, True, "token"),
}


def _store(x, layout):
    """x [pages, page, kvh, dh] on the GPU in one of the layouts that strides allow."""
    pages, page, kvh, dh = x.shape
    if layout == "head":
        return x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)
    if layout == "both":
        wide = torch.zeros((pages, 2, page, kvh, dh), dtype=x.dtype)
        wide[:, 1] = x
        return wide.cuda()[:, 1]
    return x.cuda()


def _problem(lens, page, ks, qh, kvh, dh, f8, layout, seed=0, qstd=1.0):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    perm = torch.randperm(pages, generator=g).int()
    table = torch.full((B, max(max(need), 1) + 1), -7, dtype=torch.int32)  # never read beyond need
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    p = dict(lens=lens, ks=ks, qh=qh, table=table, scales=(None, None))
    used = torch.zeros(pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        u = torch.arange(n)
        used[table[b, u // page].long(), u % page] = True
    vals, stored, scales = [], [], []
    for _ in range(2):
        x = torch.randn(pages, page, kvh, dh, generator=g)
        if f8:
            s = (0.1 + torch.rand(pages, page, kvh, generator=g)) * x.abs().amax(-1) / 448.0
            code = (x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            vals.append(code.double() * s.double()[..., None])
            raw = code.view(torch.uint8).clone()
            raw[~used] = 0x7f  # NaN
            s[~used] = math.nan
            stored.append(_store(raw, layout))
            scales.append(s.cuda())
        else:
            x = x.to(BF)
            vals.append(x.double())
            x = x.clone()
            x[~used] = math.nan  # places without a token are not read
            stored.append(_store(x, layout))
    if f8:
        p["scales"] = tuple(scales)
    p["k"], p["v"], p["kc"], p["vc"] = *vals, *stored
    p["q"] = (qstd * torch.randn(B * ks, qh * dh, generator=g)).to(BF)
    p["slots"] = torch.randperm(B * ks, generator=g).int()
    return p


def _args(p):
    return dict(q=p["q"].cuda(), k_cache=p["kc"], v_cache=p["vc"], block_table=p["table"].cuda(),
                seq_lens=torch.tensor(p["lens"], dtype=torch.int32, device="cuda"),
                sorted_slot=p["slots"].cuda(), kslots=p["ks"], q_heads=p["qh"],
                k_scale=p["scales"][0], v_scale=p["scales"][1])


def _run(p, **kw):
    return smoe.smoe_moa_decode(**{**_args(p), **kw})


def _close(p, o, lse, rows=slice(None), table=None, lens=None):
    ref, rl, size = plain.decode(p["q"], p["k"], p["v"], p["table"] if table is None else table,
                                 p["lens"] if lens is None else lens, p["slots"], p["ks"], p["qh"])
    f8 = p["scales"][0] is not None
    # fp16 weights times scales below 2^-14 of the largest lose 2^-25 of it each: with at most
    # 12000 keys of codes up to 448, and scales within 11 to 1, under 2^-9 of the mean weight's
    # share of a row whose largest value is at most 4 times its mean size
    tol = plain.HALF[BF] * ref.abs() + (WEIGHT[f8] + (2.0 ** -9 if f8 else 0.0)) * size
    assert o.dtype == BF and o.shape == p["q"].shape
    got = o.cpu().double()
    assert torch.isfinite(got[rows]).all()
    assert ((got - ref).abs() <= tol + 1e-30)[rows].all()
    lse = lse.cpu().double()
    fin = torch.isfinite(rl)
    assert torch.equal(torch.isfinite(lse)[rows], fin[rows]) and (lse[rows][~fin[rows]] < 0).all()
    err = (torch.where(fin, lse, torch.zeros_like(lse)) - torch.where(fin, rl, torch.zeros_like(rl))).abs()
    assert (err <= SCORE + plain.HALF[torch.float32] * torch.where(fin, rl, torch.zeros_like(rl)).abs())[rows].all()


@pytest.mark.parametrize("name", list(CASES))
def test_decode(name):
    p = _problem(*CASES[name])
    o, lse = _run(p)
    assert smoe.smoe_check() == 0
    _close(p, o, lse)
    o2, lse2 = _run(p)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("f8", [False, True])
def test_decode_peaked_scores(f8):
    """Queries along a key: one key in the middle takes nearly all of the weight, the
    running maximum jumps, and the scores before it lose theirs."""
    p = _problem([700, 64], 16, 2, 2, 1, 128, f8, "token", seed=2, qstd=0.05)
    for b, u in ((0, 413), (1, 0)):
        key = p["k"][int(p["table"][b, u // 16]), u % 16, 0]
        for i in range(4):
            if int(p["slots"][i]) // 2 == b:
                p["q"][i] = (3.0 * key.repeat(2) / key.norm() * 11).to(BF)
    o, lse = _run(p)
    assert smoe.smoe_check() == 0
    _close(p, o, lse)


def test_decode_without_slots_rows_apart_and_no_lse():
    p = _problem([70, 20, 9], 16, 2, 2, 2, 128, False, "token", seed=3)
    p["slots"] = torch.arange(6, dtype=torch.int32)
    o, lse = _run(p, sorted_slot=None)
    _close(p, o, lse)
    wide = torch.zeros(6, 256 + 64, dtype=BF, device="cuda")
    wide[:, 32:288] = p["q"].cuda()
    tab = torch.full((3, 20), -1, dtype=torch.int32, device="cuda")
    tab[:, 5:5 + p["table"].shape[1]] = p["table"].cuda()
    o2, _ = _run(p, q=wide[:, 32:288], block_table=tab[:, 5:5 + p["table"].shape[1]])
    assert torch.equal(o, o2) and smoe.smoe_check() == 0
    mine, ml = torch.empty_like(o), torch.empty_like(lse)
    o3, l3 = _run(p, o=mine, lse=ml)
    assert o3 is mine and l3 is ml and torch.equal(o3, o) and torch.equal(l3, lse)


def test_decode_reports_bad_tables_lengths_and_slots():
    p = _problem([40, 33, 16, 50], 16, 2, 1, 1, 64, False, "token", seed=4)
    table = p["table"].clone()
    table[0, 1] = 10 ** 6
    table[2, 0] = -1           # every key of sequence 2 is left out
    o, lse = _run(p, block_table=table.cuda())
    assert smoe.smoe_check() == -4 and smoe.smoe_check() == 0
    _close(p, o, lse, table=table)
    # lengths are clamped to what the table can hold, and to 0
    cap = p["table"].shape[1] * 16
    lens = [40, -3, 16, cap + 9]
    table = p["table"].clone()
    table[3] = torch.arange(table.shape[1]) % 4
    q = dict(p, table=table)
    kc = torch.nan_to_num(p["kc"].float(), nan=0.5).to(BF)
    vc = torch.nan_to_num(p["vc"].float(), nan=0.5).to(BF)
    q.update(kc=kc, vc=vc, k=kc.cpu().double(), v=vc.cpu().double())
    o, lse = _run(q, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    assert smoe.smoe_check() == -4
    _close(q, o, lse, lens=lens)
    # a slot that no row names is not written; the others are right
    slots = p["slots"].clone()
    slots[1], slots[5] = -1, 99
    o = torch.full_like(p["q"], 9.0).cuda()
    lse = torch.full((8, 1), 9.0, device="cuda")
    _run(p, sorted_slot=slots.cuda(), o=o, lse=lse)
    assert smoe.smoe_check() == -4
    keep = [i for i in range(8) if i not in (1, 5)]
    _close(p, o, lse, rows=keep)
    assert (o[[1, 5]] == 9).all() and (lse[[1, 5]] == 9).all()


@pytest.mark.parametrize("f8", [False, True])
def test_decode_offsets_beyond_32_bits(f8):
    """Pages at the far end of a cache of more than 2^32 bytes (and 2^32 elements in
    e4m3): the same bits as from a small cache that holds the same pages."""
    p = _problem([150, 61], 64, 2, 2, 2, 128, f8, "token", seed=5)
    o, lse = _run(p)
    pages = p["kc"].shape[0]
    far = 270000 if f8 else 140000  # x 64 x 2 x 128 elements
    big = [torch.empty((far, 64, 2, 128), dtype=p["kc"].dtype, device="cuda") for _ in range(2)]
    kw = {}
    if f8:
        sc = [torch.empty((far, 64, 2), device="cuda") for _ in range(2)]
        for s, t in zip(sc, p["scales"]):
            s[far - pages:] = t
        kw = dict(k_scale=sc[0], v_scale=sc[1])
    for b, t in zip(big, (p["kc"], p["vc"])):
        b[far - pages:] = t
    table = torch.where(p["table"] >= 0, p["table"] + (far - pages), p["table"])
    o2, lse2 = _run(p, k_cache=big[0], v_cache=big[1], block_table=table.cuda(), **kw)
    assert smoe.smoe_check() == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_decode_fetched_ranges_in_graphs_and_streams():
    """The form with fetched ranges: captured once, replayed with lengths that need them and
    lengths that do not, while another stream makes the same call."""
    p = _problem(*CASES["fetched"])
    a = _args(p)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = smoe.smoe_moa_decode(**a)
    st = torch.cuda.Stream()
    for lens in ([12000, 9000, 11000, 10500, 10, 0], [5, 0, 0, 1, 10, 0], [0] * 6, [11999, 8001, 1, 10500, 9, 0]):
        a["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        st.wait_stream(torch.cuda.current_stream())
        g.replay()
        other = smoe.smoe_moa_decode(stream=st, **a)
        now = smoe.smoe_moa_decode(**a)
        st.synchronize()
        for x in (other, now):
            assert torch.equal(out[0], x[0]) and torch.equal(out[1], x[1])
    assert smoe.smoe_check() == 0


def test_decode_empty_batch():
    c = torch.empty(0, 16, 1, 64, dtype=BF, device="cuda")
    o, lse = smoe.smoe_moa_decode(torch.empty(0, 64, dtype=BF, device="cuda"), c, c,
                                  torch.empty(0, 0, dtype=torch.int32, device="cuda"),
                                  torch.empty(0, dtype=torch.int32, device="cuda"), None, 1, 1)
    assert o.shape == (0, 64) and lse.shape == (0, 1)
    # a cache without pages, a batch without tokens
    o, lse = smoe.smoe_moa_decode(torch.ones(2, 64, dtype=BF, device="cuda"), c, c,
                                  torch.empty(2, 0, dtype=torch.int32, device="cuda"),
                                  torch.zeros(2, dtype=torch.int32, device="cuda"), None, 1, 1)
    assert smoe.smoe_check() == 0
    assert (o == 0).all() and (lse == -math.inf).all()


def test_decode_streams_and_graphs():
    """Two streams at once, and two graphs with their own workspaces replayed in turn
    while lengths and tables change under them."""
    ps = [_problem([900, 33, 0, 257], 16, 4, 2, 2, 128, f8, "token", seed=6) for f8 in (False, True)]
    args = [_args(p) for p in ps]
    want = [smoe.smoe_moa_decode(**a) for a in args]
    sts = [torch.cuda.Stream() for _ in ps]
    for st in sts:
        st.wait_stream(torch.cuda.current_stream())
    got = [smoe.smoe_moa_decode(stream=st, **a) for _ in range(3) for a, st in zip(args, sts)]
    for st in sts:
        st.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])
    graphs, outs = [], []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(smoe.smoe_moa_decode(**a))
        graphs.append(g)
    for lens in ([900, 33, 0, 257], [1, 0, 0, 2], [640, 16, 0, 200]):
        for g, a, out in zip(graphs, args, outs):
            a["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
            g.replay()
            now = smoe.smoe_moa_decode(**a)
            assert torch.equal(out[0], now[0]) and torch.equal(out[1], now[1])
    assert smoe.smoe_check() == 0


# Relative error of an e4m3 cache's weight times its scale as two bf16 numbers: 2^-16, fp32
# products 2^-24, and the score's.
PAIR = 2.0 ** -16 + 2.0 ** -20 + SCORE


def _with_scales(p, k_scale, v_scale, k_code, v_code):
    """The problem with these scales and codes (all places hold numbers)."""
    p["scales"] = k_scale.cuda(), v_scale.cuda()
    p["kc"], p["vc"] = k_code.view(torch.uint8).cuda(), v_code.view(torch.uint8).cuda()
    p["k"] = k_code.double() * k_scale.double()[..., None]
    p["v"] = v_code.double() * v_scale.double()[..., None]


def _close_pair(p, o, lse):
    ref, rl, size = plain.decode(p["q"], p["k"], p["v"], p["table"], p["lens"], p["slots"], p["ks"], p["qh"])
    assert ((o.cpu().double() - ref).abs() <= plain.HALF[BF] * ref.abs() + PAIR * size + 1e-37).all()
    assert ((lse.cpu().double() - rl).abs() <= SCORE + plain.HALF[torch.float32] * rl.abs()).all()


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("above", [0, 6, 9, 12])
@pytest.mark.parametrize("lens", [[30, 9, 32] * 20, [64, 40, 33] * 20, [2048, 700], [4096]],
                         ids=["whole", "short", "split", "long"])
@pytest.mark.parametrize("amax", [3.0, 1e-5])
def test_decode_e4m3_zero_value_row_with_a_high_score(lens, above, dh, amax):
    """A key that draws most of the weight and whose value row is 0, with the scale 1 that an
    append gives such a row: the other tokens' small weights keep their bits."""
    p = _problem(lens, 16, 2, 2, 1, dh, True, "token", seed=7)
    g = torch.Generator().manual_seed(8)
    shape = p["k"].shape
    code = [(448.0 * (2 * torch.rand(shape, generator=g) - 1)).to(torch.float8_e4m3fn).float() for _ in range(2)]
    scale = [(0.5 + torch.rand(shape[:3], generator=g)) * m / 448.0 for m in (1.7, amax)]
    code[0][..., 0] = 0.0  # the first dimension is the sink's: queries hold 8 there
    p["q"] = p["q"].float().view(-1, 2, dh).index_fill(2, torch.tensor([0]), 8.0).to(BF).view(p["q"].shape)
    for b, n in enumerate(lens):
        u = (5 * b + 3) % n
        at = int(p["table"][b, u // 16]), u % 16
        code[0][at] = 0.0
        code[0][at][0, 0] = 448.0
        scale[0][at] = above * math.sqrt(dh) / (8.0 * 448.0) if above else 1.0 / 448.0
        code[1][at], scale[1][at] = 0.0, 1.0
    _with_scales(p, *scale, *(c.to(torch.float8_e4m3fn) for c in code))
    o, lse = _run(p)
    assert smoe.smoe_check() == 0
    _close_pair(p, o, lse)


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("lens", [[30, 9, 32] * 20, [64, 40, 33] * 20, [3000]], ids=["whole", "short", "split"])
def test_decode_e4m3_scales_of_any_size(lens, dh):
    """Value scales from 2^-60 to 2^20 side by side, all codes in use."""
    p = _problem(lens, 7, 3, 2, 2, dh, True, "head", seed=9)
    g = torch.Generator().manual_seed(10)
    shape = p["k"].shape
    k_code = (448.0 * (2 * torch.rand(shape, generator=g) - 1)).to(torch.float8_e4m3fn)
    raw = torch.randint(0, 256, shape, generator=g).to(torch.uint8)
    raw[(raw & 0x7f) == 0x7f] = 1  # no NaN; 1: the smallest
    k_scale = (0.5 + torch.rand(shape[:3], generator=g)) * 1.7 / 448.0
    v_scale = torch.exp2(80 * torch.rand(shape[:3], generator=g) - 60)
    _with_scales(p, k_scale, v_scale, k_code, raw.view(torch.float8_e4m3fn))
    p["kc"], p["vc"] = (_store(t.cpu(), "head") for t in (p["kc"], p["vc"]))
    o, lse = _run(p)
    assert smoe.smoe_check() == 0
    _close_pair(p, o, lse)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("lens", [[16, 9, 3] * 15, [40, 33, 16] * 15, [2048, 700], [20000]],
                         ids=["whole", "short", "split", "long"])
def test_decode_nan_queries_give_nan(lens, f8):
    """A head whose query holds a NaN gives NaN, output and lse, whether its sequence lies in
    one range or in several; the other heads keep their bits."""
    p = _problem(lens, 16, 2, 4, 2, 64, f8, "token", seed=11)
    want = _run(p)
    rows = p["q"].shape[0]
    p["q"] = p["q"].clone()
    hit = torch.zeros(rows, 4, dtype=torch.bool)
    for i in (0, rows // 2, rows - 1):
        h = i % 4
        p["q"][i, h * 64 + (7 * i) % 64] = math.nan
        hit[i, h] = True
    o, lse = (t.cpu() for t in _run(p))
    assert smoe.smoe_check() == 0
    o = o.view(rows, 4, 64)
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(o[~hit], want[0].cpu().view(rows, 4, 64)[~hit]) and torch.equal(lse[~hit], want[1].cpu()[~hit])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("part", ["all", "middle", "one"])
def test_decode_nan_keys_give_nan(f8, part):
    """Keys of NaN: all of a sequence, all of several ranges, a single one."""
    p = _problem([3000, 50, 64], 16, 2, 2, 1, 64, f8, "token", seed=12)
    want = _run(p)
    for b, n in ((0, 3000), (1, 50)):
        for u in {"all": range(n), "middle": range(n // 3, n // 2), "one": [n // 2]}[part]:
            at = int(p["table"][b, u // 16]), u % 16
            p["kc"][at] = 0x7f if f8 else math.nan
    o, lse = _run(p)
    assert smoe.smoe_check() == 0
    on = (p["slots"] // 2 < 2).cuda()
    assert torch.isnan(o[on]).all() and torch.isnan(lse[on]).all()
    assert torch.equal(o[~on], want[0][~on]) and torch.equal(lse[~on], want[1][~on])


@pytest.mark.parametrize("lens", [[16, 9, 3] * 15, [2048, 700]], ids=["whole", "split"])
def test_decode_nan_and_infinite_values_stay_in_their_column(lens):
    p = _problem(lens, 16, 2, 2, 1, 64, False, "token", seed=14)
    want = _run(p)[0].view(-1, 2, 64)
    for b, value, at in ((0, math.nan, 5), (1, math.inf, 63)):
        u = lens[b] // 2
        p["vc"][int(p["table"][b, u // 16]), u % 16, 0, at] = value
    o = _run(p)[0].view(-1, 2, 64)
    assert smoe.smoe_check() == 0
    of = p["slots"].cuda() // 2
    assert torch.isnan(o[of == 0, :, 5]).all() and not torch.isfinite(o[of == 1, :, 63]).any()
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[of == 0, :, 5] = True
    hit[of == 1, :, 63] = True
    assert torch.equal(o[~hit], want[~hit])


def test_decode_many_short_items_for_each_warp():
    """Items that follow one another in a warp, each with the rows of its own sequence, where
    nothing between two of them makes the lanes wait (whole pages, one unit of 16 keys a
    product) and not all lanes have a row to write."""
    for ks, heads, dh in ((3, 64, 128), (2, 48, 128), (5, 64, 64)):
        p = _problem([1 + (5 * b) % 40 for b in range(90)], 16, ks, heads, heads, dh, False, "token", seed=15)
        a = _args(p)
        o, lse = smoe.smoe_moa_decode(**a)
        assert smoe.smoe_check() == 0
        _close(p, o, lse)
        for _ in range(20):
            again = smoe.smoe_moa_decode(**a)
            assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
        assert smoe.smoe_check() == 0


def test_decode_cache_with_one_key_head_of_any_stride():
    """A dimension of one has no stride that counts."""
    for f8 in (False, True):
        p = _problem([70, 9], 16, 2, 2, 1, 64, f8, "token", seed=13)
        want = _run(p)
        pages = p["kc"].shape[0]
        odd = [torch.empty(pages, 16, 64, 1, dtype=t.dtype, device="cuda").transpose(2, 3) for t in (p["kc"], p["vc"])]
        for x, t in zip(odd, (p["kc"], p["vc"])):
            x.copy_(t)
            assert x.stride(2) == 1
        o, lse = _run(p, k_cache=odd[0], v_cache=odd[1])
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        k = torch.ones(2, 64, dtype=BF, device="cuda")
        kw = dict(k_scale=p["scales"][0], v_scale=p["scales"][1], norm=False)
        a = _args(p)
        smoe.smoe_moa_cache_append(None, k, k, odd[0], odd[1], a["block_table"], a["seq_lens"], None, 1, 1, **kw)
        smoe.smoe_moa_cache_append(None, k, k, p["kc"], p["vc"], a["block_table"], a["seq_lens"], None, 1, 1, **kw)
        assert smoe.smoe_check() == 0
        assert all(torch.equal(x.view(torch.uint8), t.view(torch.uint8)) for x, t in
                   zip((odd[0].contiguous(), odd[1].contiguous()), (p["kc"], p["vc"])))
