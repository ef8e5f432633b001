"""Routing from given logits (smoe_route_select, smoe_route_select_bwd) against a plain
form in 64 bits: ids equal, gates and gradients within the rounding that the formulas
allow; scores that lie next to one another, ties, unavailable experts, groups, strides."""
import math

import pytest
import torch

import sparse_mixture_experts_smoe_b200 as smoe

from . import _plain_ops as plain

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
# A gate is a quotient of exponentials of differences of fp32 logits: the difference is
# rounded once (2^-24 of at most 32 here, as an exponent a relative 2^-19), expf, the sum
# of 16 and the quotient add under 2^-20.
GATE = 2.0 ** -18

CASES = {
    # T, E, k, score, renorm, groups, top_groups, group_top, dtype, bias
    "one_expert": (5, 1, 1, "softmax", True, 1, 1, 2, F32, False),
    "one_token": (1, 64, 8, "sigmoid", True, 8, 4, 2, F32, True),
    "odd_experts": (33, 37, 5, "softmax", False, 1, 1, 2, F32, True),
    "bf16_ties": (200, 64, 8, "softmax", True, 1, 1, 2, BF, False),
    "bf16_groups": (130, 96, 6, "sigmoid", True, 12, 3, 1, BF, True),
    "groups_of_three": (67, 12, 4, "softmax", False, 4, 2, 2, F32, True),
    "groups_of_one": (64, 16, 3, "sigmoid", False, 16, 5, 2, F32, True),
    "no_bias_groups": (90, 40, 7, "sigmoid", False, 5, 3, 2, F32, False),
    "wide": (40, 1000, 16, "softmax", True, 8, 3, 2, F32, True),
    "most_experts": (21, 1024, 16, "sigmoid", True, 64, 2, 2, BF, True),
    "all_of_them": (50, 16, 16, "sigmoid", True, 1, 1, 2, F32, True),
    "many_tokens": (1500, 256, 8, "sigmoid", True, 8, 4, 2, F32, True),
}


def _inputs(T, E, dtype, bias, seed):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g).to(dtype)
    b = 0.05 * torch.randn(E, generator=g) if bias else None
    return logits, b


def _check(logits, b, k, score, renorm, scale, groups, top_groups, group_top, dev_logits=None):
    x = logits.cuda() if dev_logits is None else dev_logits
    idx, gates = smoe.smoe_route_select(x, k, None if b is None else b.cuda(), score=score,
                                        renorm=renorm, scale=scale, groups=groups,
                                        top_groups=top_groups, group_top=group_top)
    ridx, rg = plain.select(logits, k, b, score, renorm, scale, groups, top_groups, group_top)
    assert smoe.smoe_check() == 0
    assert torch.equal(idx.cpu(), ridx)
    assert ((gates.cpu().double() - rg).abs() <= GATE * rg + 1e-37).all()
    return idx, gates, rg


@pytest.mark.parametrize("name", list(CASES))
def test_select(name):
    T, E, k, score, renorm, groups, tg, gt, dtype, bias = CASES[name]
    logits, b = _inputs(T, E, dtype, bias, 3)
    _check(logits, b, k, score, renorm, 2.5 if bias else 1.0, groups, tg, gt)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_select_scores_next_to_one_another(score, groups):
    """Biases that cancel the scores leave every rank within fp32's rounding of the
    others: the choice is the one made in 64 bits."""
    T, E, k = 40, 64, 8
    logits, _ = _inputs(1, E, F32, False, 4)
    s, _, _ = plain.scores(logits, score)
    b = (1.0 - s[0]).float()
    logits = logits.expand(T, E).contiguous()
    g = torch.Generator().manual_seed(5)
    # the rows differ in a few logits, by a few units in the last place
    bump = torch.randint(0, 4, (T, E), generator=g, dtype=torch.int32)
    logits = (logits.view(torch.int32) + bump).view(torch.float32)
    _check(logits, b, k, score, True, 1.0, groups, max(1, groups // 2), 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_select_equal_scores_go_to_the_lower_id(score):
    logits = torch.zeros(9, 48)
    logits[1] = torch.arange(48).remainder(2).float()
    for b in (None, torch.zeros(48)):
        for groups in (1, 6):
            _check(logits, b, 7, score, True, 1.0, groups, max(1, groups // 2), 2)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_select_unavailable_experts(score, renorm, dtype):
    """-inf and NaN logits and biases, rows without any expert, +inf, far negative rows."""
    T, E, k = 12, 24, 6
    logits, b = _inputs(T, E, dtype, True, 6)
    logits[0] = -math.inf
    logits[1] = math.nan
    logits[2, 3:] = -math.inf          # fewer experts than k
    logits[3, ::2] = math.nan
    logits[4, 5] = math.inf
    logits[5, [2, 9]] = math.inf
    logits[6] = -300.0 - torch.arange(E).float()  # sigmoid underflows in fp32
    logits[7, :8] = torch.finfo(dtype).min        # the type's lowest value
    b[20] = -math.inf
    b[21] = math.nan
    for groups, tg in ((1, 1), (4, 2)):
        for bias in (b, None):
            idx, gates, rg = _check(logits, bias, k, score, renorm, 1.0, groups, tg, 2)
            assert all(len(set(r)) == k for r in idx.cpu().tolist())
            assert torch.isfinite(gates).all()
            assert (gates[0] == 0).all() and (gates[1] == 0).all()
            ss, off = smoe.smoe_sort(idx, E)  # always sortable: ids distinct and in range
            assert smoe.smoe_check() == 0 and int(off[-1]) == T * k


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2), (48, 5)])
def test_select_signed_zeros_and_wide_biases(score, groups, top_groups):
    """Zeros of both signs tie; a bias that dwarfs the scores rounds them away in 32 bits."""
    T, E, k = 8, 96, 5
    logits, _ = _inputs(T, E, F32, False, 12)
    logits[0] = 0.0
    logits[0, ::3] = -0.0
    logits[1, 40:] = -0.0
    logits[1, :40] = 0.0
    _check(logits, None, k, score, True, 1.0, groups, top_groups, 2)
    g = torch.Generator().manual_seed(13)
    b = 1000.0 * torch.randint(-3, 4, (E,), generator=g).float()
    _check(logits, b, k, score, True, 1.0, groups, top_groups, 2)
    b[::4] = 3e38
    b[5] = math.inf
    _check(logits, b, k, score, False, 1.0, groups, top_groups, 1)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("E", [24, 33, 130, 512, 1001])
def test_select_bias_of_zeros(E, dtype):
    """The bias a training starts with: equal logits are equal scores."""
    logits, _ = _inputs(60, E, dtype, False, 14)
    _check(logits, torch.zeros(E), min(8, E), "sigmoid", True, 1.0, 1, 1, 2)
    _check(logits, torch.zeros(E), min(8, E), "softmax", False, 1.0, 1, 1, 2)


def test_select_strided_and_given_outputs():
    T, E, k = 45, 20, 4
    wide = torch.randn(T, 64, generator=torch.Generator().manual_seed(7)).cuda()
    x = wide[:, 8:28]
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    gates = torch.empty((T, k), device="cuda")
    out = smoe.smoe_route_select(x, k, score="softmax", topk_idx=idx, gates=gates)
    assert out[0] is idx and out[1] is gates
    ridx, rg = plain.select(x.cpu(), k, None, "softmax", True, 1.0, 1, 1, 2)
    assert torch.equal(idx.cpu(), ridx)
    assert ((gates.cpu() - rg).abs() <= GATE * rg).all()
    dg = torch.randn(T, k, device="cuda")
    assert torch.equal(smoe.smoe_route_select_bwd(x, idx, gates, dg),
                       smoe.smoe_route_select_bwd(x.contiguous(), idx, gates, dg))


def _grad_bound(logits, idx, rg, dg, score, renorm, scale):
    """Sizes that the fp32 errors of each gradient go by."""
    size = torch.zeros(logits.shape, dtype=torch.float64)
    gd = (rg * dg).abs()
    A = gd.sum(1, keepdim=True)
    size.scatter_(1, idx.long(), gd + (rg / scale * A if renorm else 0))
    if score == "softmax" and not renorm:
        size += plain.scores(logits, score)[0] * A
    return size


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("shape", [(1, 8, 3), (37, 61, 5), (300, 256, 16), (65, 1000, 8)])
def test_select_gradient(shape, score, renorm, dtype):
    T, E, k = shape
    scale = 2.5
    logits, b = _inputs(T, E, dtype, True, 8)
    dg = torch.randn(T, k, generator=torch.Generator().manual_seed(9))
    idx, gates, rg = _check(logits, b, k, score, renorm, scale, 1, 1, 2)
    got = smoe.smoe_route_select_bwd(logits.cuda(), idx, gates, dg.cuda(), score=score,
                                     renorm=renorm, scale=scale)
    assert got.dtype == dtype and smoe.smoe_check() == 0
    l64 = logits.double().requires_grad_(True)
    out = plain.gates_of(l64, idx.cpu(), b, score, renorm, scale)
    ref, = torch.autograd.grad((out * dg.double()).sum(), l64)
    # fp32: gates carry GATE, the factors and the difference a few roundings more
    tol = plain.HALF[dtype] * ref.abs() + 4 * GATE * _grad_bound(logits, idx.cpu(), rg, dg, score,
                                                                renorm, scale)
    assert ((got.cpu().double() - ref).abs() <= tol + 1e-37).all()
    # central differences of the loss along a few directions
    v = torch.randn(T, E, generator=torch.Generator().manual_seed(10), dtype=torch.float64)
    h = 1e-5
    f = lambda x: (plain.gates_of(x, idx.cpu(), b, score, renorm, scale) * dg).sum()  # noqa: E731
    num = (f(logits.double() + h * v) - f(logits.double() - h * v)) / (2 * h)
    assert abs(float((ref * v).sum() - num)) <= 1e-6 * float((ref * v).abs().sum()) + 1e-8


def test_select_gradient_of_unavailable_experts_is_zero():
    T, E, k = 6, 16, 4
    logits, _ = _inputs(T, E, F32, False, 11)
    logits[0] = -math.inf
    logits[1, 2:] = math.nan
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            x = logits.cuda()
            idx, gates = smoe.smoe_route_select(x, k, score=score, renorm=renorm)
            dl = smoe.smoe_route_select_bwd(x, idx, gates, torch.ones(T, k, device="cuda"),
                                            score=score, renorm=renorm)
            assert torch.isfinite(dl).all()
            assert (dl[0] == 0).all() and (dl[1, 2:] == 0).all()


def test_select_gradient_reports_bad_ids():
    x = torch.randn(3, 8, device="cuda")
    idx = torch.tensor([[0, 1], [8, 2], [-1, 3]], dtype=torch.int32, device="cuda")
    g = torch.full((3, 2), 0.5, device="cuda")
    dl = smoe.smoe_route_select_bwd(x, idx, g, g, score="sigmoid", renorm=False)
    assert smoe.smoe_check() == -4 and smoe.smoe_check() == 0
    assert (dl[1, [0, 1, 3, 4, 5, 6, 7]] == 0).all() and dl[1, 2] != 0


def test_select_empty_and_repeatable():
    x = torch.empty(0, 8, device="cuda")
    idx, gates = smoe.smoe_route_select(x, 2)
    assert idx.shape == (0, 2)
    assert smoe.smoe_route_select_bwd(x, idx, gates, gates).shape == (0, 8)
    x = torch.randn(700, 128, device="cuda")
    a, b = (smoe.smoe_route_select(x, 8, score="sigmoid") for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_select_in_a_graph_and_on_another_stream():
    x = torch.randn(300, 64, device="cuda")
    want = smoe.smoe_route_select(x, 6, score="sigmoid")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = smoe.smoe_route_select(x, 6, score="sigmoid", stream=st)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    idx, gates = torch.empty_like(want[0]), torch.empty_like(want[1])
    gr = torch.cuda.CUDAGraph()
    buf = x.clone()
    with torch.cuda.graph(gr):
        smoe.smoe_route_select(buf, 6, score="sigmoid", topk_idx=idx, gates=gates)
    for seed in (1, 2):
        buf.copy_(torch.randn(300, 64, generator=torch.Generator().manual_seed(seed)))
        gr.replay()
        want = smoe.smoe_route_select(buf, 6, score="sigmoid")
        assert torch.equal(idx, want[0]) and torch.equal(gates, want[1])


def _few_ranks(T, E, high, seed):
    """Rows of logits far out, where fp32 scores are all alike, in few values (many ties)."""
    g = torch.Generator().manual_seed(seed)
    return (high + torch.randint(0, 3, (T, E), generator=g)).float()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("E", [8, 64, 200, 512, 1001])
def test_select_ties_at_the_border_before_a_near_third(E, dtype):
    """The last selected rank and the next one are equal, and one behind them is not, but
    lies higher in 64 bits: scores that fp32 rounds to one number."""
    k = min(E - 3, 8)
    logits = torch.zeros(3, E)
    logits[0, :3] = torch.tensor([20.0, 20.0, 21.0])
    logits[1, -3:] = torch.tensor([20.0, 20.0, 21.0])
    logits[2, [0, E // 2, E - 1]] = torch.tensor([20.0, 20.0, 21.0])
    _check(logits.to(dtype), torch.zeros(E), 1, "sigmoid", True, 1.0, 1, 1, 2)
    _check(logits.to(dtype), torch.zeros(E), 2, "sigmoid", False, 1.0, 1, 1, 2)
    for kk in (1, k):
        _check(_few_ranks(30, E, 18.0, 20).to(dtype), torch.zeros(E), kk, "sigmoid", True, 1.0, 1, 1, 2)
        _check(_few_ranks(30, E, -20.0, 21).to(dtype), torch.full((E,), 0.5), kk, "sigmoid", True, 1.0, 1, 1, 2)
        # softmax: one expert has all of the mass, and a bias that keeps it behind the others
        logits, b = _few_ranks(30, E, -20.0, 22), torch.full((E,), 0.5)
        logits[:, E // 3], b[E // 3] = 0.0, -5.0
        _check(logits.to(dtype), b, kk, "softmax", False, 1.0, 1, 1, 2)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("E,groups", [(48, 4), (256, 8), (640, 4)])
def test_select_ties_in_groups(E, groups, dtype):
    for high, bias in ((18.0, 0.0), (-20.0, 0.5)):
        _check(_few_ranks(20, E, high, 23).to(dtype), torch.full((E,), bias), 5, "sigmoid", True, 1.0, groups, 2, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(16, 4), (96, 4), (512, 8), (96, 48)])
def test_select_group_sums_beyond_fp32(score, E, groups):
    """Biases of the type's lowest and largest value: the sum of two leaves fp32's range, and
    a group that has experts still ranks before one that has none."""
    low, high = torch.finfo(F32).min, torch.finfo(F32).max
    n = E // groups
    logits, _ = _inputs(6, E, F32, False, 24)
    none = torch.full((E,), -math.inf)
    for fill in (low, high):
        for top_groups in (1, 2):
            for where in ([groups - 1], [1, groups - 1], [0, 2], list(range(1, groups))):
                b = none.clone()
                for g in where:
                    b[g * n:(g + 1) * n] = fill
                _check(logits, b, 2, score, True, 1.0, groups, top_groups, 2)
                b[where[-1] * n] = math.inf
                _check(logits, b, 2, score, True, 1.0, groups, top_groups, 2)
    b = torch.full((E,), low)
    b[(groups - 1) * n:] = low * 0.75
    _check(logits, b, 2, score, True, 1.0, groups, 1, 2)


def test_select_most_rows():
    """2^31 - 1 rows of one expert: the row count and its next multiple of a block's rows leave 32 bits."""
    T = 2 ** 31 - 1
    x = torch.zeros((T, 1), dtype=BF, device="cuda")
    idx = torch.full((T, 1), 7, dtype=torch.int32, device="cuda")
    gates = torch.full((T, 1), 7.0, device="cuda")
    smoe.smoe_route_select(x, 1, score="sigmoid", topk_idx=idx, gates=gates)
    assert smoe.smoe_check() == 0
    assert not bool(idx.any()) and bool((gates == 1).all())
    gates.fill_(0.5)
    dl = smoe.smoe_route_select_bwd(x, idx, gates, gates, score="sigmoid", renorm=False)
    assert smoe.smoe_check() == 0 and bool((dl == 0.125).all())


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("E", [61, 64, 256])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_select_gradient_of_unavailable_experts_under_a_broken_upstream(E, dtype, bad):
    """Masked experts get 0 from a NaN or infinite upstream gradient too, whether or not a
    row is made of whole pieces; every available expert shows it."""
    T, k = 9, 4
    logits, _ = _inputs(T, E, dtype, False, 25)
    mask = torch.rand(T, E, generator=torch.Generator().manual_seed(26)) < 0.4
    logits[mask] = -math.inf
    x = logits.cuda()
    idx, gates = smoe.smoe_route_select(x, k, score="softmax", renorm=False)
    dg = torch.ones(T, k, device="cuda")
    want = smoe.smoe_route_select_bwd(x, idx, gates, dg, score="softmax", renorm=False).cpu()
    dg[2, 1] = bad
    dl = smoe.smoe_route_select_bwd(x, idx, gates, dg, score="softmax", renorm=False).cpu()
    assert smoe.smoe_check() == 0
    assert (dl[mask] == 0).all() and not torch.isfinite(dl[2][~mask[2]]).any()
    keep = [t for t in range(T) if t != 2]
    assert torch.equal(dl[keep], want[keep])
