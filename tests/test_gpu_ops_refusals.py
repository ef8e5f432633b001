"""Refusals of the routing, norm and cache calls on tensors of the wrong kind: an error of
the class that says what is wrong, nothing launched, outputs left alone."""
import pytest
import torch

import sparse_mixture_experts_smoe_b200 as smoe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _select(**kw):
    a = dict(logits=_z(4, 16), k=2, bias=None)
    a.update(kw)
    return smoe.smoe_route_select(a.pop("logits"), a.pop("k"), a.pop("bias"), **a)


@pytest.mark.parametrize("kw,error", [
    (dict(bias="short"), ValueError),
    (dict(bias="half"), TypeError), (dict(bias="cpu"), TypeError), (dict(logits="half"), TypeError),
    (dict(logits="column"), ValueError), (dict(k=17), smoe.SmoeError), (dict(k=0), smoe.SmoeError),
    (dict(groups=3), smoe.SmoeError), (dict(score="tanh"), ValueError), (dict(scale=-1.0), smoe.SmoeError),
    (dict(topk_idx="long"), TypeError), (dict(gates="strided"), ValueError)])
def test_select(kw, error):
    make = {"half": lambda n: _z(4, 16).half() if n == "logits" else _z(16).half(),
            "cpu": lambda n: torch.zeros(16), "short": lambda n: _z(15), "column": lambda n: _z(16, 4).t(),
            "long": lambda n: _z(4, 2, dtype=torch.int64), "strided": lambda n: _z(4, 4)[:, ::2]}
    kw = {n: make[v](n) if isinstance(v, str) and v in make else v for n, v in kw.items()}
    with pytest.raises(error):
        _select(**kw)


def test_select_gradient():
    x, i, g = _z(4, 16), _z(4, 2, dtype=torch.int32), _z(4, 2)
    for a in ((x, i[:3], g, g), (x, i, g[:, :1], g), (x, i, g, g.double()), (x, i.long(), g, g)):
        with pytest.raises((ValueError, TypeError)):
            smoe.smoe_route_select_bwd(*a)


def test_qk_norm():
    q, k, w, pos = _z(8, 128, dtype=BF), _z(4, 128, dtype=BF), _z(64), _z(4, dtype=torch.int32)
    kw = dict(q_heads=2, kv_heads=2, wq=w, wk=w, positions=pos, inv_freq=_z(32))
    call = lambda q=q, k=k, s=None, ks=2, **o: smoe.smoe_moa_qk_norm_rope_fwd(q, k, s, ks, **{**kw, **o})  # noqa: E731
    call()
    for bad, error in ((dict(q=q[:7]), ValueError), (dict(k=k.float()), TypeError), (dict(wq=_z(63)), ValueError),
                       (dict(positions=pos.long()), TypeError), (dict(inv_freq=_z(64)), ValueError),
                       (dict(s=_z(7, dtype=torch.int32)), ValueError), (dict(q_heads=3), ValueError),
                       (dict(positions=None), smoe.SmoeError), (dict(eps=0.0), smoe.SmoeError),
                       (dict(norm=False), smoe.SmoeError), (dict(ks=0), ValueError), (dict(kv_heads=3), ValueError),
                       (dict(q=None, q_out=q), ValueError),
                       (dict(q=_z(8, 136, dtype=BF)[:, 1:129]), smoe.SmoeError),
                       (dict(q=_z(8, 132, dtype=BF)[:, :128]), smoe.SmoeError)):
        with pytest.raises(error):
            call(**bad)
    with pytest.raises(ValueError):
        smoe.smoe_moa_qk_norm_rope_bwd(q, k, None, k, None, 2, **kw)


def _cache_args(f8=False):
    c = lambda: _z(4, 16, 2, 64, dtype=torch.uint8 if f8 else BF)  # noqa: E731
    return dict(k_cache=c(), v_cache=c(), block_table=_z(3, 2, dtype=torch.int32), seq_lens=_z(3, dtype=torch.int32),
                k_scale=_z(4, 16, 2) if f8 else None, v_scale=_z(4, 16, 2) if f8 else None)


CACHES = {
    "expanded": lambda a: a.update(k_cache=a["k_cache"][:1].expand(4, 16, 2, 64)),
    "other_shape": lambda a: a.update(v_cache=a["v_cache"][:3]),
    "other_type": lambda a: a.update(v_cache=a["v_cache"].float()),
    "one_scale": lambda a: a.update(k_scale=_z(4, 16, 2)),
    "scales_of_bf16": lambda a: a.update(k_scale=_z(4, 16, 2), v_scale=_z(4, 16, 2)),
    "lengths": lambda a: a.update(seq_lens=a["seq_lens"][:2]),
    "long_lengths": lambda a: a.update(seq_lens=a["seq_lens"].long()),
    "table": lambda a: a.update(block_table=a["block_table"].t()),
    "three_dims": lambda a: a.update(k_cache=a["k_cache"][0]),
    "inside_heads": lambda a: a.update(k_cache=_z(4, 16, 2, 128, dtype=BF)[..., ::2]),
    "odd_stride": lambda a: a.update(k_cache=_z(4, 16, 2, 68, dtype=BF)[..., :64]),
}


@pytest.mark.parametrize("name", list(CACHES))
def test_caches(name):
    a = _cache_args()
    CACHES[name](a)
    k = torch.ones(3, 128, dtype=BF, device="cuda")
    with pytest.raises((ValueError, TypeError, smoe.SmoeError)):
        smoe.smoe_moa_cache_append(None, k, k, sorted_slot=None, kslots=1, q_heads=2, norm=False, **a)
    if name != "expanded":  # a cache that is only read may be one
        with pytest.raises((ValueError, TypeError, smoe.SmoeError)):
            smoe.smoe_moa_decode(k, sorted_slot=None, kslots=1, q_heads=2, **a)
    assert smoe.smoe_check() == 0


def test_append_and_decode():
    for f8 in (False, True):
        a = _cache_args(f8)
        k = torch.ones(3, 128, dtype=BF, device="cuda")
        good = dict(q=k, sorted_slot=None, kslots=1, q_heads=2)
        o, lse = smoe.smoe_moa_decode(**good, **a)
        for bad in (dict(q=k.float()), dict(q=k[:2]), dict(kslots=2), dict(q_heads=3), dict(q_heads=1),
                    dict(sorted_slot=_z(2, dtype=torch.int32)), dict(o=o.float()), dict(lse=lse[:2])):
            with pytest.raises((ValueError, TypeError, smoe.SmoeError)):
                smoe.smoe_moa_decode(**{**good, **bad}, **a)
        good = dict(q=k, k=k, v=k, sorted_slot=None, kslots=1, q_heads=2, norm=False)
        for bad in (dict(k=k[:2]), dict(v=k[:2]), dict(v=k.float()), dict(starts=_z(3, dtype=torch.int32)),
                    dict(q=None, q_out=k), dict(q_out=k[:, ::2]), dict(wq=_z(64)), dict(inv_freq=_z(64))):
            with pytest.raises((ValueError, TypeError, smoe.SmoeError)):
                smoe.smoe_moa_cache_append(**{**good, **bad}, **a)
        assert (a["k_cache"].float() == 0).all() and smoe.smoe_check() == 0


def test_outputs_over_inputs():
    """A given output that shares memory with an input is refused, but for the calls that
    work in place."""
    x = _z(8, 16)
    with pytest.raises(ValueError, match="overlap"):
        smoe.smoe_route_select(x, 16, gates=x)
    with pytest.raises(ValueError, match="overlap"):
        smoe.smoe_route_select(x, 16, topk_idx=x.view(torch.int32))
    idx, gates = smoe.smoe_route_select(x, 2)
    with pytest.raises(ValueError, match="overlap"):
        smoe.smoe_route_select_bwd(x, idx, gates, gates, dlogits=x)
    with pytest.raises(ValueError, match="overlap"):  # the rows of a wider tensor
        smoe.smoe_route_select_bwd(_z(8, 32)[:, :16], idx, x[0].view(8, 2), gates, dlogits=x)
    buf = _z(3, 8, 128, dtype=BF).flatten()
    q, k = buf[:1024].view(8, 128), buf[1024:1536].view(4, 128)
    kw = dict(q_heads=2, kv_heads=2)
    smoe.smoe_moa_qk_norm_rope_fwd(q, k, None, 2, q_out=q, k_out=k, **kw)
    smoe.smoe_moa_qk_norm_rope_fwd(q, k, None, 2, q_out=buf[1536:2560].view(8, 128), **kw)
    for o in (dict(q_out=buf[64:1088].view(8, 128)), dict(k_out=buf[1152:1664].view(4, 128)),
              dict(q_out=buf[512:1536].view(8, 128)), dict(k_out=buf[:512].view(4, 128))):
        with pytest.raises(ValueError, match="overlap"):
            smoe.smoe_moa_qk_norm_rope_fwd(q, k, None, 2, **o, **kw)
    a = _cache_args()
    rows = _z(9, 128, dtype=BF)
    a["block_table"] += 1
    good = dict(sorted_slot=None, kslots=1, q_heads=2)
    smoe.smoe_moa_cache_append(rows[:3], rows[3:6], rows[6:], q_out=rows[:3], norm=False, **good, **a)
    for at in (1, 3, 5, 6):
        with pytest.raises(ValueError, match="overlap"):
            smoe.smoe_moa_cache_append(rows[:3], rows[3:6], rows[6:], q_out=rows[at:at + 3], norm=False, **good, **a)
    smoe.smoe_moa_decode(rows[:3], o=rows[3:6], **good, **a)
    with pytest.raises(ValueError, match="overlap"):
        smoe.smoe_moa_decode(rows[:3], o=rows[:3], **good, **a)
    with pytest.raises(ValueError, match="overlap"):
        smoe.smoe_moa_decode(rows[:3], lse=rows.view(torch.float32)[0, :6].view(3, 2), **good, **a)
    # a cache whose keys and values are one tensor cannot be written
    a["v_cache"] = a["k_cache"]
    with pytest.raises(ValueError, match="overlap"):
        smoe.smoe_moa_cache_append(None, rows[:3], rows[:3], norm=False, **good, **a)
    assert smoe.smoe_check() == 0
