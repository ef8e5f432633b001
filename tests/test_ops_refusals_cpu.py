"""Refusals of the routing, query/key norm and paged-cache entry points on the host:
every call here is turned down, or is empty, before anything touches a GPU."""
import ctypes
import math

import pytest
import torch

import sparse_mixture_experts_smoe_b200 as smoe

V = ctypes.c_void_p
P = V(0x10000)  # never dereferenced
ARG, UNSUPPORTED = -1, -2


def _call(fn, order, base, **kw):
    a = {**base, **kw}
    return fn(*[ctypes.byref(a[n]) if isinstance(a[n], ctypes.Structure) else a[n] for n in order])


SELECT = dict(logits=P, ld=64, bias=None, T=4, E=64, k=8, score=0, renorm=1, scale=1.0, groups=8,
              top_groups=4, group_top=2, dt=1, idx=P, gates=P, stream=None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(E=0), dict(k=0), dict(k=17), dict(E=2048, ld=2048, k=1), dict(ld=63),
    dict(T=1 << 28), dict(score=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf),
    dict(scale=math.nan), dict(dt=7), dict(groups=0), dict(groups=65, E=65 * 8, ld=65 * 8),
    dict(groups=7), dict(top_groups=0), dict(top_groups=9), dict(group_top=3), dict(group_top=0),
    dict(top_groups=1, k=9), dict(logits=None), dict(idx=None), dict(gates=None),
    dict(logits=V(0x10004))])
def test_select_refuses(kw):
    assert _call(smoe.lib().smoe_route_select, SELECT, SELECT, **kw) == ARG
    assert smoe.lib().smoe_last_error()


SELECT_BWD = dict(logits=P, ld=64, idx=P, gates=P, dgates=P, T=4, E=64, k=8, score=1, renorm=1,
                  scale=1.0, dt=1, dl=P, stream=None)


@pytest.mark.parametrize("kw", [dict(k=65), dict(ld=10), dict(score=-1), dict(scale=0.0), dict(dt=2),
                                dict(logits=None), dict(idx=None), dict(dgates=None), dict(dl=None)],
)
def test_select_bwd_refuses(kw):
    assert _call(smoe.lib().smoe_route_select_bwd, SELECT_BWD, SELECT_BWD, **kw) == ARG


def test_empty_calls_touch_nothing():
    L = smoe.lib()
    none = dict(logits=None, idx=None, gates=None, T=0)
    assert _call(L.smoe_route_select, SELECT, SELECT, **none) == 0
    assert _call(L.smoe_route_select_bwd, SELECT_BWD, SELECT_BWD, dgates=None, dl=None, **none) == 0
    assert _call(L.smoe_moa_qk_norm_rope_fwd, QK, QK, desc=_desc(T=0), q=None, k=None, qo=None, ko=None) == 0
    assert _call(L.smoe_moa_cache_append, APPEND, APPEND, desc=_desc(T=0), cache=_cache(B=0)) == 0
    assert _call(L.smoe_moa_decode, DECODE, DECODE, cache=_cache(B=0), q=None, o=None) == 0


def _desc(T=4, ks=2, qh=2, kvh=2, dh=128, dt=1, norm=1, inter=0, eps=1e-6):
    return smoe.QkDesc(T, ks, qh, kvh, dh, dt, norm, inter, eps)


QK = dict(desc=_desc(), q=P, ldq=256, k=P, ldk=256, slots=None, pos=P, freq=P, wq=P, wk=P, qo=P, ko=P,
          stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(desc=_desc(T=-1)), ARG), (dict(desc=_desc(ks=0)), ARG), (dict(desc=_desc(qh=0)), ARG),
    (dict(desc=_desc(dt=3)), ARG), (dict(desc=_desc(dh=96)), UNSUPPORTED),
    (dict(desc=_desc(eps=0.0)), ARG), (dict(desc=_desc(eps=math.nan)), ARG),
    (dict(desc=_desc(T=1 << 24)), ARG), (dict(desc=_desc(norm=0), freq=None, wq=None, wk=None), ARG),
    (dict(desc=_desc(norm=0)), ARG), (dict(q=None, k=None, qo=None, ko=None), ARG),
    (dict(qo=None), ARG), (dict(k=None), ARG), (dict(pos=None), ARG), (dict(ldq=255), ARG),
    (dict(ldk=260), ARG), (dict(q=V(0x10008)), ARG), (dict(ko=V(0x10004)), ARG),
    (dict(q=V(0x20000), qo=V(0x20000), ldq=512), ARG)])
def test_qk_forward_refuses(kw, rc):
    assert _call(smoe.lib().smoe_moa_qk_norm_rope_fwd, QK, QK, **kw) == rc


QKB = dict(desc=_desc(), dyq=P, lddyq=256, dyk=P, lddyk=256, q=P, ldq=256, k=P, ldk=256, slots=None,
           pos=P, freq=P, wq=P, wk=P, dq=P, dk=P, dwq=P, dwk=P, ws=P, wsb=1 << 30, stream=None)


@pytest.mark.parametrize("kw", [
    dict(dyq=None), dict(dyq=None, dyk=None, dq=None, dk=None, dwq=None, dwk=None), dict(q=None),
    dict(wsb=16), dict(ws=None), dict(ws=V(0x10008)), dict(lddyq=8), dict(dq=V(0x10002)),
    dict(pos=None), dict(desc=_desc(norm=0), wq=None, wk=None)])
def test_qk_backward_refuses(kw):
    assert _call(smoe.lib().smoe_moa_qk_norm_rope_bwd, QKB, QKB, **kw) == ARG


def _cache(B=4, kvh=2, dh=128, pages=8, page=16, max_pages=4, f8=False, **kw):
    st = (page * kvh * dh, kvh * dh, dh)
    c = smoe.KvCache(0x10000, 0x10000, 0x10000 if f8 else None, 0x10000 if f8 else None, 0x10000,
                     0x10000, *st, *st, max_pages, pages, page, max_pages, B, kvh, dh)
    for n, v in kw.items():
        setattr(c, n, v)
    return c


BAD_CACHES = [
    (dict(page=0), ARG), (dict(max_pages=-1), ARG), (dict(page=1 << 20, max_pages=1 << 12), ARG),
    (dict(dh=96), UNSUPPORTED), (dict(k_scale=0x10000), ARG), (dict(table_stride=3), ARG),
    (dict(k_page_stride=4), ARG), (dict(v_token_stride=-256), ARG), (dict(k_page_stride=1 << 36), ARG), (dict(f8=True, k_head_stride=8), ARG),
    (dict(seq_lens=None), ARG), (dict(block_table=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG),
    (dict(v=0x10008), ARG)]
APPEND = dict(desc=_desc(), q=P, ldq=256, k=P, ldk=256, v=P, ldv=256, slots=None, starts=None, freq=P,
              wq=P, wk=P, cache=_cache(), qo=P, stream=None)
DECODE = dict(q=P, ldq=256, slots=None, kslots=2, q_heads=2, cache=_cache(), o=P, lse=None, ws=P,
              wsb=1 << 30, stream=None)


@pytest.mark.parametrize("kw,rc", BAD_CACHES)
def test_caches_are_checked(kw, rc):
    L = smoe.lib()
    assert _call(L.smoe_moa_decode, DECODE, DECODE, cache=_cache(**kw)) == rc
    dh = kw.get("dh", 128)
    assert _call(L.smoe_moa_cache_append, APPEND, APPEND, cache=_cache(**kw), desc=_desc(dh=dh)) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(desc=_desc(dt=0)), UNSUPPORTED), (dict(desc=_desc(kvh=1)), ARG), (dict(desc=_desc(T=5)), ARG),
    (dict(desc=_desc(norm=0)), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(qo=None), ARG),
    (dict(ldv=4), ARG), (dict(q=V(0x20000), qo=V(0x20000), ldq=512), ARG)])
def test_append_refuses(kw, rc):
    assert _call(smoe.lib().smoe_moa_cache_append, APPEND, APPEND, **kw) == rc


@pytest.mark.parametrize("kw", [
    dict(kslots=0), dict(kslots=129), dict(q_heads=3), dict(q_heads=0), dict(q=None), dict(o=None),
    dict(cache=_cache(B=64, page=1 << 18, max_pages=1 << 12)), dict(ldq=250), dict(ws=None), dict(wsb=64), dict(ws=V(0x10010)), dict(o=V(0x10004))])
def test_decode_refuses(kw):
    assert _call(smoe.lib().smoe_moa_decode, DECODE, DECODE, **kw) == ARG


def test_workspace_sizes():
    L = smoe.lib()
    size = L.smoe_moa_decode_workspace_size
    assert size(4, 2, 3, 2, 128) == 0 and size(4, 0, 2, 2, 128) == 0 and size(4, 2, 2, 2, 96) == 0
    assert 0 < size(4, 2, 2, 2, 64) < size(4, 2, 2, 2, 128)
    assert L.smoe_moa_qk_norm_rope_bwd_workspace_size(ctypes.byref(_desc(dh=96))) == 0
    assert L.smoe_moa_qk_norm_rope_bwd_workspace_size(ctypes.byref(_desc())) > 0


def test_python_refuses_tensors_off_the_gpu():
    x = torch.zeros(4, 8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    c = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16)
    for f in (lambda: smoe.smoe_route_select(x, 2), lambda: smoe.smoe_route_select(None, 2),
              lambda: smoe.smoe_route_select_bwd(x, i, x, x),
              lambda: smoe.smoe_moa_qk_norm_rope_fwd(c.view(-1, 64), None, None, 1, q_heads=1, kv_heads=1),
              lambda: smoe.smoe_moa_cache_append(None, x, x, c, c, i, i[0], None, 1, 1),
              lambda: smoe.smoe_moa_decode(x, c, c, i, i[0], None, 1, 1)):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(ValueError):
        smoe.smoe_moa_qk_norm_rope_fwd(None, None, None, 1, q_heads=1, kv_heads=1)
