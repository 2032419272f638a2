"""The key/value cache entry points without a GPU: refusals before anything is launched, and the plain bookkeeping."""
import ctypes

import pytest
import torch

import gemm_affine_int4_gb300 as g4
from kv_ref import plan_reference

P = ctypes.c_void_p
A = P(0x10000)


def plan(**c):
    a = dict(kv=A, q=A, table=A, width=4, free=A, cap=64, count=A, slots=A, pos=A, T=8, cu=A, kvo=P(0x20000),
             co=P(0x20000), info=A, B=4, page=16)
    a.update(c)
    return g4.lib().gai4_kv_plan(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(kv=None), 1), (dict(table=None), 1), (dict(info=None), 1), (dict(slots=None), 1), (dict(width=0), 1),
    (dict(cap=0), 1), (dict(T=-1), 1), (dict(B=0), 1), (dict(B=8193), 2), (dict(page=48), 2), (dict(page=8), 2),
    (dict(page=512), 2), (dict(slots=P(0x10004)), 3), (dict(kv=P(0x10002)), 3), (dict(kvo=A), 1), (dict(co=A), 1),
    (dict(width=1 << 40), 1), (dict(T=1 << 32), 1)])
def test_plan_refusals(change, status):
    assert plan(**change) == status


def append(**c):
    a = dict(k=A, ks=1024, v=A, vs=1024, slots=A, kp=A, ksc=A, kb=A, vp=A, vsc=A, vb=A, dt=2, gs=64, T=3, hkv=8, d=128,
             nb=10, page=64)
    a.update(c)
    return g4.lib().gai4_kv_append(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(k=None), 1), (dict(kp=None), 1), (dict(vb=None), 1), (dict(slots=None), 1), (dict(ks=1023), 1),
    (dict(vs=0), 1), (dict(T=-1), 1), (dict(hkv=0), 1), (dict(nb=0), 1), (dict(dt=3), 2), (dict(gs=16), 2),
    (dict(gs=128, d=64, ks=512), 2), (dict(d=96), 2), (dict(page=20), 2), (dict(kp=P(0x10004)), 3),
    (dict(vsc=P(0x10008)), 3), (dict(k=P(0x10001)), 3), (dict(dt=0, k=P(0x10002)), 3), (dict(slots=P(0x10004)), 3),
    (dict(T=0), 0), (dict(T=0, k=None, v=None, slots=None), 0)])
def test_append_refusals(change, status):
    assert append(**change) == status


@pytest.mark.parametrize("change,status", [
    (dict(out=None), 1), (dict(out=P(0x10008)), 3), (dict(slots=None), 1), (dict(p=None), 1), (dict(gs=48), 2),
    (dict(T=0, out=None, slots=None), 0)])
def test_read_refusals(change, status):
    a = dict(p=A, s=A, b=A, slots=A, out=A, dt=2, gs=64, T=3, hkv=8, d=128, nb=10, page=64)
    a.update(change)
    assert g4.lib().gai4_kv_read(*a.values(), None) == status


def attention(**c):
    a = dict(q=A, qs=4096, kp=A, ksc=A, kb=A, vp=A, vsc=A, vb=A, table=A, width=4, kv=A, cu=A, out=A, os=4096, lse=None,
             dt=2, gs=64, B=2, T=2, max_q=1, hq=32, hkv=8, d=128, nb=10, page=64, scale=0.1, window=0, ws=A,
             ws_bytes=1 << 40)
    a.update(c)
    return g4.lib().gai4_kv_attention(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(kp=None), 1), (dict(table=None), 1), (dict(kv=None), 1),
    (dict(cu=None), 1), (dict(qs=4095), 1), (dict(os=100), 1), (dict(B=0), 1), (dict(T=-1), 1), (dict(max_q=-1), 1),
    (dict(hq=33), 1), (dict(hq=0), 1), (dict(hkv=0), 1), (dict(window=-1), 1), (dict(width=0), 1), (dict(nb=0), 1),
    (dict(dt=5), 2), (dict(gs=256), 2), (dict(d=80), 2), (dict(page=100), 2), (dict(q=P(0x10001)), 3),
    (dict(kp=P(0x10008)), 3), (dict(cu=P(0x10002)), 3), (dict(ws=P(0x10004)), 3), (dict(T=0), 0)])
def test_attention_refusals(change, status):
    assert attention(**change) == status


def test_workspace_refusals():
    need = g4.gai4_kv_attention_workspace_bytes(32, 8, 128, torch.bfloat16)
    if need:
        assert attention(ws=None) == g4.GAI4_ERR_WORKSPACE
        assert attention(ws_bytes=need - 1) == g4.GAI4_ERR_WORKSPACE
    assert g4.lib().gai4_kv_attention_workspace_bytes(33, 8, 128, 2) == 0
    assert g4.lib().gai4_kv_attention_workspace_bytes(32, 8, 100, 2) == 0


def test_binding_refuses_wrong_shapes():
    kc = g4.gai4_kv_cache(2, 2, 16, 64, 32, torch.float32, device="cpu")
    x = torch.zeros(3, 2, 64)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        g4.gai4_kv_append(x[:, :1], x, slots, kc, kc, group_size=32)          # heads
    with pytest.raises(ValueError):
        g4.gai4_kv_append(x, x, slots.int(), kc, kc, group_size=32)           # slot type
    with pytest.raises(ValueError):
        g4.gai4_kv_append(x.half(), x.half(), slots, kc, kc, group_size=32)   # type
    with pytest.raises(ValueError):
        g4.gai4_kv_append(x, x, slots, kc, kc, group_size=64)                 # group size
    with pytest.raises(ValueError):
        g4.gai4_kv_append(x, x, slots, kc, kc, group_size=32)                 # not on a GPU


def test_plain_bookkeeping_keeps_every_page_once():
    """The reference itself: pages in rows and on the free stack stay a partition of the pool."""
    import random
    rng = random.Random(5)
    page, width, nb, B = 16, 6, 60, 9
    table, kv, free, count = [[-1] * width for _ in range(B)], [0] * B, list(range(nb)), nb
    for _ in range(200):
        q = [-1 if rng.random() < 0.1 else min(rng.choice([0, 1, 1, 20]), width * page - k) for k in kv]
        p = plan_reference(kv, q, table, free, count, page, 400)
        assert p["info"][:1] == [0] and not any(p["info"])
        table, free, count, kv = p["table"], p["free"], p["count"], p["kv_lens"]
        held = [b for r in range(B) for b in table[r][:-(-kv[r] // page)]]
        assert sorted(held + free[:count]) == list(range(nb))
