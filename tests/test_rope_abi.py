"""Rotary entry points: what they refuse, on the host, before anything is launched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def kv4():
    from int4_kv_cache_append_b200 import kv4
    return kv4


def rope_cfg(kv4, **kw):
    base = dict(rotary_dim=128, max_pos=64, layout=0, base=10000.0)
    base.update(kw)
    return kv4.RopeGeometry(**base).c()


@pytest.mark.parametrize("kw,status", [
    (dict(rotary_dim=0), 1), (dict(rotary_dim=12), 2), (dict(rotary_dim=136), 2), (dict(max_pos=0), 1), (dict(base=1.0), 1),
    (dict(base=float("nan")), 1), (dict(base=float("inf")), 1), (dict(scaling=9), 1), (dict(scaling=1, factor=0.0), 1),
    (dict(scaling=2, factor=float("inf")), 1), (dict(scaling=3, factor=4.0), 1), (dict(scaling=3, factor=4.0, original_max_pos=64, beta_fast=1.0), 1),
    (dict(scaling=4, factor=4.0), 1), (dict(scaling=4, factor=4.0, original_max_pos=64, low_freq_factor=4.0), 1),
    (dict(attention_factor=-1.0), 1),
])
def test_table_refusals(kv4, kw, status):
    assert kv4.lib.kv4_rope_table(ctypes.byref(rope_cfg(kv4, **kw)), ctypes.c_void_p(1 << 20), None) == status


def test_table_pointer_refusals(kv4):
    assert kv4.lib.kv4_rope_table(ctypes.byref(rope_cfg(kv4)), None, None) == 1
    assert kv4.lib.kv4_rope_table(ctypes.byref(rope_cfg(kv4)), ctypes.c_void_p((1 << 20) + 8), None) == 1
    assert kv4.lib.kv4_rope_table(None, ctypes.c_void_p(1 << 20), None) == 1


V = ctypes.c_void_p
A = 1 << 20  # an aligned address that nothing reads


def params(kv4, **kw):
    base = dict(table=A, max_pos=64, rotary_dim=64, layout=0, weight_dtype=0, q_weight=None, k_weight=None, eps=1e-6)
    base.update(kw)
    return kv4.kv4_rope_params(**base)


def rope(kv4, p, T=2, Hq=4, Hkv=2, D=64, q=A, qd=1, qs=None, k=A, kd=1, ks=None, pos=A, qo=A, qod=1, qos=None, ko=A, kod=1, kos=None):
    d = lambda s, H: H * D if s is None else s  # noqa: E731
    return kv4.lib.kv4_rope(ctypes.byref(p) if p is not None else None, T, Hq, Hkv, D, V(q), qd, d(qs, Hq), V(k), kd, d(ks, Hkv), V(pos),
                            V(qo), qod, d(qos, Hq), V(ko), kod, d(kos, Hkv), None)


@pytest.mark.parametrize("kw,status", [
    (dict(table=None), 1), (dict(table=A + 8), 1), (dict(max_pos=0), 1), (dict(rotary_dim=0), 1), (dict(rotary_dim=72), 1), (dict(rotary_dim=20), 2),
    (dict(layout=2), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(q_weight=A, weight_dtype=5), 1), (dict(k_weight=A + 4, weight_dtype=1), 1),
])
def test_params_refusals(kv4, kw, status):
    assert rope(kv4, params(kv4, **kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(Hq=-1), 1), (dict(D=96), 2), (dict(q=None), 1), (dict(ko=None), 1), (dict(pos=None), 1), (dict(q=A + 4), 1),
    (dict(q=A + 8, qd=0), 1), (dict(qs=255), 1), (dict(qs=258), 1), (dict(ks=100), 1), (dict(kd=3), 1), (dict(qod=2), 1), (dict(qos=512), 1),
    (dict(T=1 << 25, Hq=4, Hkv=2), 2), (dict(T=0), 0), (dict(Hq=0, Hkv=0), 0),
])
def test_rope_refusals(kv4, kw, status):
    assert rope(kv4, params(kv4), **kw) == status


def test_rope_null_params(kv4):
    assert rope(kv4, None) == 1


def _cfg(kv4, **kw):
    base = dict(num_layers=2, num_q_heads=4, num_kv_heads=2, head_dim=64, page_size=16, num_sinks=4, recent_window=16, hadamard_block=64, max_seqs=8,
                max_pages=10)
    base.update(kw)
    return kv4.kv4_config(**base)


def append(kv4, h, p, layer=0, T=2, q=A, qd=1, qs=256, k=A, kd=1, ks=128, v=A, vd=1, vs=128, slot=A, pos=A, la=A, pt=A, stride=1, qo=A, qod=1, qos=256):
    return kv4.lib.kv4_append_rope(V(h), layer, T, ctypes.byref(p), V(q), qd, qs, V(k), kd, ks, V(v), vd, vs, V(slot), V(pos), V(la), V(pt), stride, V(qo),
                                   qod, qos, None)


def test_append_and_gather_refusals(kv4):
    h = kv4.kv4_cache_init(_cfg(kv4), 1 << 20, 1 << 21)
    m = kv4.kv4_cache_init(_cfg(kv4, num_sinks=0, recent_window=0, hadamard_block=1, value_format=2, key_bits=3, value_bits=3), 1 << 20, 0)
    b = kv4.kv4_bf16_cache_init(_cfg(kv4), 1 << 20)
    try:
        p = params(kv4)
        for kw in (dict(layer=2), dict(layer=-1), dict(T=-1), dict(stride=0), dict(slot=None), dict(pos=None), dict(la=None), dict(pt=None), dict(k=None),
                   dict(v=None), dict(ks=127), dict(ks=130), dict(v=A + 2), dict(qo=None), dict(qod=0), dict(qd=7)):
            assert append(kv4, h, p, **kw) == 1, kw
        assert append(kv4, None, p) == 1
        assert append(kv4, h, params(kv4, rotary_dim=128)) == 1
        assert append(kv4, h, p, T=1 << 25) == 2
        assert append(kv4, h, p, T=0) == 0
        assert append(kv4, m, p) == 6
        g = lambda h, layer=0, T=2, slot=A, pos=A, pt=A, stride=1, k=A, v=A, dt=1: kv4.lib.kv4_gather(  # noqa: E731
            V(h), layer, T, V(slot), V(pos), None, V(pt), stride, V(k), V(v), dt, None)
        for kw in (dict(layer=2), dict(T=-1), dict(slot=None), dict(pos=None), dict(pt=None), dict(stride=0), dict(k=A + 8), dict(v=A + 4), dict(dt=3)):
            assert g(h, **kw) == 1, kw
        assert g(None) == 1
        assert g(m) == 6
        assert g(h, T=0) == 0 and g(h, k=None, v=None) == 0 and g(b, T=0) == 0
        assert g(h, T=1 << 26) == 2
    finally:
        for x in (h, m, b):
            kv4.kv4_cache_destroy(x)
