"""Rotary table, norm and rotation, fused append and read-back on the GPU against NumPy and the CPU
oracle.

The arithmetic up to the quantiser is fixed step by step, so fp32 outputs and cache bytes are
compared exactly.  A 16-bit output is the fp32 value rounded to nearest."""
import dataclasses

import numpy as np
import pytest
import torch

from int4_kv_cache_append_b200 import workload as W
from oracle import oracle as O

import kv4_testlib as T
import rope_ref as R

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def kv4():
    from int4_kv_cache_append_b200 import kv4
    return kv4


@pytest.fixture(autouse=True)
def no_device_error(kv4):
    yield
    assert kv4.kv4_get_device_error() == 0


def rand(shape, dt, seed, scale=1.0):
    g = np.random.default_rng(seed)
    return torch.from_numpy((g.standard_normal(shape) * scale).astype(np.float32)).to(TYPES[dt]).cuda()


def f32(t):
    return t.float().cpu().numpy()


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


@pytest.mark.parametrize("scaling,kw", [
    ("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=2.0)), ("yarn", dict(factor=4.0, orig=4096)), ("yarn", dict(factor=8.0, orig=40)),
    ("bands", dict(factor=8.0, orig=8192)),
])
@pytest.mark.parametrize("dim,max_pos,base", [(8, 1, 10000.0), (64, 1000, 10000.0), (128, 131072, 1000000.0), (24, 33, 500000.0)])
def test_table(kv4, scaling, kw, dim, max_pos, base):
    code = dict(none=0, linear=1, ntk=2, yarn=3, bands=4)[scaling]
    geo = kv4.RopeGeometry(dim, max_pos, 0, base, code, kw.get("factor", 1.0), kw.get("orig", 0))
    guard = torch.full((max_pos * dim + 64,), 7.0, device="cuda")
    kv4.kv4_rope_table(geo.c(), guard)
    got = guard[:max_pos * dim].view(max_pos, dim // 2, 2).cpu().numpy().astype(np.float64)
    assert bool((guard[max_pos * dim:] == 7.0).all())
    ref = R.table64(*R.frequencies(dim, base, scaling, **kw), max_pos)
    # half a step of fp32, and the angle: at most 1.3e5 rad, its frequency and product a few 2^-53 off
    assert np.all(np.abs(got - ref) <= np.abs(ref) * 2.0 ** -24 + 1e-9)


# (T, Hq, Hkv, D, R, layout, q type, out type, weight type or None)
ROPE_CASES = [
    (1, 4, 2, 64, 64, 0, "bf16", "f32", "bf16"), (7, 32, 8, 128, 128, 0, "bf16", "f32", "bf16"), (7, 5, 3, 128, 128, 1, "f32", "f32", "f32"),
    (130, 32, 8, 128, 64, 1, "bf16", "bf16", "f32"), (33, 8, 1, 64, 24, 0, "f16", "f16", "f16"), (33, 8, 1, 128, 8, 1, "f16", "f32", None),
    (64, 32, 8, 128, 120, 0, "f32", "f32", None), (700, 32, 8, 128, 128, 0, "bf16", "f32", "bf16"), (3, 0, 2, 64, 64, 1, "bf16", "f32", "f32"),
    (2, 1, 0, 64, 8, 0, "f32", "bf16", "f32"),
]


@pytest.mark.parametrize("case", ROPE_CASES, ids=[str(c) for c in ROPE_CASES])
def test_rope_matches(kv4, case):
    n, Hq, Hkv, D, dim, layout, dt, odt, wdt = case
    geo = kv4.RopeGeometry(dim, 5000, layout, 10000.0)
    qw, kw = (rand((D,), wdt, s) if wdt else None for s in (1, 2))
    rope = kv4.Rope(geo, qw, kw, eps=1e-6)
    fused = rand((n, (Hq + 2 * Hkv) * D), dt, 3, 2.0)
    q = fused[:, :Hq * D].view(n, Hq, D) if Hq else None
    k = fused[:, Hq * D:(Hq + Hkv) * D].view(n, Hkv, D) if Hkv else None
    pos = i32(np.random.default_rng(4).integers(0, 5000, n))
    outs = [torch.full((n, x.shape[1], D), 9.0, dtype=TYPES[odt], device="cuda") if x is not None else None for x in (q, k)]
    rope.apply(q, k, pos, *outs)
    table = rope.table.cpu().numpy()
    for x, w, o in ((q, qw, outs[0]), (k, kw, outs[1])):
        if x is None:
            continue
        ref = R.rope32(f32(x), f32(w) if w is not None else None, 1e-6, table, pos.cpu().numpy(), dim, layout)
        assert np.array_equal(f32(o), f32(torch.from_numpy(ref).to(TYPES[odt])))


def test_rope_in_place_and_strided(kv4):
    n, Hq, Hkv, D = 19, 8, 2, 128
    rope = kv4.Rope(kv4.RopeGeometry(D, 64), rand((D,), "f32", 1), rand((D,), "f32", 2))
    fused = rand((n, (Hq + 2 * Hkv) * D), "bf16", 3)
    keep = fused.clone()
    pos = i32(np.arange(n))
    ref = rope.apply(keep[:, :Hq * D].view(n, Hq, D), keep[:, Hq * D:(Hq + Hkv) * D].view(n, Hkv, D), pos)
    q, k = fused[:, :Hq * D].view(n, Hq, D), fused[:, Hq * D:(Hq + Hkv) * D].view(n, Hkv, D)
    rope.apply(q, k, pos, q, k)
    assert torch.equal(q, ref[0]) and torch.equal(k, ref[1])
    assert torch.equal(fused[:, (Hq + Hkv) * D:], keep[:, (Hq + Hkv) * D:])


def test_rope_padding_and_bad_positions(kv4):
    rope = kv4.Rope(kv4.RopeGeometry(64, 16))
    q = rand((4, 2, 64), "f32", 5)
    out = torch.full_like(q, 3.0)
    rope.apply(q, None, i32([0, -1, 15, -1]), out)
    assert kv4.kv4_get_device_error() == 0
    assert bool((out[1] == 3).all()) and bool((out[3] == 3).all()) and torch.equal(out[0], q[0])
    out.fill_(3.0)
    rope.apply(q, None, i32([16, 1, -2, 2]), out)
    assert kv4.kv4_get_device_error() == kv4.KV4_DEVERR_LENGTH
    assert bool((out[0] == 3).all()) and bool((out[2] == 3).all()) and not bool((out[1] == 3).all())


def test_norm_extremes(kv4):
    """Zero vectors, vectors whose squares leave the fp32 range (r is then 0, or 1 / sqrt(eps)), infinities."""
    D = 128
    w = torch.ones(D, device="cuda")
    x = rand((6, 1, D), "f32", 8)
    x[1] = 0
    x[2] *= 1e25
    x[3] *= 1e-30
    x[4, 0, 3] = float("inf")
    x[5, 0, 0] = float("nan")
    rope = kv4.Rope(kv4.RopeGeometry(8, 4), w, None, eps=1e-6)
    out, _ = rope.apply(x, None, i32([0] * 6))
    with np.errstate(all="ignore"):
        ref = R.rope32(f32(x), f32(w), 1e-6, rope.table.cpu().numpy(), np.zeros(6, int), 8, 0)
    assert np.array_equal(f32(out), ref, equal_nan=True)


# (name, D, G, Hkv, P, s, w, h, lens, rotary dim, layout, k type, v type, value_format, rotate values, signs)
APPEND_CASES = [
    ("int4-d128", 128, 4, 2, 16, 4, 16, 128, (300, 37, 1, 4, 5, 20, 21, 129), 128, 0, "bf16", "bf16", 0, False, None),
    ("int4-d64-p48", 64, 2, 3, 48, 2, 8, 64, (50, 17, 3, 97), 24, 1, "f32", "f16", 0, False, None),
    ("int4-signs-rotv", 128, 1, 2, 32, 0, 24, 32, (90, 24, 25, 2), 128, 1, "bf16", "f32", 0, True, (0x9E3779B9, 0x12345678, 0xDEADBEEF, 0x0F0F0F0F)),
    ("int4-no-side", 128, 2, 1, 64, 0, 0, 1, (65, 64), 64, 0, "f16", "bf16", 0, False, None),
    ("vbf", 128, 4, 2, 16, 4, 16, 128, (120, 33), 128, 0, "bf16", "bf16", 1, False, None),
    ("vbf-d64", 64, 1, 2, 16, 19, 13, 16, (100, 19, 20, 31), 64, 1, "f32", "f32", 1, False, None),
]


def tokens(wl, dt, seed, heads, scale=1.0):
    b, p = T.prefill_tokens(wl.lens)
    return b, p, rand((b.size, heads, wl.D), dt, seed, scale)


@pytest.mark.parametrize("case", APPEND_CASES, ids=[c[0] for c in APPEND_CASES])
@pytest.mark.parametrize("norm", [True, False], ids=["norm", "plain"])
def test_append_bytes_exact(kv4, case, norm):
    name, D, G, Hkv, P, s, w, h, lens, dim, layout, kdt, vdt, vf, rotv, signs = case
    wl = W.make_workload(name, 17, 1, len(lens), G * Hkv, Hkv, D, P, s, w, h, lambda r: list(lens), W.F32, W.F32, W.F32, 2, 20.0)
    cache = kv4.Cache(T.geometry(wl, value_format=vf), fill=0xA5)
    if signs:
        kv4.kv4_set_rotation_signs(cache.handle, signs)
    if rotv:
        kv4.kv4_set_value_rotation(cache.handle, True)
    qw, kw = (rand((D,), "f32", i) if norm else None for i in (1, 2))
    rope = kv4.Rope(kv4.RopeGeometry(dim, 512, layout, 10000.0), qw, kw)
    b, p, K = tokens(wl, kdt, 5, Hkv)
    V = tokens(wl, vdt, 6, Hkv)[2]
    q = tokens(wl, "bf16", 7, wl.Hq)[2]
    pt = torch.from_numpy(wl.page_table).cuda()
    q_out = torch.zeros(q.shape, device="cuda")
    cache.append_rope(0, rope, q, K, V, i32(b), i32(p), i32(wl.lens), pt, q_out=q_out)
    table = rope.table.cpu().numpy()
    Kr = R.rope32(f32(K), f32(kw) if norm else None, 1e-6, table, p, dim, layout)
    cfg = O.Config(wl.Hq, Hkv, D, P, s, w, h, wl.B, signs or (0, 0, 0, 0), int(rotv), vf)
    pool = np.full(O.page_bytes(cfg) * max(wl.num_pages, 1), 0xA5, np.uint8)
    side = np.full(O.side_slot_bytes(cfg) * wl.B, 0xA5, np.uint8)
    O.append(cfg, pool, side, Kr, f32(V), b, p, wl.lens, wl.page_table, O.F32, O.F32)
    gp, gs = cache.layer_views(0)
    assert np.array_equal(gp.cpu().numpy(), pool) and np.array_equal(gs.cpu().numpy()[:side.size], side)
    assert np.array_equal(f32(q_out), R.rope32(f32(q), f32(qw) if norm else None, 1e-6, table, p, dim, layout))

    # read back: scale and zero in fp32 (one rounding of a fused product and sum), then log2(h) sums of
    # the inverse rotation, each at most half a step of a partial sum of at most h max|x| (before / h)
    for lens_dev in (i32(wl.lens), None):
        for dt in ("f32", "bf16"):
            ko, vo = cache.gather(0, i32(b), i32(p), pt, lens_dev, dtype=TYPES[dt])
            for i, L in enumerate(wl.lens):
                rows = b == i
                for g in range(Hkv):
                    kh, vh, region = O.dequant_seq(cfg, pool, side, wl.page_table[i], i, int(L), g)
                    sel = np.ones(int(L), bool) if lens_dev is not None else region == 1
                    H = np.array([O.fwht_f64(np.eye(D)[j], h) for j in range(D)])
                    bits = np.array([((signs or (0,) * 4)[j >> 5] >> (j & 31)) & 1 for j in range(D)])
                    un = lambda x: (x @ H / h) * (1 - 2 * bits)  # noqa: E731
                    for got, ref, rot in ((f32(ko)[rows][:, g], kh, True), (f32(vo)[rows][:, g], vh, rotv)):
                        big = np.abs(ref).max(-1, keepdims=True)
                        ref = un(ref) if rot else ref
                        tol = (np.log2(h) + 1) * 2.0 ** -24 * big + (2.0 ** -8 * np.abs(ref) if dt == "bf16" else 0) + (1e-3 * 2.0 ** -8 * big if dt == "bf16" else 0)
                        assert np.all((np.abs(got - ref) <= tol)[sel])


@pytest.mark.parametrize("D,kb,vb,P,dim,layout", [(128, 3, 3, 16, 128, 0), (64, 1, 2, 16, 64, 1), (128, 8, 8, 48, 64, 0), (64, 5, 4, 32, 16, 0), (128, 7, 3, 64, 128, 1)])
def test_append_mixed_exact(kv4, D, kb, vb, P, dim, layout):
    lens, Hkv = (33, 1, 120, 0, 64), 2
    wl = W.make_workload("mixed", 19, 1, len(lens), 2 * Hkv, Hkv, D, P, 0, 0, 1, lambda r: list(lens), W.F32, W.F32, W.F32, 2, 4.0)
    cache = kv4.Cache(kv4.Geometry(1, wl.Hq, Hkv, D, P, 0, 0, 1, wl.B, wl.num_pages, kv4.KV4_KEYS_MIXED, kb, vb), fill=0xA5)
    kw = rand((D,), "bf16", 2)
    rope = kv4.Rope(kv4.RopeGeometry(dim, 200, layout), None, kw)
    b, p, K = tokens(wl, "bf16", 5, Hkv)
    V = tokens(wl, "bf16", 6, Hkv)[2]
    # the allocation is scored on rotated keys
    _, Kr = rope.apply(None, K, i32(p), k_out=torch.zeros(K.shape, device="cuda"))
    ref = R.rope32(f32(K), f32(kw), 1e-6, rope.table.cpu().numpy(), p, dim, layout)
    assert np.array_equal(f32(Kr), ref)
    cache.allocate_key_bits(0, Kr)
    widths, sigma = cache.key_allocation(0)
    pt = torch.from_numpy(wl.page_table).cuda()
    cache.append_rope(0, rope, None, K, V, i32(b), i32(p), None, pt)
    cfg = O.GtqConfig(wl.Hq, Hkv, D, P, kb, vb)
    pool = np.full(O.gtq_sizes(cfg)["page_bytes"] * wl.num_pages, 0xA5, np.uint8)
    O.gtq_append(cfg, widths, sigma, pool, ref, f32(V), b, p, wl.page_table)
    assert np.array_equal(cache.layer_views(0)[0].cpu().numpy(), pool)
    ko, vo = cache.gather(0, i32(b), i32(p), pt, i32(wl.lens), dtype=torch.float32)
    for i, L in enumerate(lens):
        for g in range(Hkv):
            kh, vh = O.gtq_dequant_seq(cfg, widths, sigma, pool, wl.page_table[i], L, g)
            # a key is two products; a value's step is rounded once (relative to step times code, at
            # most the range), and the fused product and sum once
            assert np.all(np.abs(f32(ko)[b == i][:, g] - kh) <= 3 * 2.0 ** -24 * np.abs(kh))
            span = np.ptp(vh, axis=-1, keepdims=True) if L else 0
            assert np.all(np.abs(f32(vo)[b == i][:, g] - vh) <= 2.0 ** -24 * (np.abs(vh) + 1.01 * span + 1e-30))


def test_bf16_pool(kv4):
    lens, Hkv, D = (40, 1, 17), 2, 128
    wl = W.make_workload("bf16", 23, 1, 3, 4 * Hkv, Hkv, D, 32, 0, 0, 1, lambda r: list(lens), W.F32, W.F32, W.F32, 2, 4.0)
    geo = T.geometry(wl)
    a, c = kv4.BF16Cache(geo), kv4.BF16Cache(geo)
    for x in (a, c):
        x.pool.fill_(0xA5)
    rope = kv4.Rope(kv4.RopeGeometry(D, 64, 1), rand((D,), "f32", 1), rand((D,), "f32", 2))
    b, p, K = tokens(wl, "bf16", 5, Hkv)
    V = tokens(wl, "bf16", 6, Hkv)[2]
    q = tokens(wl, "bf16", 7, wl.Hq)[2]
    pt = torch.from_numpy(wl.page_table).cuda()
    qo = a.append_rope(0, rope, q, K, V, i32(b), i32(p), None, pt)
    q2, Kr = rope.apply(q, K, i32(p), k_out=torch.empty(K.shape, device="cuda"))
    c.append(0, Kr, V, i32(b), i32(p), pt)
    assert torch.equal(a.pool, c.pool) and torch.equal(qo, q2)
    ko, vo = a.gather(0, i32(b), i32(p), pt)
    assert torch.equal(ko, Kr.to(torch.bfloat16)) and torch.equal(vo, V)


def _small(kv4, max_pos=512, lens=(40, 21), P=16):
    wl = W.make_workload("small", 29, 1, len(lens), 8, 2, 128, P, 4, 16, 128, lambda r: list(lens), W.F32, W.F32, W.F32, 2, 4.0)
    cache = kv4.Cache(T.geometry(wl), fill=0xA5)
    rope = kv4.Rope(kv4.RopeGeometry(128, max_pos), rand((128,), "f32", 1), rand((128,), "f32", 2))
    return wl, cache, rope, torch.from_numpy(wl.page_table).cuda()


def test_padding_rows_are_left_alone(kv4):
    wl, cache, rope, pt = _small(kv4)
    b, p, K = tokens(wl, "bf16", 5, 2)
    V, q = tokens(wl, "bf16", 6, 2)[2], tokens(wl, "bf16", 7, 8)[2]
    pad = np.arange(b.size) % 3 == 1
    before = [x.clone() for x in cache.layer_views(0)]
    q_out = torch.full(q.shape, 5.0, device="cuda")
    cache.append_rope(0, rope, q, K, V, i32(np.full_like(b, -1)), i32(p), i32(wl.lens), pt, q_out=q_out)
    assert all(torch.equal(x, y) for x, y in zip(before, cache.layer_views(0))) and bool((q_out == 5).all())
    cache.append_rope(0, rope, q, K, V, i32(np.where(pad, -1, b)), i32(np.where(pad, -1, p)), i32(wl.lens), pt, q_out=q_out)
    ref, other = _small(kv4)[1], i32(np.nonzero(~pad)[0])
    sel = lambda x: x[other.long()].contiguous()  # noqa: E731
    q_ref = ref.append_rope(0, rope, sel(q), sel(K), sel(V), i32(b[~pad]), i32(p[~pad]), i32(wl.lens), pt)
    assert all(torch.equal(x, y) for x, y in zip(ref.layer_views(0), cache.layer_views(0)))
    assert torch.equal(q_out[other.long()].to(torch.bfloat16), q_ref) and bool((q_out[torch.from_numpy(pad).cuda()] == 5).all())
    out = torch.full((b.size, 2, 128), 6.0, device="cuda")
    cache.gather(0, i32(np.where(pad, -1, b)), i32(p), pt, i32(wl.lens), k_out=out, v_out=out.clone())
    assert bool((out[torch.from_numpy(pad).cuda()] == 6).all()) and not bool((out[other.long()] == 6).any())


def test_bad_rows_set_error_bits(kv4):
    wl, cache, rope, pt = _small(kv4, max_pos=30)
    K = rand((1, 2, 128), "bf16", 5)
    q = rand((1, 8, 128), "bf16", 6)
    before = [x.clone() for x in cache.layer_views(0)]
    bad_page = pt.clone()
    bad_page[0, 0] = wl.num_pages
    for slot, pos, table, bit in ((0, 30, pt, kv4.KV4_DEVERR_LENGTH), (-2, 0, pt, kv4.KV4_DEVERR_LENGTH), (wl.B, 0, pt, kv4.KV4_DEVERR_LENGTH),
                                  (0, -1, pt, kv4.KV4_DEVERR_LENGTH), (0, 16 * wl.stride, pt, kv4.KV4_DEVERR_LENGTH),
                                  (0, 0, bad_page, kv4.KV4_DEVERR_PAGE_RANGE)):
        q_out = torch.full(q.shape, 5.0, device="cuda")
        cache.append_rope(0, rope, q, K, K, i32([slot]), i32([pos]), i32(wl.lens), table, q_out=q_out)
        assert kv4.kv4_get_device_error() == bit and bool((q_out == 5).all())
    for slot, pos, table, bit in ((0, int(wl.lens[0]), pt, kv4.KV4_DEVERR_LENGTH), (wl.B, 0, pt, kv4.KV4_DEVERR_LENGTH), (0, 0, bad_page, kv4.KV4_DEVERR_PAGE_RANGE)):
        out = torch.full((1, 2, 128), 6.0, device="cuda")
        cache.gather(0, i32([slot]), i32([pos]), table, i32(wl.lens), k_out=out, v_out=out.clone())
        assert kv4.kv4_get_device_error() == bit and bool((out == 6).all())
    assert all(torch.equal(x, y) for x, y in zip(before, cache.layer_views(0)))


def test_range_overflow_is_reported(kv4):
    wl, cache, rope, pt = _small(kv4)
    K = rand((1, 2, 128), "f32", 5)
    V = K * 1e6
    cache.append_rope(0, rope, None, K, V, i32([0]), i32([0]), i32(wl.lens), pt)
    assert kv4.kv4_get_device_error() == kv4.KV4_DEVERR_RANGE


def test_steps_match_prefill_and_decode(kv4):
    """A serving run: prefill through append_rope in two unequal chunks, then single tokens; the cache
    equals one built by the oracle from the rotated keys, and the decode its attention."""
    wl, cache, rope, pt = _small(kv4, lens=(75, 40, 17, 50))
    b, p, K = tokens(wl, "bf16", 5, 2)
    V, q = tokens(wl, "bf16", 6, 2)[2], tokens(wl, "bf16", 7, 8)[2]
    lens = np.asarray(wl.lens)
    cfg = O.Config(wl.Hq, wl.Hkv, wl.D, wl.P, wl.s, wl.w, wl.h, wl.B)
    pool = np.full(O.page_bytes(cfg) * wl.num_pages, 0xA5, np.uint8)
    side = np.full(O.side_slot_bytes(cfg) * wl.B, 0xA5, np.uint8)
    Kr = R.rope32(f32(K), f32(rope.k_weight), 1e-6, rope.table.cpu().numpy(), p, 128, 0)
    steps = [(0, lens // 3), (lens // 3, lens - 3), (lens - 3, lens - 2), (lens - 2, lens - 1), (lens - 1, lens)]
    q_last = torch.empty((wl.B, 8, 128), dtype=torch.bfloat16, device="cuda")
    for lo, hi in steps:
        sel = np.nonzero((p >= np.broadcast_to(lo, lens.shape)[b]) & (p < hi[b]))[0]
        at = torch.from_numpy(sel).cuda()
        qo = cache.append_rope(0, rope, q[at], K[at], V[at], i32(b[sel]), i32(p[sel]), i32(hi), pt)
        O.append(cfg, pool, side, Kr[sel], f32(V)[sel], b[sel], p[sel], hi.astype(np.int32), wl.page_table, O.F32, O.F32)
        q_last = qo
    gp, gs = cache.layer_views(0)
    assert np.array_equal(gp.cpu().numpy(), pool) and np.array_equal(gs.cpu().numpy(), side)
    out, lse = T.gpu_decode(cache, wl, q_last.view(torch.int16).cpu().numpy().view(np.uint16))
    ref, ref_lse = T.oracle_decode(wl, cfg, pool, side, q_last.view(torch.int16).cpu().numpy().view(np.uint16))
    T.assert_close(out, ref, lse, ref_lse, what="append_rope then decode")


def test_captured_and_on_another_stream(kv4):
    wl, cache, rope, pt = _small(kv4)
    b, p, K = tokens(wl, "bf16", 5, 2)
    V, q = tokens(wl, "bf16", 6, 2)[2], tokens(wl, "bf16", 7, 8)[2]
    bd, pd, ld = i32(b), i32(p), i32(wl.lens)
    ref = cache.append_rope(0, rope, q, K, V, bd, pd, ld, pt)
    rk, rv = cache.gather(0, bd, pd, pt, ld)
    want = [x.clone() for x in cache.layer_views(0)]
    q_out, ko, vo = torch.zeros_like(ref), torch.zeros_like(rk), torch.zeros_like(rv)
    for x in cache.layer_views(0):
        x.fill_(0xA5)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        cache.append_rope(0, rope, q, K, V, bd, pd, ld, pt, q_out=q_out)
        cache.gather(0, bd, pd, pt, ld, k_out=ko, v_out=vo)
    for _ in range(2):
        q_out.zero_(), ko.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(q_out, ref) and torch.equal(ko, rk) and torch.equal(vo, rv)
        assert all(torch.equal(x, y) for x, y in zip(want, cache.layer_views(0)))


def test_far_offsets(kv4):
    """Tokens and token strides whose element offsets pass 32 bits."""
    n, D, stride = 5, 64, 1 << 29
    big = torch.empty((n - 1) * stride + 4 * D, dtype=torch.bfloat16, device="cuda")
    q = torch.as_strided(big, (n, 4, D), (stride, D, 1))
    src = rand((n, 4, D), "bf16", 5)
    q.copy_(src)
    rope = kv4.Rope(kv4.RopeGeometry(D, 64))
    pos = i32(np.arange(n))
    assert torch.equal(rope.apply(q, None, pos)[0], rope.apply(src, None, pos)[0])


def test_python_checks(kv4):
    rope = kv4.Rope(kv4.RopeGeometry(64, 16), rand((64,), "f32", 1))
    q = rand((2, 2, 128), "f32", 5)
    with pytest.raises(ValueError):
        rope.apply(q, None, i32([0, 1]))  # weights of 64, heads of 128
    q = rand((2, 2, 64), "f32", 5)
    with pytest.raises(ValueError):
        rope.apply(q, None, torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        rope.apply(q.transpose(0, 1), None, i32([0, 1]))
    with pytest.raises(ValueError):
        rope.apply(q, None, i32([0]))
    with pytest.raises(ValueError):
        rope.apply(q.double(), None, i32([0, 1]))
    with pytest.raises(ValueError):
        kv4.Rope(kv4.RopeGeometry(64, 16), torch.ones(64))  # weights on the host


def test_gather_of_repeated_and_no_positions(kv4):
    wl = W.make_workload("twice", 3, 1, 2, 8, 2, 128, 16, 4, 16, 128, lambda _: [40, 21], W.F32, W.F32, W.F32, 2, 6.0)
    cache = T.gpu_cache_from_host_inputs(wl)
    pt, lens = torch.from_numpy(wl.page_table).cuda(), torch.from_numpy(wl.lens).cuda()
    b, p = T.prefill_tokens(wl.lens)
    k, v = cache.gather(0, i32(b), i32(p), pt, lens)
    pick = np.array([0, 60, 0, 0, 39, 60])
    k2, v2 = cache.gather(0, i32(b[pick]), i32(p[pick]), pt, lens)
    assert torch.equal(k2, k[pick]) and torch.equal(v2, v[pick])
    k0, v0 = cache.gather(0, i32([]), i32([]), pt, lens)
    assert k0.shape == v0.shape == (0, 2, 128)
