"""Norm, rotation and fused append of many tokens, where the kernels take runs of heads a warp and a key
together with its value.  Exact against NumPy and the CPU oracle, as in test_gpu_rope.py."""
import numpy as np
import pytest
import torch

from int4_kv_cache_append_b200 import workload as W
from oracle import oracle as O

import kv4_testlib as T
import rope_ref as R
from test_gpu_rope import f32, i32, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv4():
    from int4_kv_cache_append_b200 import kv4
    return kv4


@pytest.fixture(autouse=True)
def no_device_error(kv4):
    yield
    assert kv4.kv4_get_device_error() == 0


def many(D):
    """More vectors than this take the many-token form: 64 warps an SM, each with 256 / D vectors."""
    return torch.cuda.get_device_properties(0).multi_processor_count * 64 * (256 // D)


# (T, Hq, Hkv, D, R, layout, norm): head counts that are no multiple of a warp's passes
ROPE = [
    (4001, 5, 1, 128, 128, 0, True), (2001, 9, 3, 128, 64, 1, False), (2000, 20, 1, 128, 120, 0, True), (1700, 33, 3, 128, 128, 1, True),
    (8001, 5, 1, 64, 64, 0, True), (3401, 9, 3, 64, 24, 0, True), (2001, 20, 1, 64, 64, 1, False), (1100, 35, 3, 64, 8, 0, True),
    (20001, 0, 1, 128, 128, 0, True), (19001, 1, 0, 128, 128, 1, False),
]


@pytest.mark.parametrize("case", ROPE, ids=[str(c) for c in ROPE])
@pytest.mark.parametrize("dt,odt,in_place", [("bf16", "bf16", False), ("f16", "f16", True), ("bf16", "f16", False), ("f32", "bf16", False)])
def test_rope_matches(kv4, case, dt, odt, in_place):
    n, Hq, Hkv, D, dim, layout, norm = case
    assert n * (Hq + Hkv) > many(D)
    rope = kv4.Rope(kv4.RopeGeometry(dim, 5000, layout, 10000.0), *((rand((D,), "bf16", s) if norm else None) for s in (1, 2)))
    fused = rand((n, (Hq + 2 * Hkv) * D), dt, 3, 2.0)
    keep = fused.clone()
    at = lambda t, lo, H: t[:, lo * D:(lo + H) * D].view(n, H, D) if H else None  # noqa: E731
    q, k = at(fused, 0, Hq), at(fused, Hq, Hkv)
    pos = np.random.default_rng(4).integers(0, 5000, n)
    pos[::97] = -1
    outs = [q, k] if in_place else [None if x is None else torch.full(x.shape, 9.0, dtype=T_[odt], device="cuda") for x in (q, k)]
    rope.apply(q, k, i32(pos), *outs)
    table, live = rope.table.cpu().numpy(), pos >= 0
    for x, w, o in ((at(keep, 0, Hq), rope.q_weight, outs[0]), (at(keep, Hq, Hkv), rope.k_weight, outs[1])):
        if x is None:
            continue
        ref = R.rope32(f32(x), f32(w) if norm else None, 1e-6, table, pos, dim, layout)
        assert np.array_equal(f32(o)[live], f32(torch.from_numpy(ref).to(T_[odt]))[live])
        assert np.array_equal(f32(o)[~live], f32(x)[~live] if in_place else np.full_like(ref[~live], 9.0))
    assert torch.equal(fused[:, (Hq + Hkv) * D:], keep[:, (Hq + Hkv) * D:])


T_ = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# (name, D, G, Hkv, P, s, w, h, lens, rotary dim, layout, k type, v type, value_format)
APPEND = [
    ("int4-d128", 128, 4, 3, 16, 4, 128, 128, (1500, 400, 37, 400), 128, 0, "bf16", "bf16", 0),
    ("int4-d64", 64, 2, 5, 48, 2, 24, 64, (2000, 17, 600), 24, 1, "f32", "f16", 0),
    ("int4-no-side", 128, 1, 1, 64, 0, 0, 1, (8000, 1000), 64, 0, "f16", "bf16", 0),
    ("vbf-d128", 128, 4, 3, 16, 4, 16, 128, (1500, 800), 128, 0, "bf16", "bf16", 1),
    ("vbf-d64", 64, 4, 1, 16, 19, 13, 16, (6000, 700), 64, 1, "f32", "f32", 1),
]


def inputs(wl, kdt, vdt):
    b, p = T.prefill_tokens(wl.lens)
    mk = lambda dt, seed, H: rand((b.size, H, wl.D), dt, seed)  # noqa: E731
    return b, p, mk("bf16", 7, wl.Hq), mk(kdt, 5, wl.Hkv), mk(vdt, 6, wl.Hkv)


@pytest.mark.parametrize("case", APPEND, ids=[c[0] for c in APPEND])
def test_append_bytes_exact(kv4, case):
    name, D, G, Hkv, P, s, w, h, lens, dim, layout, kdt, vdt, vf = case
    wl = W.make_workload(name, 17, 1, len(lens), G * Hkv, Hkv, D, P, s, w, h, lambda r: list(lens), W.F32, W.F32, W.F32, 2, 20.0)
    b, p, q, K, V = inputs(wl, kdt, vdt)
    assert b.size * (G + 2) * Hkv > many(D)
    cache = kv4.Cache(T.geometry(wl, value_format=vf), fill=0xA5)
    rope = kv4.Rope(kv4.RopeGeometry(dim, 8192, layout), rand((D,), "f32", 1), rand((D,), "f32", 2))
    pt = torch.from_numpy(wl.page_table).cuda()
    for q_out in (torch.zeros(q.shape, device="cuda"), torch.zeros_like(q)):
        cache.append_rope(0, rope, q, K, V, i32(b), i32(p), i32(wl.lens), pt, q_out=q_out)
        table = rope.table.cpu().numpy()
        ref = R.rope32(f32(q), f32(rope.q_weight), 1e-6, table, p, dim, layout)
        assert np.array_equal(f32(q_out), f32(torch.from_numpy(ref).to(q_out.dtype)))
    cfg = O.Config(wl.Hq, Hkv, D, P, s, w, h, wl.B, (0, 0, 0, 0), 0, vf)
    pool = np.full(O.page_bytes(cfg) * wl.num_pages, 0xA5, np.uint8)
    side = np.full(max(O.side_slot_bytes(cfg) * wl.B, 1), 0xA5, np.uint8)
    O.append(cfg, pool, side, R.rope32(f32(K), f32(rope.k_weight), 1e-6, table, p, dim, layout), f32(V), b, p, wl.lens, wl.page_table, O.F32, O.F32)
    gp, gs = cache.layer_views(0)
    n = min(side.size, gs.numel())
    assert np.array_equal(gp.cpu().numpy(), pool) and np.array_equal(gs.cpu().numpy()[:n], side[:n])


@pytest.mark.parametrize("D,G,Hkv,lens", [(128, 4, 3, (1500, 700)), (64, 2, 5, (1900, 300))])
def test_append_mixed_exact(kv4, D, G, Hkv, lens):
    wl = W.make_workload("mixed", 19, 1, len(lens), G * Hkv, Hkv, D, 16, 0, 0, 1, lambda r: list(lens), W.F32, W.F32, W.F32, 2, 4.0)
    b, p, q, K, V = inputs(wl, "bf16", "bf16")
    assert b.size * (G + 2) * Hkv > many(D)
    cache = kv4.Cache(kv4.Geometry(1, wl.Hq, Hkv, D, 16, 0, 0, 1, wl.B, wl.num_pages, kv4.KV4_KEYS_MIXED, 3, 3), fill=0xA5)
    rope = kv4.Rope(kv4.RopeGeometry(D, 2048), rand((D,), "bf16", 1), rand((D,), "bf16", 2))
    cache.allocate_key_bits(0, K[:256].contiguous())
    widths, sigma = cache.key_allocation(0)
    q_out = cache.append_rope(0, rope, q, K, V, i32(b), i32(p), None, torch.from_numpy(wl.page_table).cuda())
    table = rope.table.cpu().numpy()
    ref = R.rope32(f32(q), f32(rope.q_weight), 1e-6, table, p, D, 0)
    assert np.array_equal(f32(q_out), f32(torch.from_numpy(ref).to(torch.bfloat16)))
    cfg = O.GtqConfig(wl.Hq, Hkv, D, 16, 3, 3)
    pool = np.full(O.gtq_sizes(cfg)["page_bytes"] * wl.num_pages, 0xA5, np.uint8)
    O.gtq_append(cfg, widths, sigma, pool, R.rope32(f32(K), f32(rope.k_weight), 1e-6, table, p, D, 0), f32(V), b, p, wl.page_table)
    assert np.array_equal(cache.layer_views(0)[0].cpu().numpy(), pool)


def test_append_bf16_pool(kv4):
    wl = W.make_workload("bf16", 23, 1, 2, 12, 3, 128, 32, 0, 0, 1, lambda r: [1500, 700], W.F32, W.F32, W.F32, 2, 4.0)
    b, p, q, K, V = inputs(wl, "bf16", "bf16")
    assert b.size * 18 > many(128)
    a, c = kv4.BF16Cache(T.geometry(wl)), kv4.BF16Cache(T.geometry(wl))
    for x in (a, c):
        x.pool.fill_(0xA5)
    rope = kv4.Rope(kv4.RopeGeometry(128, 2048, 1), rand((128,), "f32", 1), rand((128,), "f32", 2))
    pt = torch.from_numpy(wl.page_table).cuda()
    q_out = a.append_rope(0, rope, q, K, V, i32(b), i32(p), None, pt)
    table = rope.table.cpu().numpy()
    ref = [R.rope32(f32(x), f32(w), 1e-6, table, p, 128, 1) for x, w in ((q, rope.q_weight), (K, rope.k_weight))]
    assert np.array_equal(f32(q_out), f32(torch.from_numpy(ref[0]).to(torch.bfloat16)))
    c.append(0, torch.from_numpy(ref[1]).cuda(), V, i32(b), i32(p), pt)
    assert torch.equal(a.pool, c.pool)
