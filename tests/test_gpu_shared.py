"""kv4_decode_attn_shared against the oracle's fp64 attention on the same cache bytes.

The oracle knows nothing of groups: it attends each sequence's own page-table row.  Tolerance, per
query head and output element.  Inside the prefix the query is rounded to fp16, q_i (1 + e_i) with
|e_i| <= 2^-11, the same e for every position, so to first order the output moves by sum_i e_i q_i
Cov_p(k_i, v) / sqrt(D) and the log-sum by sum_i e_i q_i mean_p(k_i) / sqrt(D), at most 2^-11 times
the sums of magnitudes; with d a bound of a logit's error the second order is below 2 d^2 times the
mean distance of v from the output.  A probability and a value are rounded to fp16 (each at most
2^-11 of p |v|, or 2^-25 absolute for a probability below fp16's normal range).  The fp32 and
integer steps are held to 2e-4 of the outputs' scale and 1e-4 of the log-sum."""
import ctypes

import numpy as np
import pytest
import torch

from int4_kv_cache_append_b200 import workload as W
from oracle import oracle as O

import kv4_testlib as T

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv4():
    from int4_kv_cache_append_b200 import kv4
    return kv4


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


# (name, D, G, Hkv, P, s, w, h, group sizes, prefix lengths, lengths past the prefix, copies, q type, options)
# A length past the prefix may be negative: that sequence ends inside the prefix.
CASES = [
    ("one-group", 128, 4, 2, 16, 4, 16, 128, [3], [200], [40, 1, 77], False, W.BF16, {}),
    ("ragged", 128, 4, 2, 16, 4, 16, 128, [1, 5, 2], [64, 333, 17], [10, 0, 3, 100, 20, 31, 5, 300], False, W.BF16, {}),
    ("d64-g1-h1", 64, 1, 2, 16, 2, 8, 1, [4, 3], [100, 48], [5, 6, 7, 8, 9, 10, 1], False, W.F32, {}),
    ("d64-g2-p48", 64, 2, 3, 48, 0, 24, 16, [7], [500], list(range(1, 8)), False, W.BF16, {}),
    ("no-side", 128, 2, 2, 32, 0, 0, 64, [2, 2], [128, 70], [0, 1, 16, 26], False, W.BF16, {}),
    ("sinks-only", 128, 4, 1, 16, 19, 0, 16, [3, 1], [90, 18], [4, 4, 4, 200], False, W.F32, {}),
    ("recent-reaches-in", 128, 4, 2, 16, 4, 128, 128, [4], [300], [1, 60, 127, 200], False, W.BF16, {}),
    ("shorter-than-prefix", 128, 4, 2, 16, 4, 16, 128, [5], [400], [50, -100, -383, -400, -399], False, W.BF16, {}),
    ("copies", 128, 4, 2, 16, 4, 16, 128, [3, 2], [160, 96], [40, 1, 77, 20, 20], True, W.BF16, {}),
    ("many-rows", 128, 4, 1, 64, 16, 32, 128, [40], [600], list(np.arange(40) * 5 + 1), False, W.BF16, {}),
    ("many-rows-d64", 64, 4, 1, 16, 4, 16, 64, [33, 1], [260, 20], list(np.arange(34) + 1), False, W.BF16, {}),
    ("tiny-prefixes", 128, 4, 2, 16, 4, 16, 128, [2, 2, 2, 2], [0, 3, 15, 16], [30, 40, 50, 60, 1, 2, 3, 4], False, W.BF16, {}),
    ("outside-rows", 128, 4, 2, 16, 4, 16, 128, [2, 0, 3], [100, 50, 64], [5, 6, 7, 8, 9], False, W.BF16, dict(before=2, after=3)),
    ("long-side", 128, 2, 2, 16, 5, 300, 128, [3], [700], [10, 200, 400], False, W.BF16, {}),
    ("signs-rotv", 128, 4, 2, 16, 4, 16, 128, [3], [150], [10, 20, 30], False, W.BF16,
     dict(signs=(0x9E3779B9, 0x12345678, 0xDEADBEEF, 0x0F0F0F0F), rotv=True)),
    ("rotv-d64", 64, 4, 2, 16, 4, 16, 32, [3], [150], [10, 20, 30], False, W.F32, dict(rotv=True)),
    ("b300", 64, 2, 1, 16, 4, 16, 64, [100, 60, 140], [96, 33, 64], list(np.random.default_rng(3).integers(0, 40, 300)), False, W.BF16, {}),
    ("long", 128, 4, 2, 16, 4, 128, 128, [6, 2], [3001, 5000], [100, 1, 700, 12, 13, 14, 15, 900], False, W.BF16, {}),
]
IDS = [c[0] for c in CASES]


class Built:
    pass


def build(case, kv4=None, fill=0xA5):
    """The workload, the oracle's cache and (with kv4) the GPU's, of one case."""
    name, D, G, Hkv, P, s, w, h, sizes, prefix, past, copies, qt, opt = case
    before, after = opt.get("before", 0), opt.get("after", 0)
    group = np.repeat(np.arange(len(sizes)), sizes)
    lens = [60 + i for i in range(before)] + [max(0, prefix[g] + d) for g, d in zip(group, past)] + [41 + i for i in range(after)]
    r = Built()
    r.wl = wl = W.make_workload(name, 31, 1, len(lens), G * Hkv, Hkv, D, P, s, w, h, lambda _: [max(x, 1) for x in lens], W.F32, W.F32, qt, 2, 6.0)
    wl.lens = np.asarray(lens, np.int32)
    r.start = before + np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    r.prefix = np.asarray(prefix, np.int32)
    # the group's first row has pages for the whole prefix, whatever its own length
    src = np.arange(wl.B)
    extra = []
    for g, n in enumerate(sizes):
        if not n:
            continue
        b0 = r.start[g]
        src[b0:b0 + n] = b0
        need = -(-max(prefix[g], 1) // P)
        have = -(-max(lens[b0], 1) // P)
        if need > wl.page_table.shape[1]:
            wl.page_table = np.pad(wl.page_table, ((0, 0), (0, need - wl.page_table.shape[1])))
        if need > have:
            wl.page_table[b0, have:need] = wl.num_pages + np.arange(need - have)
            wl.num_pages += need - have
        longest = b0 + int(np.argmax(lens[b0:b0 + n]))
        for b in range(b0, b0 + n):
            k = min(prefix[g] // P, -(-lens[b] // P))
            if not copies:
                wl.page_table[b, :k] = wl.page_table[b0, :k]
        if lens[longest] > lens[b0]:  # the prefix pages past the first row's own length are filled by a longer one
            extra.append((longest, b0, lens[b0], min(prefix[g], lens[longest])))
    b, p = T.prefill_tokens(wl.lens)
    shared = p < np.concatenate([np.zeros(before, int), r.prefix[group], np.zeros(after, int)])[b]
    K, V = wl.kv_inputs(0, np.where(shared, src[b], b), p)
    r.cfg = O.Config(wl.Hq, Hkv, D, P, s, w, h, wl.B, opt.get("signs", (0, 0, 0, 0)), int(opt.get("rotv", False)), 0)
    r.pool = np.full(O.page_bytes(r.cfg) * wl.num_pages, fill, np.uint8)
    r.side = np.full(max(O.side_slot_bytes(r.cfg) * wl.B, 1), fill, np.uint8)
    O.append(r.cfg, r.pool, r.side, K, V, b, p, wl.lens, wl.page_table)
    for _, b0, lo, hi in extra:
        q = np.arange(lo, hi, dtype=np.int32)
        Kx, Vx = wl.kv_inputs(0, np.full(q.size, b0), q)
        keep = r.side.copy()
        O.append(r.cfg, r.pool, r.side, Kx, Vx, np.full(q.size, b0, np.int32), q, wl.lens, wl.page_table)
        r.side[:] = keep
    if kv4 is not None:
        r.cache = kv4.Cache(T.geometry(wl))
        if opt.get("signs"):
            kv4.kv4_set_rotation_signs(r.cache.handle, opt["signs"])
        if opt.get("rotv"):
            kv4.kv4_set_value_rotation(r.cache.handle, True)
        gp, gs = r.cache.layer_views(0)
        gp.copy_(torch.from_numpy(r.pool))
        if gs.numel():
            gs.copy_(torch.from_numpy(r.side[:gs.numel()]))
        r.pt, r.lens = torch.from_numpy(wl.page_table).cuda(), torch.from_numpy(wl.lens).cuda()
        r.start_d, r.prefix_d = i32(r.start), i32(r.prefix)
        r.q = T.to_dev(wl.q_input(0))
    return r


def reference(r):
    """(out, lse, bound of out [B][Hq][D], bound of lse [B][Hq]) of the workload's queries."""
    wl, cfg = r.wl, r.cfg
    q = wl.q_input(0)
    ref, lse = T.oracle_decode(wl, cfg, r.pool, r.side, q)
    q64 = (W.bf16_to_f32(q) if q.dtype == np.uint16 else q).astype(np.float64)
    G, D, h = wl.Hq // wl.Hkv, wl.D, wl.h
    sg = np.array([1 - 2 * ((cfg.sign_bits[i >> 5] >> (i & 31)) & 1) for i in range(D)])
    bo, bl = np.zeros((wl.B, wl.Hq, D)), np.zeros((wl.B, wl.Hq))
    u = 1.05 * 2.0 ** -11
    for b, L in enumerate(wl.lens):
        for g in range(wl.Hkv if L else 0):
            k, v, _ = O.dequant_seq(cfg, r.pool, r.side, wl.page_table[b], b, int(L), g)
            for j in range(g * G, g * G + G):
                qr = np.abs(O.fwht_f64(q64[b, j] * sg, h) / h) / np.sqrt(D)
                x = k @ (O.fwht_f64(q64[b, j] * sg, h) / h) / np.sqrt(D)
                p = np.exp(x - x.max())
                total = p.sum()
                p /= total
                o, km, d = p @ v, p @ k, u * (np.abs(k) @ qr).max()
                cov = (k - km).T @ ((v - o) * p[:, None])
                e = u * (qr @ np.abs(cov) + 2 * (p @ np.abs(v))) + 2 * d * d * (p @ np.abs(v - o)) + 2.0 ** -25 * np.abs(v).sum(0) / total
                if cfg.rotate_values:  # rotated back: signed sums of a block's errors over h
                    e = np.repeat(e.reshape(-1, h).mean(1), h)
                bo[b, j] = e + 2e-4 * max(1.0, np.abs(ref[b, j]).max())
                bl[b, j] = u * (qr @ np.abs(km)) + d * d + 1e-4
    return ref, lse, bo, bl


def check(r, out, lse, want, half_step=0.0):
    ref, ref_lse, bo, bl = want
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - ref)
    tol = bo + half_step * np.abs(ref)
    assert np.all(err <= tol), f"worst {np.max(err / tol):.2f} of the bound at {np.unravel_index(np.argmax(err / tol), err.shape)}"
    if lse is not None:
        got = lse.cpu().numpy().astype(np.float64)
        live = np.isfinite(ref_lse)
        assert np.array_equal(live, np.isfinite(got)) and np.all(got[~live] == -np.inf)
        assert np.all(np.abs(got - ref_lse)[live] <= bl[live])


@gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_matches_oracle(kv4, case):
    r = build(case, kv4)
    want = reference(r)
    lse = torch.full((r.wl.B, r.wl.Hq), float("nan"), device="cuda")
    out = torch.full((r.wl.B, r.wl.Hq, r.wl.D), float("nan"), device="cuda")
    r.cache.decode_shared(0, r.q, r.pt, r.lens, r.start_d, r.prefix_d, out=out, lse=lse)
    check(r, out, lse, want)
    # a second call on the used workspace, with a hint, in 16 bits
    for dt, half in ((torch.bfloat16, 2.0 ** -8), (torch.float16, 2.0 ** -11)):
        o2 = r.cache.decode_shared(0, r.q, r.pt, r.lens, r.start_d, r.prefix_d, out=torch.empty(out.shape, dtype=dt, device="cuda"),
                                   max_len_hint=int(r.wl.lens.max()) or 1)
        check(r, o2, None, want, half)
    assert kv4.kv4_get_device_error() == 0


@gpu
def test_no_groups_is_plain_decode(kv4):
    r = build(CASES[1], kv4)
    ref_lse, lse = (torch.empty((r.wl.B, r.wl.Hq), device="cuda") for _ in range(2))
    ref = r.cache.decode(0, r.q, r.pt, r.lens, lse=ref_lse)
    out = r.cache.decode_shared(0, r.q, r.pt, r.lens, i32([0]), i32([]), out=torch.empty_like(ref), lse=lse)
    T.assert_close(out.cpu().numpy(), ref.cpu().numpy().astype(np.float64), lse.cpu().numpy(), ref_lse.cpu().numpy(), what="no groups")


@gpu
@pytest.mark.parametrize("start", [[0, 5, 3, 8], [-1, 3, 5, 8], [0, 3, 5, 9], [5, 4, 3, 2]])
def test_bad_groups_share_nothing(kv4, start):
    """Groups that are not consecutive rows set the error bit; the outputs are those of the plain decode."""
    r = build(CASES[1], kv4)
    ref = r.cache.decode(0, r.q, r.pt, r.lens)
    out = r.cache.decode_shared(0, r.q, r.pt, r.lens, i32(start), r.prefix_d, out=torch.empty_like(ref))
    assert kv4.kv4_get_device_error() == kv4.KV4_DEVERR_GROUP
    T.assert_close(out.cpu().numpy(), ref.cpu().numpy().astype(np.float64), what="bad groups")


@gpu
def test_bad_page_sets_error_bit(kv4):
    r = build(CASES[0], kv4)
    bad = r.pt.clone()
    bad[0, 3] = r.wl.num_pages + 7
    r.cache.decode_shared(0, r.q, bad, r.lens, r.start_d, r.prefix_d)
    assert kv4.kv4_get_device_error() & kv4.KV4_DEVERR_PAGE_RANGE
    want = reference(r)
    check(r, r.cache.decode_shared(0, r.q, r.pt, r.lens, r.start_d, r.prefix_d), None, want, 2.0 ** -8)
    assert kv4.kv4_get_device_error() == 0


@gpu
def test_unwritten_pages_do_not_leak(kv4):
    """NaN patterns in every position that no sequence holds (behind the last one, in the unused rows of
    tiles and side caches) change nothing."""
    for name in ("shorter-than-prefix", "ragged", "recent-reaches-in", "no-side", "rotv-d64"):
        a, b = (build(CASES[IDS.index(name)], kv4, fill) for fill in (0xA5, 0xFF))
        x, y = (r.cache.decode_shared(0, r.q, r.pt, r.lens, r.start_d, r.prefix_d) for r in (a, b))
        assert bool(torch.isfinite(x).all()) and torch.equal(x, y)


@gpu
def test_page_ids_do_not_matter(kv4):
    """The same pages under other ids: bit-identical outputs; so are two calls in a row."""
    r = build(CASES[1], kv4)
    a = r.cache.decode_shared(0, r.q, r.pt, r.lens, r.start_d, r.prefix_d, out=torch.empty(r.q.shape, device="cuda"))
    perm = np.random.default_rng(5).permutation(r.wl.num_pages)
    pb = O.page_bytes(r.cfg)
    pool = np.empty_like(r.pool).reshape(-1, pb)
    pool[perm] = r.pool.reshape(-1, pb)
    r.cache.layer_views(0)[0].copy_(torch.from_numpy(pool.reshape(-1)))
    pt = torch.from_numpy(perm[r.wl.page_table].astype(np.int32)).cuda()
    b = r.cache.decode_shared(0, r.q, pt, r.lens, r.start_d, r.prefix_d, out=torch.empty(r.q.shape, device="cuda"))
    assert torch.equal(a, b)


@gpu
def test_captured_replayed_and_two_streams(kv4):
    r, r2 = build(CASES[1], kv4), build(CASES[3], kv4)
    want = [x.cache.decode_shared(0, x.q, x.pt, x.lens, x.start_d, x.prefix_d).clone() for x in (r, r2)]
    outs = [torch.zeros_like(x) for x in want]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        r.cache.decode_shared(0, r.q, r.pt, r.lens, r.start_d, r.prefix_d, out=outs[0])
        r.cache.decode_shared(0, r.q, r.pt, r.lens, r.start_d, r.prefix_d, out=outs[0])
    for _ in range(3):
        outs[0].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            r2.cache.decode_shared(0, r2.q, r2.pt, r2.lens, r2.start_d, r2.prefix_d, out=outs[1])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


@gpu
def test_two_calls_at_once_with_their_own_workspaces(kv4):
    r = build(CASES[IDS.index("long")], kv4)
    want = r.cache.decode_shared(0, r.q, r.pt, r.lens, r.start_d, r.prefix_d)
    n = kv4.kv4_decode_shared_workspace_bytes(r.cache.handle, r.wl.B, len(r.prefix))
    torch.cuda.synchronize()
    runs = []
    for _ in range(2):
        st, ws, out = torch.cuda.Stream(), torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), torch.empty_like(want)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for _ in range(4):
                r.cache.decode_shared(0, r.q, r.pt, r.lens, r.start_d, r.prefix_d, out=out, workspace=ws)
        runs.append(out)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in runs)


@gpu
def test_large_query_magnitudes(kv4):
    """Queries far from one: normalised by a power of two before they are rounded."""
    r = build(CASES[2], kv4)
    for f in (2.0 ** 40, 2.0 ** -40, 0.0):
        q = r.q * f
        ref = r.cache.decode(0, q, r.pt, r.lens)
        out = r.cache.decode_shared(0, q, r.pt, r.lens, r.start_d, r.prefix_d, out=torch.empty_like(ref))
        assert bool(torch.isfinite(out).all())
        if f < 1:  # all logits (nearly) equal: the mean of the values; P and V are off by 2^-11 each
            tol = 2.0 ** -10 * 1.05 * 8 + 2e-4
            assert float((out - ref).abs().max()) <= tol * max(1.0, float(ref.abs().max()))


def test_refusals_without_gpu(kv4):
    lib, V = kv4.lib, ctypes.c_void_p
    A = 1 << 20
    geo = dict(num_layers=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, num_sinks=4, recent_window=16, hadamard_block=128, max_seqs=8, max_pages=10)
    h = kv4.kv4_cache_init(kv4.kv4_config(**geo), A, A)
    vb = kv4.kv4_cache_init(kv4.kv4_config(**dict(geo, value_format=1)), A, A)
    mx = kv4.kv4_cache_init(kv4.kv4_config(**dict(geo, num_sinks=0, recent_window=0, hadamard_block=1, value_format=2, key_bits=3, value_bits=3)), A, 0)
    bf = kv4.kv4_bf16_cache_init(kv4.kv4_config(**geo), A)

    def call(h, layer=0, B=4, q=A, qd=1, pt=A, stride=4, lens=A, n=1, start=A, prefix=A, hint=0, out=A, od=1, ws=A, wsb=1 << 40):
        return lib.kv4_decode_attn_shared(V(h), layer, B, V(q), qd, V(pt), stride, V(lens), n, V(start), V(prefix), hint, V(out), od, None, V(ws),
                                          ctypes.c_size_t(wsb), None)

    try:
        for kw in (dict(layer=2), dict(layer=-1), dict(B=-1), dict(B=9), dict(q=None), dict(qd=3), dict(pt=None), dict(stride=0), dict(lens=None), dict(n=-1),
                   dict(n=(1 << 20) + 1), dict(start=None), dict(prefix=None), dict(hint=-1), dict(out=None), dict(out=A + 8), dict(od=3)):
            assert call(h, **kw) == kv4.KV4_ERR_INVALID_ARG, kw
        assert call(h, ws=None) == kv4.KV4_ERR_WORKSPACE and call(h, ws=A + 8) == kv4.KV4_ERR_WORKSPACE
        assert call(h, B=0) == 0
        assert call(None) == 1 and call(mx) == 1 and call(bf) == 1 and call(vb) == kv4.KV4_ERR_UNSUPPORTED
        n = ctypes.c_size_t()
        ws = lambda h, B, g: lib.kv4_decode_shared_workspace_bytes(V(h), B, g, ctypes.byref(n))  # noqa: E731
        assert ws(h, -1, 1) == 1 and ws(h, 1, -1) == 1 and ws(mx, 1, 1) == 1 and ws(vb, 1, 1) == 2 and ws(None, 1, 1) == 1
    finally:
        for x in (h, vb, mx, bf):
            kv4.kv4_cache_destroy(x)


@gpu
def test_workspace_too_small(kv4):
    r = build(CASES[0], kv4)
    n = kv4.kv4_decode_shared_workspace_bytes(r.cache.handle, r.wl.B, 1)
    with pytest.raises(kv4.KV4Error) as e:
        r.cache.decode_shared(0, r.q, r.pt, r.lens, r.start_d, r.prefix_d, workspace=torch.empty(n - 16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == kv4.KV4_ERR_WORKSPACE


@gpu
def test_values_beyond_fp16(kv4):
    """A value vector whose INT4 scale reaches values past the fp16 range, among ordinary ones."""
    r = build(CASES[0], kv4)
    L, hot = 240, 133
    wl = r.wl
    b = np.zeros(2, np.int32)
    p = np.array([hot, 70], np.int32)
    K, V = wl.kv_inputs(0, b, p)
    V[0] = np.linspace(-60000.0, 500000.0, V[0].size).reshape(V[0].shape)
    V[1] = np.linspace(3e-4, 5e-4, V[1].size).reshape(V[1].shape)
    K[0] = -20 * wl.kv_inputs(0, b[:1], p[:1])[0][0]
    keep = r.side.copy()
    O.append(r.cfg, r.pool, r.side, K, V, b, p, wl.lens, wl.page_table)
    assert np.array_equal(keep, r.side)
    r.cache.layer_views(0)[0].copy_(torch.from_numpy(r.pool))
    want = reference(r)
    out = r.cache.decode_shared(0, r.q, r.pt, r.lens, r.start_d, r.prefix_d, out=torch.empty(r.q.shape, device="cuda"))
    assert np.isfinite(want[0]).all() and want[2].max() < 1e5
    check(r, out, None, want)


@gpu
@pytest.mark.parametrize("name", ["ragged", "b300", "long"])
def test_wait_limit_failure_path_reports_and_recovers(kv4, name):
    """The bounded waits made to run out by the test hook: the error bit is set, the kernels end, the
    context stays usable and the next call is right."""
    r = build(CASES[IDS.index(name)], kv4)
    want = reference(r)
    n = kv4.kv4_decode_shared_workspace_bytes(r.cache.handle, r.wl.B, len(r.prefix))
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    kv4.kv4_debug_force_wait_timeout(r.cache.handle, True)
    try:
        r.cache.decode_shared(0, r.q, r.pt, r.lens, r.start_d, r.prefix_d, workspace=ws)
        torch.cuda.synchronize()
    finally:
        kv4.kv4_debug_force_wait_timeout(r.cache.handle, False)
    assert kv4.kv4_get_device_error() & kv4.KV4_DEVERR_WAIT_LIMIT
    lse = torch.empty((r.wl.B, r.wl.Hq), device="cuda")
    out = r.cache.decode_shared(0, r.q, r.pt, r.lens, r.start_d, r.prefix_d, lse=lse, workspace=ws)
    check(r, out, lse, want, 2.0 ** -8)
    assert kv4.kv4_get_device_error() == 0


@gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_query_stays_in_its_row(kv4, bad):
    r = build(CASES[IDS.index("many-rows")], kv4)
    want = r.cache.decode_shared(0, r.q, r.pt, r.lens, r.start_d, r.prefix_d)
    q = r.q.clone()
    q[3, 1] = bad
    got = r.cache.decode_shared(0, q, r.pt, r.lens, r.start_d, r.prefix_d)
    other = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
    other[3, 1] = False
    assert torch.equal(got[other], want[other])


@gpu
def test_python_checks(kv4):
    r = build(CASES[0], kv4)
    call = lambda **kw: r.cache.decode_shared(0, r.q, r.pt, r.lens, r.start_d, r.prefix_d, **kw)  # noqa: E731
    for kw in (dict(lse=torch.empty(r.wl.B, 1, device="cuda")), dict(lse=torch.empty(r.wl.B, r.wl.Hq, dtype=torch.float64, device="cuda")),
               dict(out=torch.empty(r.wl.B, r.wl.Hq, 1, device="cuda")), dict(workspace=torch.empty(1 << 20, device="cuda"))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ValueError):
        r.cache.decode_shared(0, r.q.transpose(0, 1).contiguous().transpose(0, 1), r.pt, r.lens, r.start_d, r.prefix_d)
    with pytest.raises(ValueError):
        r.cache.decode_shared(0, r.q, r.pt, r.lens, r.start_d[:1], r.prefix_d)
