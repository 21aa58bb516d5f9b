"""kv4_decode_attn_shared on prefixes of many units a thread block: the straight softmax path, buffers
used again, segments and groups that change inside a block, running maxima raised in later units.
Tolerances: the derived bounds of shared_long.reference."""
import numpy as np
import pytest
import torch

import shared_long as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv4():
    from int4_kv_cache_append_b200 import kv4
    return kv4


@pytest.fixture(autouse=True)
def no_device_error(kv4):
    yield
    assert kv4.kv4_get_device_error() == 0


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# (name, arguments of batch)
CASES = {
    "ten-units-a-block": dict(D=128, G=4, Hkv=8, P=16, s=4, w=16, h=128, sizes=[2, 1, 3, 2], prefix=[9000, 5003, 9007, 3000], past=[40, 1, 300, 5, 77, -700, 8, 9]),
    "two-row-blocks": dict(D=128, G=4, Hkv=4, P=64, s=16, w=32, h=64, sizes=[17, 4], prefix=[8000, 6050], past=[3 * i + 1 for i in range(21)]),
    "two-row-blocks-d64-p48": dict(D=64, G=2, Hkv=4, P=48, s=0, w=24, h=16, sizes=[40, 2], prefix=[6000, 9001], past=[2 * i for i in range(42)]),
    "one-query-head-d64": dict(D=64, G=1, Hkv=8, P=32, s=4, w=0, h=64, sizes=[3, 2, 2], prefix=[4111, 6000, 3001], past=[0, 9, 2, 30, 4, 50, 6]),
    "rows-end-inside": dict(D=128, G=2, Hkv=8, P=16, s=4, w=128, h=128, sizes=[6], prefix=[11000], past=[5, -3, -130, -4000, -10990, 200]),
}


@pytest.mark.parametrize("name", CASES)
def test_matches_oracle(kv4, name):
    r = L.to_gpu(L.batch(**CASES[name]))
    assert L.units(r) > 4 * sms()
    out, lse = L.decode(r)
    L.check(r, out, lse, L.picks_of(r))
    again = L.decode(r)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def growing(step, stride):
    """Keys whose logits rise by `step` (log2) every `stride` positions, for queries along u."""
    def edit(g, K, V):
        n, Hkv, D = K.shape
        u = np.full(D, 1 / np.sqrt(D), np.float32)
        K *= 0.5
        K += ((np.arange(n) // stride) * (step * np.log(2) * np.sqrt(D) / 20)).astype(np.float32)[:, None, None] * u
    return edit


@pytest.mark.parametrize("step,stride", [(13.0, 1500), (2.5, 250), (-13.0, 1500)])
def test_maxima_raised_in_later_units(kv4, step, stride):
    """Logits that rise (or fall) along the prefix: outputs and sums are rescaled in mid-segment."""
    r = L.to_gpu(L.batch(128, 4, 8, 16, 4, 16, 128, [3, 2], [9000, 8000], [10, 20, 30, 40, 50], edit=growing(step, stride)))
    assert L.units(r) > 4 * sms()
    q = (0.5 * r.q + 20 / np.sqrt(r.D)).astype(np.float32)
    out, lse = L.decode(r, q)
    L.check(r, out, lse, L.picks_of(r), q=q)


def test_large_values_in_mid_segment(kv4):
    """Value vectors whose codes reach past fp16, in single units far from a segment's ends."""
    hot = (3333, 3334, 6001)

    def edit(g, K, V):
        for i in hot:
            V[i] = np.linspace(-60000.0, 500000.0, V[i].size).reshape(V[i].shape)
            K[i] = 0.05 * K[i]  # a logit near zero
        K[1000] += 3  # some position that matters more than the large ones
    r = L.to_gpu(L.batch(128, 4, 8, 16, 4, 16, 128, [2, 2], [9000, 7000], [10, 20, 30, 40], edit=edit))
    assert L.units(r) > 4 * sms()
    out, lse = L.decode(r)
    L.check(r, out, lse, L.picks_of(r))


def test_two_streams_and_replay(kv4):
    r = L.to_gpu(L.batch(**CASES["ten-units-a-block"]))
    want = L.decode(r)
    n = kv4.kv4_decode_shared_workspace_bytes(r.cache.handle, r.B, len(r.sizes))
    q = torch.from_numpy(r.q).cuda()
    torch.cuda.synchronize()
    runs = []
    for _ in range(2):
        st, ws, out = torch.cuda.Stream(), torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), torch.empty_like(want[0])
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for _ in range(4):
                r.cache.decode_shared(0, q, r.table_d, r.lens_d, r.start_d, r.prefix_d, out=out, workspace=ws)
        runs.append(out)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[0]) for x in runs)
    g, out = torch.cuda.CUDAGraph(), torch.zeros_like(want[0])
    with torch.cuda.graph(g):
        r.cache.decode_shared(0, q, r.table_d, r.lens_d, r.start_d, r.prefix_d, out=out)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0])


def test_scaled_and_ordinary_queries_in_one_group(kv4):
    """Every third query is 2^17 as large: past fp16 once rotated, so its row is scaled by a power of two and
    its neighbours' are not.  Keys of 2^-15 keep its logits moderate."""
    def edit(g, K, V):
        K *= 2.0 ** -15

    r = L.batch(128, 4, 2, 16, 0, 0, 64, [5, 3], [1500, 900], [0, 16, 32, 5, 40, 0, 7, 20], edit=edit, scale=2.0 ** -15)
    big = (np.arange(r.B * r.Hq) % 3 == 1).reshape(r.B, r.Hq)
    q = r.q.copy()
    q[big] *= 2.0 ** 17
    # what enters fp16: the rotated query in log2 units, times 64
    rot = np.array([np.abs(L.O.fwht_f64(x.astype(np.float64), 64)).max() for x in q.reshape(-1, 128)]).reshape(big.shape) / np.log(2) / np.sqrt(128)
    assert rot[big].min() > 32768 > rot[~big].max()
    L.to_gpu(r)
    out, lse = L.decode(r, q)
    L.check(r, out, lse, [(b, j) for b in range(r.B) for j in range(r.Hq)], q=q)


@pytest.mark.parametrize("f", [2.0 ** 40, 2.0 ** 90])
def test_enormous_queries_pick_the_largest_logit(kv4, f):
    """With one key far along the query, the output is that position's value.  The logits are 1e12 and more
    apart, so no rounding of a query or a product (relative 2^-11) changes the order."""
    at = 777

    def edit(g, K, V):
        K *= 0.05
        K[at] = 4.0
    r = L.to_gpu(L.batch(128, 4, 2, 16, 4, 16, 128, [4], [1500], [1, 20, 33, 40], edit=edit))
    q = (np.abs(r.q) * f).astype(np.float32)
    out = L.decode(r, q)[0].cpu().numpy().astype(np.float64)
    for b in range(r.B):
        for g in range(r.Hkv):
            k, v, _ = L.O.dequant_seq(r.cfg, r.pool, r.side, r.table[b], b, int(r.lens[b]), g)
            for j in range(g * r.G, (g + 1) * r.G):
                x = k @ L.O.fwht_f64(q[b, j].astype(np.float64) / f, r.h) / r.h
                others = np.delete(x, at)
                assert x[at] > 2 * others.max() > 0  # far more than 2^-11 ahead
                assert np.all(np.abs(out[b, j] - v[at]) <= 1.05 * 2.0 ** -10 * np.abs(v[at]) + 2e-4)


@pytest.mark.parametrize("P,prefix", [(64, [2000, 130]), (48, [1000, 47]), (32, [527, 300])])
def test_prefix_that_ends_inside_a_page(kv4, P, prefix):
    """What lies past a prefix's last whole page is each row's own page, whatever prefix_len counts."""
    r = L.to_gpu(L.batch(128, 4, 2, P, 4, 16, 128, [3, 2], prefix, [40, 1, 200, 30, 99], ends_differ=True))
    out, lse = L.decode(r)
    L.check(r, out, lse, L.picks_of(r, 4))


@pytest.mark.parametrize("name", ["ten-units-a-block", "two-row-blocks-d64-p48"])
def test_waits_that_run_out_in_mid_pipeline(kv4, name):
    """The bounded waits made to run out (1 ms) with most units of every block to come: the error bit is set,
    the call ends soon after, and the next one is right."""
    r = L.to_gpu(L.batch(**CASES[name]))
    want = L.decode(r)
    ws = torch.full((kv4.kv4_decode_shared_workspace_bytes(r.cache.handle, r.B, len(r.sizes)),), 0xA5, dtype=torch.uint8, device="cuda")
    at = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    kv4.kv4_debug_force_wait_timeout(r.cache.handle, True)
    try:
        at[0].record()
        L.decode(r, workspace=ws)
        at[1].record()
        torch.cuda.synchronize()
    finally:
        kv4.kv4_debug_force_wait_timeout(r.cache.handle, False)
    assert kv4.kv4_get_device_error() & kv4.KV4_DEVERR_WAIT_LIMIT
    assert at[0].elapsed_time(at[1]) < 200
    got = L.decode(r, workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("below", [25.6, 27.0])
def test_many_small_probabilities_are_not_lost(kv4, below):
    """One position ahead of all others by 2^`below`: the 1200 after it that a thread block takes with it add
    up to 2e-5 of the sum, and with values of 1000 where all other values are zero they are the output."""
    def edit(g, K, V):
        u = np.full(K.shape[2], 1 / np.sqrt(K.shape[2]), np.float32)
        K *= 0.05
        K -= (K @ u)[..., None] * u
        K[40] += (below * np.log(2) * np.sqrt(K.shape[2]) / 20) * u
        V *= 100
        V += 1000
        V[:41] = 0
        V[1280:] = 0
    r = L.to_gpu(L.batch(128, 4, 8, 16, 0, 0, 128, [2, 2], [12000, 12000], [0, 16, 0, 0], edit=edit))
    assert L.units(r) > 10 * sms()
    q = np.full_like(r.q, 20 / np.sqrt(r.D))
    out, lse = L.decode(r, q)
    L.check(r, out, lse, [(b, j) for b in range(2) for j in range(4)], q=q, floor=2.0 ** -29)


def test_a_group_of_one_row_shares_nothing(kv4):
    """Rows that form groups of one get what a call without groups gives, bit for bit."""
    r = L.to_gpu(L.batch(128, 4, 2, 16, 4, 16, 128, [1, 3, 1, 1, 2], [900, 700, 30, 2000, 500], [5, 6, 7, 8, 9, 10, 11, 12]))
    out, lse = L.decode(r)
    L.check(r, out, lse, L.picks_of(r, 4))
    r.start_d, r.prefix_d = r.start_d[:1], r.prefix_d[:0]
    plain = L.decode(r)
    r.start_d, r.prefix_d = torch.arange(r.B + 1, device="cuda", dtype=torch.int32), torch.full((r.B,), 10000, device="cuda", dtype=torch.int32)
    single = L.decode(r)
    assert torch.equal(single[0], plain[0]) and torch.equal(single[1], plain[1])
