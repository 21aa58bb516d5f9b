"""Shared-prefix batches long enough for a thread block of the prefix kernel to take many 128-position
units, with the cache bytes of the CPU oracle, and an fp64 reference of chosen query heads.

A group's prefix is appended once, through its first row; the other rows append what is theirs: the
positions past the shared pages, their sinks and their recent window.  ``reference`` and its bound
are those of test_gpu_shared.py, on the dequantised cache, for any queries."""
import numpy as np
import torch

from oracle import oracle as O

UNIT = 128  # positions of a unit
ROWS = 64   # query rows of a segment


class Batch:
    pass


def units(r):
    """Units of the prefix kernel: per group of two rows and more, KV head and block of query rows, the 128-position tiles
    from the tile of the first position past the sinks to the end of the whole pages of the prefix."""
    total = 0
    for n, p in zip(r.sizes, r.prefix):
        if n == 1:
            continue
        te = p // r.P * r.P // 16
        tiles = -(-(te - r.s // 16) // (UNIT // 16)) if 16 * te > r.s else 0
        total += r.Hkv * -(-n * r.G // ROWS) * tiles
    return total


def batch(D, G, Hkv, P, s, w, h, sizes, prefix, past, seed=0, edit=None, ends_differ=False, scale=1.0):
    """past[b]: row b's length beyond its group's prefix (negative: it ends inside).  edit(group, K, V)
    changes a group's prefix [length][Hkv][D] in place.  ends_differ: positions of a prefix that lie past
    its last whole page are each row's own.  scale: of the keys past the prefixes."""
    rng = np.random.default_rng(seed)
    r = Batch()
    r.D, r.G, r.Hkv, r.P, r.s, r.w, r.h, r.sizes, r.prefix = D, G, Hkv, P, s, w, h, sizes, list(prefix)
    r.Hq, r.B = G * Hkv, sum(sizes)
    r.group = np.repeat(np.arange(len(sizes)), sizes)
    r.start = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    r.lens = np.array([prefix[g] + d for g, d in zip(r.group, past)], np.int32)
    assert all(past[b] >= 0 for b in r.start[:-1]), "the first row of a group covers its prefix"
    whole = [p // P * P for p in prefix]
    need = [-(-int(L) // P) for L in r.lens]
    r.table = np.zeros((r.B, max(need)), np.int32)
    used = 0
    for b, (g, n) in enumerate(zip(r.group, need)):
        k = 0 if b == r.start[g] else min(n, whole[g] // P)
        r.table[b, :k] = r.table[r.start[g], :k]
        r.table[b, k:n] = np.arange(used, used + n - k)
        used += n - k
    r.pages = used
    r.table = rng.permutation(used).astype(np.int32)[r.table]
    r.cfg = O.Config(r.Hq, Hkv, D, P, s, w, h, r.B, (0, 0, 0, 0), 0, 0)
    r.pool = np.full(O.page_bytes(r.cfg) * used, 0xA5, np.uint8)
    r.side = np.full(max(O.side_slot_bytes(r.cfg) * r.B, 1), 0xA5, np.uint8)
    for g, p in enumerate(prefix):
        K, V = (rng.standard_normal((p, Hkv, D)).astype(np.float32) for _ in range(2))
        if edit is not None:
            edit(g, K, V)
        for b in range(r.start[g], r.start[g + 1]):
            L = int(r.lens[b])
            Kt, Vt = (rng.standard_normal((max(L - whole[g], 0), Hkv, D)).astype(np.float32) for _ in range(2))
            Kt *= np.float32(scale)
            if not ends_differ:
                n = min(p, L) - whole[g]
                if n > 0:
                    Kt[:n], Vt[:n] = K[whole[g]:whole[g] + n], V[whole[g]:whole[g] + n]
            mine = np.arange(L)
            if b != r.start[g]:
                mine = mine[(mine < s) | (mine >= min(whole[g], L - w))]
            at = mine < whole[g]
            O.append(r.cfg, r.pool, r.side, np.concatenate([K[mine[at]], Kt[mine[~at] - whole[g]]]),
                     np.concatenate([V[mine[at]], Vt[mine[~at] - whole[g]]]), np.full(mine.size, b, np.int32), mine.astype(np.int32), r.lens, r.table)
    r.q = rng.standard_normal((r.B, r.Hq, D)).astype(np.float32)
    return r


def to_gpu(r):
    from int4_kv_cache_append_b200 import kv4
    r.cache = kv4.Cache(kv4.Geometry(1, r.Hq, r.Hkv, r.D, r.P, r.s, r.w, r.h, r.B, r.pages), fill=0xA5)
    pool, side = r.cache.layer_views(0)
    pool.copy_(torch.from_numpy(r.pool))
    n = min(side.numel(), r.side.size)
    side[:n].copy_(torch.from_numpy(r.side[:n]))
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    r.table_d, r.lens_d, r.start_d, r.prefix_d = dev(r.table), dev(r.lens), dev(r.start), dev(r.prefix)
    return r


def decode(r, q=None, **kw):
    """fp32 (out, lse) of the shared decode."""
    q = torch.from_numpy(r.q if q is None else q).cuda()
    out, lse = torch.full(q.shape, float("nan"), device="cuda"), torch.full(q.shape[:2], float("nan"), device="cuda")
    r.cache.decode_shared(0, q, r.table_d, r.lens_d, r.start_d, r.prefix_d, out=out, lse=lse, **kw)
    return out, lse


def reference(r, picks, q=None, floor=2.0 ** -25):
    """[(out [D], its bound [D], log-sum, its bound)] of the (row, query head) picks.  floor: what a
    probability may lose below fp16's normal range, of the row's largest."""
    q = r.q if q is None else q
    u = 1.05 * 2.0 ** -11
    res, last, kv = [], None, None
    for b, j in sorted(picks):
        if last != (b, j // r.G):
            last, kv = (b, j // r.G), O.dequant_seq(r.cfg, r.pool, r.side, r.table[b], b, int(r.lens[b]), j // r.G)[:2]
        k, v = kv
        qs = O.fwht_f64(q[b, j].astype(np.float64), r.h) / r.h / np.sqrt(r.D)
        x = k @ qs
        e = np.exp(x - x.max())
        total = e.sum()
        p = e / total
        qr = np.abs(qs)
        o, km, d = p @ v, p @ k, u * (np.abs(k) @ qr).max()
        cov = (k - km).T @ ((v - o) * p[:, None])
        bound = u * (qr @ np.abs(cov) + 2 * (p @ np.abs(v))) + 2 * d * d * (p @ np.abs(v - o)) + floor * np.abs(v).sum(0) / total
        res.append((o, bound + 2e-4 * max(1.0, np.abs(o).max()), x.max() + np.log(total), u * (qr @ np.abs(km)) + d * d + 1e-4))
    return res


def check(r, out, lse, picks, **kw):
    out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    for (b, j), (o, bo, ls, bl) in zip(sorted(picks), reference(r, picks, **kw)):
        err = np.abs(out[b, j] - o)
        assert np.all(err <= bo), f"row {b} head {j}: worst {np.max(err / bo):.2f} of the bound"
        assert abs(lse[b, j] - ls) <= bl, f"row {b} head {j}: log-sum off by {abs(lse[b, j] - ls):.2e}, bound {bl:.2e}"


def picks_of(r, per_row=2, seed=1):
    """A few query heads of every row, each KV head's among them."""
    rng = np.random.default_rng(seed)
    return sorted({(b, int(j)) for b in range(r.B) for j in [(b * r.G + b) % r.Hq, *rng.integers(0, r.Hq, per_row - 1)]})
