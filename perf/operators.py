"""Cases of the operators around the paged KV cache: the cos/sin table of a rotary embedding, the
per-head norm and rotation of queries and keys, the append that rotates and quantises on the way
(read back as values), and decode attention for batches whose sequences share a long prefix.

``run`` computes an operator either in its plain form (elementary torch operations) or, with
``own`` set, through the library.  ``exact`` restates the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

BF16 = torch.bfloat16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a small model's table for its whole context, no scaling
        {"name": "table-8k", "op": "table", "R": 64, "max_pos": 8192, "base": 10000.0, "scaling": "none", "factor": 1.0, "orig": 0},
        # a long-context table: frequencies blended for 4x the trained length
        {"name": "table-128k-yarn", "op": "table", "R": 128, "max_pos": 131072, "base": 1000000.0, "scaling": "yarn", "factor": 4.0, "orig": 32768},
        # one decode step of 64 sequences before an attention that keeps its own cache
        {"name": "rope-step-64", "op": "rope", "T": 64, "Hq": 32, "Hkv": 8, "D": 128, "R": 128, "layout": "half", "norm": True},
        # a prefill: 16383 tokens, half of each head rotated, neighbouring pairs
        {"name": "rope-prefill-16k", "op": "rope", "T": 16383, "Hq": 32, "Hkv": 8, "D": 128, "R": 64, "layout": "interleaved", "norm": True},
        # one decode step of the 8B loop: 128 sequences, one token each, read back as values
        {"name": "append-step-128", "op": "append", "fmt": "int4", "B": 128, "chunk": 1, "context": 600, "read": "new", "Hq": 32, "Hkv": 8, "D": 128,
         "R": 128, "layout": "half", "norm": True, "P": 16, "s": 16, "w": 128, "h": 128, "lens_seed": 5},
        # chunked prefill: 8 sequences append 512 tokens each and read their whole contexts back
        {"name": "append-chunk-8x512", "op": "append", "fmt": "int4", "B": 8, "chunk": 512, "context": 4000, "read": "all", "Hq": 32, "Hkv": 8, "D": 128,
         "R": 128, "layout": "half", "norm": True, "P": 16, "s": 4, "w": 128, "h": 128, "lens_seed": 6},
        # the mixed bit-width cache (K3V3): a ragged prefill of 5 prompts
        {"name": "append-mixed-5x401", "op": "append", "fmt": "mixed", "B": 5, "chunk": 401, "context": 0, "read": "new", "Hq": 32, "Hkv": 8, "D": 128,
         "R": 128, "layout": "half", "norm": False, "P": 16, "s": 0, "w": 0, "h": 1, "lens_seed": 7},
        # a refill: 16 prompts of about 1000 tokens in 64-position pages, rotation in blocks of 64
        {"name": "append-refill-16k", "op": "append", "fmt": "int4", "B": 16, "chunk": 1000, "context": 0, "read": "new", "Hq": 32, "Hkv": 8, "D": 128,
         "R": 128, "layout": "interleaved", "norm": True, "P": 64, "s": 4, "w": 256, "h": 64, "lens_seed": 8},
        # four answers to one short prompt on a tiny model: latency
        {"name": "shared-tiny-4", "op": "shared", "groups": 1, "per": 4, "ragged": False, "prefix": 256, "suffix": 64, "Hq": 2, "Hkv": 1, "D": 64, "P": 16,
         "s": 4, "w": 32, "h": 64, "lens_seed": 9},
        # rollouts: 8 prompts of about 2000 tokens, 8 answers each, part way through
        {"name": "shared-8x8-2k", "op": "shared", "groups": 8, "per": 8, "ragged": False, "prefix": 2048, "suffix": 2048, "Hq": 32, "Hkv": 8, "D": 128, "P": 16,
         "s": 4, "w": 128, "h": 128, "lens_seed": 10},
        # ragged groups of up to 16 answers over prompts of up to 8192 tokens
        {"name": "shared-16x16-8k", "op": "shared", "groups": 16, "per": 16, "ragged": True, "prefix": 8192, "suffix": 1024, "Hq": 32, "Hkv": 8, "D": 128, "P": 16,
         "s": 4, "w": 128, "h": 64, "lens_seed": 11},
        # 128 answers to one prompt of 16384 tokens: many query rows on the same keys
        {"name": "shared-1x128-16k", "op": "shared", "groups": 1, "per": 128, "ragged": False, "prefix": 16384, "suffix": 1024, "Hq": 32, "Hkv": 8, "D": 128, "P": 64,
         "s": 16, "w": 128, "h": 128, "lens_seed": 12},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "rope", "append", "append", "shared", "shared"])
    D = rng.choice([64, 128, 128])
    R = 8 * rng.randint(2, D // 8) if rng.random() < 0.5 else D
    if op == "table":
        return {"op": op, "R": 8 * rng.randint(2, 16), "max_pos": _log_int(rng, 64, 131072), "base": rng.choice([10000.0, 500000.0, 1000000.0]),
                "scaling": rng.choice(["none", "linear", "ntk", "yarn", "bands"]), "factor": rng.choice([2.0, 4.0, 8.0]), "orig": rng.choice([2048, 8192, 32768])}
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4])
    layout = rng.choice(["half", "interleaved"])
    norm = rng.random() < 0.7
    if op == "rope":
        return {"op": op, "T": _log_int(rng, 1, 16383), "Hq": Hq, "Hkv": Hkv, "D": D, "R": R, "layout": layout, "norm": norm}
    if op == "append":
        fmt = rng.choice(["int4", "int4", "mixed"])
        B = _log_int(rng, 1, 64)
        chunk = _log_int(rng, 1, max(1, min(1000, 16000 // B)))
        context = rng.randint(0, max(1, 32000 // B - chunk)) if rng.random() < 0.6 else 0
        s, w, h = (0, 0, 1) if fmt == "mixed" else (rng.choice([0, 4, 16]), rng.choice([0, 32, 128]), rng.choice([1, 16, 64]))
        return {"op": op, "fmt": fmt, "B": B, "chunk": chunk, "context": context, "read": rng.choice(["new", "all"]), "Hq": Hq, "Hkv": Hkv, "D": D, "R": R,
                "layout": layout, "norm": norm, "P": rng.choice([16, 32, 48, 64]), "s": s, "w": w, "h": h, "lens_seed": rng.randint(0, 1 << 20)}
    groups = _log_int(rng, 1, 16)
    prefix = _log_int(rng, 17, min(16384, 131072 // groups))
    per = _log_int(rng, 1, max(1, min(128, 256 // groups, 2000000 // (groups * (prefix + 1024)))))
    return {"op": op, "groups": groups, "per": per, "ragged": rng.random() < 0.5, "prefix": prefix,
            "suffix": _log_int(rng, 1, 1024), "Hq": Hq, "Hkv": Hkv, "D": D, "P": rng.choice([16, 32, 48, 64]), "s": rng.choice([0, 4, 16]),
            "w": rng.choice([0, 32, 128]), "h": rng.choice([1, 16, 64]), "lens_seed": rng.randint(0, 1 << 20)}


def work(case):
    op = case["op"]
    if op == "table":
        n = case["max_pos"] * case["R"] // 2
        return {"bytes": 8 * n, "flops": 12 * n}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if op == "rope":
        T, H = case["T"], Hq + Hkv
        return {"bytes": T * (2 * H * D * 2 + 4 + 4 * case["R"]), "flops": T * H * D * 6}
    if op == "append":
        p = _append_plan(case)
        T, N = len(p["pos"]), len(p["read_pos"])
        row = 6 * D // 8 + 8 if case["fmt"] == "mixed" else D + 8  # K3V3, or INT4 with its scales and zeros
        kept = int(((p["pos"] < case["s"]) | (p["pos"] >= p["lens"][p["slot"]] - case["w"])).sum()) if case["s"] + case["w"] else 0
        fresh = T * (2 * (Hq + 2 * Hkv) * D + 2 * Hq * D + Hkv * row + 4 * case["R"]) + kept * Hkv * (2 * D + 4)
        return {"bytes": fresh + N * Hkv * (row + 4 * D), "flops": T * (Hq + Hkv) * D * 6 + (T + N) * Hkv * D * (4 + 2 * int(math.log2(case["h"])))}
    p = _shared_plan(case)
    m_end = np.maximum(case["s"], p["lens"] - case["w"])
    n8 = int(np.minimum(p["lens"], case["s"] + case["w"]).sum())
    first = np.clip(p["prefix"][p["group"]], case["s"], m_end)
    n4 = int((m_end - first).sum()) + int(np.maximum(0, np.minimum(p["prefix"], _group_max(p, m_end)) - case["s"]).sum())
    B = len(p["lens"])
    return {"bytes": Hkv * (n4 * (D + 8) + n8 * (2 * D + 4)) + 4 * B * Hq * D, "flops": 4 * Hq * D * int(p["lens"].sum())}


def _group_max(p, x):
    return np.array([x[a:b].max() if b > a else 0 for a, b in zip(p["start"][:-1], p["start"][1:])])


# ------------------------------------------------------------------ plans: lengths and pages of a case

def _pages(rng, rows, P, shared=None):
    """Page tables [B][stride] over a shuffled pool.  shared: (group of each row, whole pages of each group's prefix)."""
    need = [-(-int(L) // P) for L in rows]
    table = np.zeros((len(rows), max(max(need), 1)), np.int64)
    owner, used = {}, 0
    for b, n in enumerate(need):
        g = shared[0][b] if shared is not None else b
        whole = min(n, int(shared[1][g])) if g in owner else 0
        table[b, :whole] = table[owner.setdefault(g, b), :whole]
        table[b, whole:n] = np.arange(used, used + n - whole)
        used += n - whole
    ids = list(range(max(used, 1)))
    rng.shuffle(ids)
    return np.array(ids, np.int32)[table], len(ids)


def _append_plan(case):
    rng = random.Random(case["lens_seed"])
    B, chunk = case["B"], case["chunk"]
    new = [chunk if chunk == 1 else max(1, chunk - rng.randint(0, chunk // 4)) for _ in range(B)]
    old = [rng.randint(0, case["context"]) for _ in range(B)]
    lens = np.array([a + b for a, b in zip(old, new)], np.int32)
    table, pages = _pages(rng, lens, case["P"])
    cat = lambda lo, hi: np.concatenate([np.arange(a, b, dtype=np.int32) for a, b in zip(lo, hi)])  # noqa: E731
    rep = lambda n: np.repeat(np.arange(B, dtype=np.int32), n)  # noqa: E731
    lo = old if case["read"] == "new" else [0] * B
    return {"lens": lens, "old": np.array(old, np.int32), "table": table, "pages": pages, "slot": rep(new), "pos": cat(old, lens), "old_slot": rep(old),
            "old_pos": cat([0] * B, old), "read_slot": rep([n - a for a, n in zip(lo, lens)]), "read_pos": cat(lo, lens)}


def _shared_plan(case):
    rng = random.Random(case["lens_seed"])
    G = case["groups"]
    per = [rng.randint(1, case["per"]) if case["ragged"] else case["per"] for _ in range(G)]
    prefix = np.array([case["prefix"] - (rng.randint(0, case["prefix"] // 2) if case["ragged"] else 0) for _ in range(G)], np.int32)
    start = np.concatenate([[0], np.cumsum(per)]).astype(np.int32)
    group = np.repeat(np.arange(G), per)
    lens = np.array([prefix[g] + rng.randint(1, case["suffix"]) for g in group], np.int32)
    table, pages = _pages(rng, lens, case["P"], (group, prefix // case["P"]))
    return {"lens": lens, "prefix": prefix, "start": start, "group": group, "table": table, "pages": pages, "per": per}


# ------------------------------------------------------------------ inputs

def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _randn(gen, *shape, dtype=BF16):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _frequencies(case):
    """Angle of pair i per position, in 64 bits, and the factor on cos and sin."""
    R, base, f, L = case["R"], case["base"], case["factor"], case["orig"]
    i = torch.arange(R // 2, dtype=torch.float64)
    kind = case["scaling"]
    if kind == "ntk":
        return (base * f ** (R / (R - 2))) ** (-2 * i / R), 1.0
    inv = base ** (-2 * i / R)
    if kind == "linear":
        return inv / f, 1.0
    if kind == "yarn":  # rotations over the trained length: 32 and more are kept, 1 and fewer divided
        dim = lambda n: R * math.log(L / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), R - 1)
        ramp = ((i - low) / (high - low if high > low else 0.001)).clamp(0, 1)
        return inv / f * ramp + inv * (1 - ramp), 0.1 * math.log(f) + 1.0
    if kind == "bands":  # wavelengths up to L / 4 are kept, those past L / 1 divided, blended between
        turns = L * inv / (2 * math.pi)
        smooth = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return (1 - smooth) * inv / f + smooth * inv, 1.0
    return inv, 1.0


def _table(freq, mult, max_pos):
    a = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * freq.cuda()
    return torch.stack([(a.cos() * mult).float(), (a.sin() * mult).float()], -1)


def _rope_inputs(gen, case, T, max_pos):
    Hq, Hkv, D, R = case["Hq"], case["Hkv"], case["D"], case["R"]
    qkv = _randn(gen, T, (Hq + 2 * Hkv) * D)  # the fused projection's output; a few strong rotary pairs in the keys
    strong = torch.randint(0, Hkv * D, (2 * Hkv,), generator=gen, device="cuda")
    qkv[:, Hq * D + strong] *= 8
    s = {"qkv": qkv, "q": qkv[:, :Hq * D].view(T, Hq, D), "k": qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D), "v": qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)}
    s["freq"], s["mult"] = _frequencies({"R": R, "base": 1000000.0, "scaling": "none", "factor": 1.0, "orig": 0})
    s["table"] = _table(s["freq"], s["mult"], max_pos)
    s["qw"], s["kw"] = ((1 + 0.2 * _randn(gen, D, dtype=torch.float32)).to(BF16) for _ in range(2)) if case["norm"] else (None, None)
    if own:
        from int4_kv_cache_append_b200 import kv4
        geo = kv4.RopeGeometry(R, max_pos, kv4.KV4_ROPE_HALF if case["layout"] == "half" else kv4.KV4_ROPE_INTERLEAVED, 1000000.0)
        s["rope"] = kv4.Rope(geo, q_weight=s["qw"], k_weight=s["kw"], eps=1e-6)
    return s


def _allocation(gen, Hkv, D, bits):
    """Block widths and scales of a mixed bit-width layer: one bit at a time to the block of largest energy 4^-bits."""
    sigma = torch.exp(0.5 * torch.randn(Hkv, D // 2, generator=gen, device="cuda")).cpu().numpy().astype(np.float32)
    width = np.zeros((Hkv, D // 2), np.int64)
    rows = np.arange(Hkv)
    for _ in range(bits * D // 2):
        gain = np.where(width < 8, sigma.astype(np.float64) ** 2 * 4.0 ** -width, -1)
        width[rows, gain.argmax(1)] += 1
    return width.astype(np.uint8), sigma


def _store(case, pages, slots, gen):
    """The plain paged store: one code per element, its parameters beside it."""
    P, Hkv, D = case["P"], case["Hkv"], case["D"]
    z = lambda *shape, dt=torch.uint8: torch.zeros(*shape, dtype=dt, device="cuda")  # noqa: E731
    st = {"k4": z(pages, P, Hkv, D), "v4": z(pages, P, Hkv, D), "kp": z(pages, P, Hkv, 2, dt=torch.float16), "vp": z(pages, P, Hkv, 2, dt=torch.float16)}
    rows = max(case["s"] + case["w"], 1)
    st |= {"k8": z(slots, rows, Hkv, D, dt=torch.int8), "v8": z(slots, rows, Hkv, D, dt=torch.int8), "p8": z(slots, rows, Hkv, 2, dt=torch.float16)}
    st["H"] = _hadamard(D, case["h"])
    if case.get("fmt") == "mixed":
        width, sigma = _allocation(gen, Hkv, D, 3)
        st |= {"width": width, "sigma": sigma, "kwid": _dev(np.tile(width, 2)).float(), "ksig": _dev(np.tile(sigma, 2))}
    return st


def _hadamard(D, h):
    H = torch.ones(1, 1, dtype=torch.float64)
    while H.shape[0] < h:
        H = torch.cat([torch.cat([H, H], 1), torch.cat([H, -H], 1)], 0)
    return torch.block_diag(*[H] * (D // h)).cuda()


def _cache(case, pages, slots, st):
    from int4_kv_cache_append_b200 import kv4
    mixed = case.get("fmt") == "mixed"
    geo = kv4.Geometry(1, case["Hq"], case["Hkv"], case["D"], case["P"], case["s"], case["w"], case["h"], slots, pages,
                       kv4.KV4_KEYS_MIXED if mixed else kv4.KV4_VALUES_INT4, 3 if mixed else 0, 3 if mixed else 0)
    cache = kv4.Cache(geo)
    if mixed:
        kv4.kv4_set_key_allocation(cache.handle, 0, st["width"], st["sigma"])
    return cache


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "table":
        # the base moves with the seed: another seed is another table
        c = dict(case, base=case["base"] * (1 + (seed % 1000) / 1000))
        s["table_case"] = c
        s["freq"], s["mult"] = _frequencies(c)
        if own:
            from int4_kv_cache_append_b200 import kv4
            kind = {"none": kv4.KV4_ROPE_SCALE_NONE, "linear": kv4.KV4_ROPE_SCALE_LINEAR, "ntk": kv4.KV4_ROPE_SCALE_NTK, "yarn": kv4.KV4_ROPE_SCALE_YARN,
                    "bands": kv4.KV4_ROPE_SCALE_BANDS}[c["scaling"]]
            s["rope"] = kv4.Rope(kv4.RopeGeometry(c["R"], c["max_pos"], kv4.KV4_ROPE_HALF, c["base"], kind, c["factor"], c["orig"], 1.0, 4.0, 32.0, 1.0))
        return s
    if op == "rope":
        T = case["T"]
        s |= _rope_inputs(gen, case, T, 32768)
        s["pos"] = torch.randint(0, 32768, (T,), generator=gen, device="cuda", dtype=torch.int32)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"].contiguous()), torch.empty_like(s["k"].contiguous())
        return s
    p = _append_plan(case) if op == "append" else _shared_plan(case)
    slots = len(p["lens"])
    s |= {"lens": _dev(p["lens"]), "table_pages": _dev(p["table"])}
    st = s["store"] = _store(case, p["pages"], slots, gen)
    if own:
        s["cache"] = _cache(case, p["pages"], slots, st)
    if op == "append":
        s |= {k: _dev(p[k]) for k in ("slot", "pos", "read_slot", "read_pos")}
        T, N = len(p["pos"]), len(p["read_pos"])
        s |= _rope_inputs(gen, case, T, int(p["lens"].max()))
        s["q_out"] = torch.empty_like(s["q"].contiguous())
        s["k_read"], s["v_read"] = (torch.empty(N, case["Hkv"], case["D"], dtype=BF16, device="cuda") for _ in range(2))
        fill_slot, fill_pos, limit = _dev(p["old_slot"]), _dev(p["old_pos"]), _dev(p["old"])
    else:
        s |= {"start": _dev(p["start"]), "prefix": _dev(p["prefix"]), "group": _dev(p["group"])}
        s["q"] = _randn(gen, slots, case["Hq"], case["D"])
        rows = np.zeros((case["groups"], max(p["per"])), np.int64)
        valid = np.zeros(rows.shape, bool)
        for g, n in enumerate(p["per"]):
            rows[g, :n], valid[g, :n] = np.arange(p["start"][g], p["start"][g + 1]), True
        s |= {"rows": _dev(rows), "row_valid": _dev(valid), "first_row": _dev(p["start"][:-1].astype(np.int64))}
        s["out"] = torch.empty(slots, case["Hq"], case["D"], dtype=BF16, device="cuda")
        # every sequence's own tokens, and the prefix of each group once per sequence's side cache
        whole = (p["prefix"] // case["P"] * case["P"])[p["group"]]
        whole[p["start"][:-1]] = 0
        b = np.concatenate([np.full(n - a, i, np.int32) for i, (a, n) in enumerate(zip(whole, p["lens"]))])
        q = np.concatenate([np.arange(a, n, dtype=np.int32) for a, n in zip(whole, p["lens"])])
        tail = [np.unique(np.concatenate([np.arange(min(case["s"], a)), np.arange(max(0, min(a, n - case["w"])), a)])).astype(np.int32) for a, n in zip(whole, p["lens"])]
        fill_slot = _dev(np.concatenate([b] + [np.full(len(t), i, np.int32) for i, t in enumerate(tail)]))
        fill_pos, limit = _dev(np.concatenate([q] + tail)), s["lens"]
        own_from = (p["prefix"] // case["P"] * case["P"])[p["group"]]
        s["max_prefix"], s["max_own"], s["own_from"] = int(p["prefix"].max()), int((p["lens"] - own_from).max()), _dev(own_from)
    # what the cache holds before the call: keys with a few strong channels, values, both from (slot's first owner, position)
    for lo in range(0, fill_pos.numel(), 32768):
        fs, fp = fill_slot[lo:lo + 32768], fill_pos[lo:lo + 32768]
        k, v = _context(case, s, fs, fp, seed)
        _plain_append(case, st, k.float(), v.float(), fs.long(), fp.long(), limit, s["table_pages"])
        if own:
            s["cache"].append(0, k, v, fs, fp, limit, s["table_pages"])
    return s


def _context(case, s, slot, pos, seed):
    """Keys and values by physical place, so that a shared position has the same values whoever writes it."""
    P = case["P"]
    page = s["table_pages"][slot.long(), (pos // P).long()].long() * P + (pos % P).long()
    i = torch.arange(case["Hkv"] * case["D"], device="cuda")
    out = []
    for salt in (1, 2):
        x = ((page[:, None] * 1000003 + i) * 7919 + seed * 104729 + salt * 15485863) & 0xFFFFFFFF
        for shift, mul in ((16, 0x45D9F3B), (16, 0x45D9F3B), (16, 1)):
            x = ((x ^ (x >> shift)) * mul) & 0xFFFFFFFF
        u = (x.double() + 0.5) / 4294967296.0
        z = torch.erfinv(2 * u - 1).float() * math.sqrt(2.0)
        if salt == 1:
            z = torch.where(i % 61 == 7, 8 * z, z)
        out.append(z.view(-1, case["Hkv"], case["D"]).to(BF16))
    return out


# ------------------------------------------------------------------ the plain forms

def _norm(x, w):
    if w is None:
        return x
    r = torch.rsqrt(x.double().square().mean(-1, keepdim=True) + 1e-6).float()
    return x * r * w.float()


def _rotate(x, cs, R, layout):
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = (x[..., :R // 2], x[..., R // 2:R]) if layout == "half" else (x[..., 0:R:2], x[..., 1:R:2])
    u, v = a * c - b * s, b * c + a * s
    y = torch.cat([u, v], -1) if layout == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([y, x[..., R:]], -1)


def _half_toward(x, up):
    """fp16 of x rounded toward +inf (up) or -inf."""
    h = x.half()
    off = (h.float() < x) if up else (h.float() > x)
    bits = h.view(torch.int16).int()
    away = (h > 0) == up
    step = torch.where(bits == 0, 1 if up else -32767, torch.where(bits == -32768, 1 if up else -32767, torch.where(away, bits + 1, bits - 1)))
    return torch.where(off, step.short().view(torch.float16), h)


def _int4(x, top=15):
    """Codes, and (scale or range, zero) as fp16."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    z = _half_toward(lo, False)
    by = x.new_full((), top)  # a tensor: a division by a plain number may be a product with its reciprocal
    s = _half_toward((hi - z.float()) / by if top == 15 else hi - z.float(), True)
    step = s.float() if top == 15 else s.float() / by
    c = torch.where(step > 0, ((x - z.float()) / step).round().clamp(0, top), torch.zeros_like(x))
    return c.to(torch.uint8), torch.cat([s, z], -1)


def _int8(x):
    s = _half_toward(x.abs().amax(-1, keepdim=True) / x.new_full((), 127), True)
    c = torch.where(s.float() > 0, (x / s.float()).round().clamp(-127, 127), torch.zeros_like(x))
    return c.to(torch.int8), s


def _mixed_keys(x, st):
    w, sg = st["kwid"], st["ksig"]
    s = _half_toward((torch.where(w > 0, x.abs() / sg, torch.zeros_like(x))).amax(-1, keepdim=True), True)
    c = torch.floor((x / (sg * s.float()) + 1) * torch.exp2(w - 1)).clamp(min=0).minimum(torch.exp2(w) - 1)
    return torch.where((w > 0) & (s.float() > 0), c, torch.zeros_like(c)).to(torch.uint8), torch.cat([s, torch.zeros_like(s)], -1)


def _plain_append(case, st, k, v, slot, pos, lens, pages):
    """Quantises k, v [T][Hkv][D] in 32 bits and writes the codes and parameters of each token."""
    at = (pages[slot, pos // case["P"]].long(), pos % case["P"])
    if case.get("fmt") == "mixed":
        (st["k4"][at], st["kp"][at]), (st["v4"][at], st["vp"][at]) = _mixed_keys(k, st), _int4(v, 7)
        return
    k = (k.double() @ st["H"].T).float()
    (st["k4"][at], st["kp"][at]), (st["v4"][at], st["vp"][at]) = _int4(k), _int4(v)
    if case["s"] + case["w"]:
        keep = (pos < case["s"]) | ((pos >= lens[slot] - case["w"]) & (case["w"] > 0))
        row = torch.where(pos < case["s"], pos, case["s"] + pos % max(case["w"], 1))
        at = (slot[keep], row[keep])
        (kc, ks), (vc, vs) = _int8(k[keep]), _int8(v[keep])
        st["k8"][at], st["v8"][at], st["p8"][at] = kc, vc, torch.cat([ks, vs], -1)


def _values4(case, st, page, off):
    """Keys (in the stored basis) and values of pages' rows, in 32 bits."""
    kp, vp = st["kp"][page, off].float(), st["vp"][page, off].float()
    kc, vc = st["k4"][page, off].float(), st["v4"][page, off].float()
    if case.get("fmt") == "mixed":
        k = torch.where(st["kwid"] > 0, kp[..., :1] * st["ksig"] * ((2 * kc + 1) * torch.exp2(-st["kwid"]) - 1), torch.zeros_like(kc))
        return k, vp[..., 1:] + vp[..., :1] / vp.new_full((), 7) * vc
    return kp[..., 1:] + kp[..., :1] * kc, vp[..., 1:] + vp[..., :1] * vc


def _values8(st, slot, row):
    p = st["p8"][slot, row].float()
    return st["k8"][slot, row].float() * p[..., :1], st["v8"][slot, row].float() * p[..., 1:]


def _run_append(s):
    case, st = s["case"], s["store"]
    cs = s["table"][s["pos"].long()]
    q = _rotate(_norm(s["q"].float(), s["qw"]), cs, case["R"], case["layout"])
    k = _rotate(_norm(s["k"].float(), s["kw"]), cs, case["R"], case["layout"])
    _plain_append(case, st, k, s["v"].float(), s["slot"].long(), s["pos"].long(), s["lens"], s["table_pages"])
    slot, pos = s["read_slot"].long(), s["read_pos"].long()
    k, v = _values4(case, st, s["table_pages"][slot, pos // case["P"]].long(), pos % case["P"])
    if case["s"] + case["w"]:
        L = s["lens"][slot].long()
        side = (pos < case["s"]) | (pos >= (L - case["w"]).clamp(min=case["s"]))
        row = torch.where(pos < case["s"], pos, case["s"] + pos % max(case["w"], 1)).clamp(max=case["s"] + case["w"] - 1)
        k8, v8 = _values8(st, slot, row)
        k, v = torch.where(side[:, None, None], k8, k), torch.where(side[:, None, None], v8, v)
    if case["fmt"] != "mixed":
        k = k @ st["H"].float() / case["h"]
    return q.to(BF16), k.to(BF16), v.to(BF16)


def _run_shared(s):
    """Scores of three blocks of keys (each group's shared pages, each sequence's own pages, its side rows), one softmax."""
    case, st = s["case"], s["store"]
    P, Hq, Hkv, D, w, ns = case["P"], case["Hq"], case["Hkv"], case["D"], case["w"], case["s"]
    B, G, n = s["lens"].numel(), case["groups"], s["rows"].shape[1]
    L, m_end = s["lens"].long(), (s["lens"].long() - w).clamp(min=ns)
    q = ((s["q"].float() @ st["H"].T.float()) / (case["h"] * math.sqrt(D))).view(B, Hkv, Hq // Hkv, D)

    pos = torch.arange(s["max_prefix"] // P * P, device="cuda")
    page = s["table_pages"][s["first_row"]][:, pos // P].long()
    pk, pv = _values4(case, st, page, (pos % P).expand(G, -1))
    qg = q[s["rows"]].permute(0, 2, 1, 3, 4).reshape(G, Hkv, n * Hq // Hkv, D)
    sp = (qg @ pk.permute(0, 2, 3, 1)).view(G, Hkv, n, Hq // Hkv, pos.numel()).permute(0, 2, 1, 3, 4)
    upto = torch.minimum(s["own_from"], m_end)
    sp = sp[s["row_valid"]].masked_fill(~((pos >= ns) & (pos < upto[:, None]))[:, None, None], -math.inf)

    opos = s["own_from"][:, None] + torch.arange(s["max_own"], device="cuda")
    live = (opos >= ns) & (opos < m_end[:, None])
    oc = opos.clamp(max=s["table_pages"].shape[1] * P - 1)
    ok, ov = _values4(case, st, s["table_pages"].gather(1, oc // P).long(), oc % P)
    so = (q @ ok.permute(0, 2, 3, 1)).masked_fill(~live[:, None, None], -math.inf)

    row = torch.arange(max(ns + w, 1), device="cuda")
    rec = (L[:, None] - 1) - (L[:, None] - 1 - (row - ns)) % max(w, 1)
    live = torch.where(row < ns, row < L[:, None], (rec >= ns) & (rec >= L[:, None] - w)) & (row < ns + w)
    k8, v8 = _values8(st, torch.arange(B, device="cuda")[:, None], row)
    s8 = (q @ k8.permute(0, 2, 3, 1)).masked_fill(~live[:, None, None], -math.inf)

    top = torch.cat([sp, so, s8], -1).amax(-1, keepdim=True)
    ep, eo, e8 = ((x - top).exp() for x in (sp, so, s8))
    total = ep.sum(-1, keepdim=True) + eo.sum(-1, keepdim=True) + e8.sum(-1, keepdim=True)
    padded = ep.new_zeros(G, n, *ep.shape[1:])
    padded[s["row_valid"]] = ep
    op = (padded.permute(0, 2, 1, 3, 4).reshape(G, Hkv, n * Hq // Hkv, ep.shape[-1]) @ pv.permute(0, 2, 1, 3)).view(G, Hkv, n, Hq // Hkv, D).permute(0, 2, 1, 3, 4)
    out = op[s["row_valid"]] + eo @ ov.permute(0, 2, 1, 3) + e8 @ v8.permute(0, 2, 1, 3)
    return (out / total).view(B, Hq, D).to(BF16)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        if op == "table":
            return s["rope"].build()
        if op == "rope":
            return s["rope"].apply(s["q"], s["k"], s["pos"], q_out=s["q_out"], k_out=s["k_out"])
        if op == "append":
            q = s["cache"].append_rope(0, s["rope"], s["q"], s["k"], s["v"], s["slot"], s["pos"], s["lens"], s["table_pages"], q_out=s["q_out"])
            return (q, *s["cache"].gather(0, s["read_slot"], s["read_pos"], s["table_pages"], s["lens"], k_out=s["k_read"], v_out=s["v_read"]))
        return s["cache"].decode_shared(0, s["q"], s["table_pages"], s["lens"], s["start"], s["prefix"], out=s["out"])
    if op == "table":
        return _table(s["freq"], s["mult"], case["max_pos"])
    if op == "rope":
        cs = s["table"][s["pos"].long()]
        return tuple(_rotate(_norm(x.float(), w), cs, case["R"], case["layout"]).to(BF16) for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])))
    return _run_append(s) if op == "append" else _run_shared(s)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_half(x, up):
    """x rounded to a multiple of its fp16 step, toward +inf or -inf, in 64 bits."""
    _, e = torch.frexp(x.abs().clamp(min=2.0 ** -14))
    step = torch.ldexp(torch.ones_like(x), e - 11)
    return (torch.ceil(x / step) if up else torch.floor(x / step)) * step


def _exact_rope(x, w, pos, freq_table, R, layout):
    """Every pair as a complex number times cos + i sin."""
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * w.double()
    turn = torch.view_as_complex(freq_table.double().contiguous())[pos.long()][:, None]
    pairs = torch.stack([x[..., :R // 2], x[..., R // 2:R]], -1) if layout == "half" else x[..., :R].unflatten(-1, (R // 2, 2))
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    out = x.clone()
    out[..., :R] = y.transpose(-1, -2).flatten(-2) if layout == "half" else y.flatten(-2)
    return out


def _exact_affine(x, top, half_of_step):
    zero = _exact_half(x.min(-1, keepdim=True).values, False)
    span = x.max(-1, keepdim=True).values - zero
    step = _exact_half(span / top, True) if half_of_step else _exact_half(span, True) / top
    return zero + step * ((x - zero) / step).round().clamp(0, top)


def _exact_symmetric(x):
    step = _exact_half(x.abs().max(-1, keepdim=True).values / 127, True)
    return step * (x / step).round().clamp(-127, 127)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "table":
        c = s["table_case"]
        freq, mult = _frequencies(c)
        turns = torch.outer(torch.arange(c["max_pos"], dtype=torch.float64), freq / (2 * math.pi))
        z = torch.polar(torch.full_like(turns, mult), 2 * math.pi * (turns - turns.round()))
        return torch.view_as_real(z)
    if op == "rope":
        return tuple(_exact_rope(x, w, s["pos"], s["table"], case["R"], case["layout"]) for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])))
    st, P, ns, w = s["store"], case["P"], case["s"], case["w"]
    if op == "append":
        q = _exact_rope(s["q"], s["qw"], s["pos"], s["table"], case["R"], case["layout"])
        k = _exact_rope(s["k"], s["kw"], s["pos"], s["table"], case["R"], case["layout"])
        v = s["v"].double()
        # the old positions as they are stored, the new ones by the definition
        p = _append_plan(case)
        slot, pos = s["read_slot"].long(), s["read_pos"].long()
        L, old = s["lens"].long()[slot], _dev(p["old"]).long()[slot]
        first = torch.cumsum(torch.cat([torch.zeros(1, dtype=torch.long), torch.from_numpy(np.bincount(p["slot"], minlength=case["B"]))]), 0).cuda()[slot]
        token = (first + pos - old).clamp(min=0)
        side = ((pos < ns) | (pos >= torch.maximum(L - w, torch.full_like(L, ns)))) if ns + w else torch.zeros_like(pos, dtype=torch.bool)
        if case["fmt"] == "mixed":
            wd, sg = st["kwid"].double(), st["ksig"].double()
            sc = _exact_half((k.abs() / sg * (wd > 0)).max(-1, keepdim=True).values, True)
            c = torch.minimum(torch.floor((k / (sg * sc) + 1) * 2 ** (wd - 1)).clamp(min=0), 2 ** wd - 1)
            k4, v4 = sc * sg * ((2 * c + 1) * 2 ** -wd - 1) * (wd > 0), _exact_affine(v, 7, False)
            k8, v8 = k4, v4
        else:
            k = k @ st["H"].T
            k4, v4, k8, v8 = _exact_affine(k, 15, True), _exact_affine(v, 15, True), _exact_symmetric(k), _exact_symmetric(v)
        m = side[:, None, None]
        kn, vn = torch.where(m, k8[token], k4[token]), torch.where(m, v8[token], v4[token])
        at = s["table_pages"][slot, pos // P].long(), pos % P
        (ks, kz), (vs, vz) = (st[n][at].double().split(1, -1) for n in ("kp", "vp"))
        if case["fmt"] == "mixed":
            ko, vo = ks * sg * ((2 * st["k4"][at] + 1) * 2 ** -wd - 1) * (wd > 0), vz + vs / 7 * st["v4"][at]
        else:
            ko, vo = kz + ks * st["k4"][at], vz + vs * st["v4"][at]
        m = (pos >= old)[:, None, None]
        # an old position that the call's window still covers keeps the side row its own append wrote
        row = torch.where(pos < ns, pos, ns + pos % max(w, 1)).clamp(max=max(ns + w - 1, 0))
        ks, vs = st["p8"][slot, row].double().split(1, -1)
        kr, vr = ks * st["k8"][slot, row], vs * st["v8"][slot, row]
        ko, vo = torch.where(side[:, None, None], kr, ko), torch.where(side[:, None, None], vr, vo)
        k, v = torch.where(m, kn, ko), torch.where(m, vn, vo)
        if case["fmt"] == "mixed":
            # bf16 values on a 7-step grid often lie on the border of two codes, where the format's own 32-bit division decides
            return q, k, None
        return q, k @ st["H"] / case["h"], v
    # one sequence at a time over its whole length, one softmax
    out = torch.empty(len(s["lens"]), case["Hq"], case["D"], dtype=torch.float64, device="cuda")
    for b, L in enumerate(s["lens"].tolist()):
        pos = torch.arange(L, device="cuda")
        page, off = s["table_pages"][b, pos // P].long(), pos % P
        k4 = st["kp"][page, off].double()
        k = k4[..., 1:] + k4[..., :1] * st["k4"][page, off]
        v4 = st["vp"][page, off].double()
        v = v4[..., 1:] + v4[..., :1] * st["v4"][page, off]
        near = torch.cat([pos[:min(ns, L)], pos[max(min(ns, L), L - w):]])
        row = torch.where(near < ns, near, ns + near % max(w, 1))
        k[near] = st["k8"][b, row] * st["p8"][b, row][..., :1].double()
        v[near] = st["v8"][b, row] * st["p8"][b, row][..., 1:].double()
        q = (s["q"][b].double() @ st["H"].T / case["h"]).view(case["Hkv"], -1, case["D"])
        a = torch.softmax(torch.einsum("hgd,thd->hgt", q, k) / math.sqrt(case["D"]), -1)
        out[b] = torch.einsum("hgt,thd->hgd", a, v).reshape(case["Hq"], case["D"])
    return out
