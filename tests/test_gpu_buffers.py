"""Buffers that the cache objects make themselves: workspaces, and outputs on a given stream."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv4():
    from int4_kv_cache_append_b200 import kv4
    return kv4


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def small(kv4, B=64, L=40, cls="Cache", Hkv=2, D=64):
    """A cache of B sequences of L random tokens, and what the calls take."""
    P = 16
    pages = -(-L // P)
    cache = getattr(kv4, cls)(kv4.Geometry(1, 2 * Hkv, Hkv, D, P, 0, 0, 1, B, B * pages))
    table = i32(np.arange(B * pages).reshape(B, pages))
    b, p = np.repeat(np.arange(B), L), np.tile(np.arange(L), B)
    K, V = (torch.randn(B * L, Hkv, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    lens = i32(np.full(B, L))
    if cls == "Cache":
        cache.append(0, K, V, i32(b), i32(p), lens, table)
    else:
        cache.append(0, K, V, i32(b), i32(p), table)
    return cache, table, lens, torch.randn(B, 2 * Hkv, D, device="cuda", dtype=torch.bfloat16)


def groups(B, n):
    return i32(np.linspace(0, B, n + 1).round()), i32(np.zeros(n))


def test_many_batch_shapes_keep_memory_bounded(kv4):
    cache, table, lens, q = small(kv4)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for B in range(1, 65, 3):
        for n in range(1, B + 1, 5):
            cache.decode_shared(0, q[:B], table, lens[:B], *groups(B, n))
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() - before <= 2 * kv4.kv4_decode_shared_workspace_bytes(cache.handle, 64, 64) + (1 << 20)
    cache.close()
    assert torch.cuda.memory_allocated() - before <= 1 << 20


@pytest.mark.parametrize("cls,shared", [("Cache", False), ("Cache", True), ("BF16Cache", False)])
def test_a_captured_call_keeps_its_workspace(kv4, cls, shared):
    """A larger call after the capture takes a larger workspace; the replay then still writes to memory of
    its own."""
    cache, table, lens, q = small(kv4, cls=cls, B=256)

    def call(B, out=None):
        if shared:
            return cache.decode_shared(0, q[:B], table, lens[:B], *fixed[B], out=out)
        return cache.decode(0, q[:B], table, lens[:B], out=out)

    fixed = {B: groups(B, 1) for B in (3, 256)}
    want = call(3).clone()
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(3, out)
    call(256)
    torch.cuda.synchronize()
    # takes every block that the allocator has free
    free = torch.cuda.memory_reserved() - torch.cuda.memory_allocated()
    sizes = [s for s in (64 << 20, 16 << 20, 4 << 20, 2 << 20, 1 << 20, 1 << 18) for _ in range(min(32, free // s + 1))]
    others = [torch.full((s,), 77, dtype=torch.uint8, device="cuda") for s in sizes]
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(bool((x == 77).all()) for x in others)


def test_calls_on_two_streams_have_their_own_workspaces(kv4):
    cache, table, lens, q = small(kv4, L=1000)
    gs = groups(64, 8)
    want = [cache.decode(0, q, table, lens), cache.decode_shared(0, q, table, lens, *gs)]
    torch.cuda.synchronize()
    outs = [[torch.empty_like(x) for x in want] for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in outs]
    for _ in range(4):
        for st, o in zip(streams, outs):
            cache.decode(0, q, table, lens, out=o[0], stream=st)
            cache.decode_shared(0, q, table, lens, *gs, out=o[1], stream=st.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for o in outs for x, y in zip(o, want))
