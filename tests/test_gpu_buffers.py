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


def calls(kv4):
    """name -> call(stream) that makes its own output."""
    cache, table, lens, q = small(kv4, L=200)
    bf = small(kv4, L=200, cls="BF16Cache")
    rope = kv4.Rope(kv4.RopeGeometry(64, 256))
    T = 64
    x = torch.randn(T, 8, 64, device="cuda", dtype=torch.bfloat16)
    pos, slot = i32(np.arange(T) + 100), i32(np.arange(T))
    gs = groups(64, 4)
    return {
        "table": lambda st: kv4.Rope(kv4.RopeGeometry(64, 256), stream=st).table,
        "rope-q": lambda st: rope.apply(x[:, :4], None, pos, stream=st)[0],
        "rope-k": lambda st: rope.apply(None, x[:, 4:6], pos, stream=st)[1],
        "append": lambda st: cache.append_rope(0, rope, x[:, :4], x[:, 4:6], x[:, 6:], slot, pos, lens, table, stream=st),
        "gather-k": lambda st: cache.gather(0, slot, pos, table, lens, stream=st)[0],
        "gather-v": lambda st: cache.gather(0, slot, pos, table, lens, stream=st)[1],
        "decode": lambda st: cache.decode(0, q, table, lens, stream=st),
        "shared": lambda st: cache.decode_shared(0, q, table, lens, *gs, stream=st),
        "bf16": lambda st: bf[0].decode(0, bf[3], *bf[1:3], stream=st),
    }


NAMES = ("table", "rope-q", "rope-k", "append", "gather-k", "gather-v", "decode", "shared", "bf16")
DELAY = 100_000_000  # cycles


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_output_on_another_stream_is_not_pending_memory(kv4, name, raw):
    """Memory that the current stream still has writes pending for is not handed to a call on another."""
    call = calls(kv4)[name]
    st = torch.cuda.Stream()
    want = call(None).clone()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.empty_like(want) for _ in range(64)]
    torch.cuda._sleep(DELAY)
    for x in held:
        x.fill_(7)
    del held, x
    got = call(st.cuda_stream if raw else st)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_output_on_another_stream_lives_until_the_current_one_has_read_it(kv4, name):
    call = calls(kv4)[name]
    st = torch.cuda.Stream()
    want = call(None).clone()
    kept = torch.empty_like(want)
    torch.cuda.synchronize()
    got = call(st)
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda._sleep(DELAY)
    kept.copy_(got)
    del got
    with torch.cuda.stream(st):  # what st allocates next
        for _ in range(64):
            torch.empty_like(want).fill_(7)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)
