"""ctypes binding of libkv4.so (C ABI in include/kv4.h).

Each function has the name of the C entry point it wraps and only marshals arguments: torch
CUDA tensors become device pointers, streams become cudaStream_t handles, and a non-OK status
raises ``KV4Error``.  All computation happens in the CUDA kernels of libkv4.so; there is no
fallback path, and importing this module fails loudly when the library is missing.

``Cache`` and ``BF16Cache`` are conveniences that allocate the caller-owned buffers with torch
(PyTorch is used here for device memory and streams only).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkv4.so")

(KV4_OK, KV4_ERR_INVALID_ARG, KV4_ERR_UNSUPPORTED, KV4_ERR_WORKSPACE, KV4_ERR_CUDA, KV4_ERR_DEVICE,
 KV4_ERR_NO_ALLOCATION) = range(7)
KV4_F32, KV4_BF16, KV4_F16 = 0, 1, 2
KV4_DEVERR_PAGE_RANGE, KV4_DEVERR_WAIT_LIMIT, KV4_DEVERR_LENGTH, KV4_DEVERR_RANGE, KV4_DEVERR_RECORD = 0x1, 0x2, 0x4, 0x8, 0x10
KV4_DEVERR_GROUP = 0x20

# every entry point declared in include/kv4.h
SYMBOLS = (
    "kv4_query_sizes", "kv4_cache_init", "kv4_cache_destroy", "kv4_append", "kv4_decode_workspace_bytes",
    "kv4_decode_attn", "kv4_decode_attn_static", "kv4_set_decode_overlap", "kv4_debug_force_wait_timeout",
    "kv4_set_rotation_signs", "kv4_set_value_rotation", "kv4_bf16_query_sizes", "kv4_bf16_cache_init",
    "kv4_bf16_append", "kv4_bf16_decode_workspace_bytes", "kv4_bf16_decode_attn", "kv4_get_device_error",
    "kv4_launch_count", "kv4_status_string", "kv4_version", "kv4_allocate_key_bits", "kv4_set_key_allocation",
    "kv4_get_key_allocation", "kv4_debug_mixed_row_copies", "kv4_rope_table", "kv4_rope", "kv4_append_rope",
    "kv4_gather", "kv4_decode_shared_workspace_bytes", "kv4_decode_attn_shared",
)


class KV4Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")
        self.status = status


KV4_VALUES_INT4, KV4_VALUES_BF16, KV4_KEYS_MIXED = 0, 1, 2


class kv4_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "num_layers", "num_q_heads", "num_kv_heads", "head_dim", "page_size", "num_sinks",
        "recent_window", "hadamard_block", "max_seqs", "max_pages", "value_format", "key_bits", "value_bits")]


KV4_ROPE_HALF, KV4_ROPE_INTERLEAVED = 0, 1
(KV4_ROPE_SCALE_NONE, KV4_ROPE_SCALE_LINEAR, KV4_ROPE_SCALE_NTK, KV4_ROPE_SCALE_YARN,
 KV4_ROPE_SCALE_BANDS) = range(5)


class kv4_rope_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("rotary_dim", "max_pos", "scaling", "original_max_pos")] + [
        (n, ctypes.c_double) for n in ("base", "factor", "low_freq_factor", "high_freq_factor", "beta_fast",
                                       "beta_slow", "attention_factor")]


class kv4_rope_params(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("max_pos", ctypes.c_int), ("rotary_dim", ctypes.c_int),
                ("layout", ctypes.c_int), ("weight_dtype", ctypes.c_int), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing; build it with `python -m int4_kv_cache_append_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, S, U = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint64
    cfgp = ctypes.POINTER(kv4_config)
    LL, ropep = ctypes.c_int64, ctypes.POINTER(kv4_rope_params)
    i32p = ctypes.c_void_p
    sig = {
        "kv4_query_sizes": (I, [cfgp, ctypes.POINTER(S), ctypes.POINTER(S)]),
        "kv4_cache_init": (I, [cfgp, P, P, ctypes.POINTER(P)]),
        "kv4_cache_destroy": (None, [P]),
        "kv4_append": (I, [P, I, I, P, I, P, I, i32p, i32p, i32p, i32p, I, P]),
        "kv4_decode_workspace_bytes": (I, [P, I, ctypes.POINTER(S)]),
        "kv4_decode_attn": (I, [P, I, I, P, I, i32p, I, i32p, I, P, P, P, S, P]),
        "kv4_decode_attn_static": (I, [P, I, I, P, I, i32p, I, i32p, I, P, P, P]),
        "kv4_set_decode_overlap": (I, [P, I]),
        "kv4_debug_force_wait_timeout": (I, [P, I]),
        "kv4_debug_mixed_row_copies": (I, [P, I]),
        "kv4_set_rotation_signs": (I, [P, P]),
        "kv4_set_value_rotation": (I, [P, I]),
        "kv4_bf16_query_sizes": (I, [cfgp, ctypes.POINTER(S)]),
        "kv4_bf16_cache_init": (I, [cfgp, P, ctypes.POINTER(P)]),
        "kv4_bf16_append": (I, [P, I, I, P, I, P, I, i32p, i32p, i32p, I, P]),
        "kv4_bf16_decode_workspace_bytes": (I, [P, I, ctypes.POINTER(S)]),
        "kv4_bf16_decode_attn": (I, [P, I, I, P, I, i32p, I, i32p, I, P, P, P, S, P]),
        "kv4_get_device_error": (I, [ctypes.POINTER(ctypes.c_uint32)]),
        "kv4_launch_count": (U, []),
        "kv4_status_string": (ctypes.c_char_p, [I]),
        "kv4_version": (I, []),
        "kv4_allocate_key_bits": (I, [P, I, I, P, I, P]),
        "kv4_set_key_allocation": (I, [P, I, P, P, P]),
        "kv4_get_key_allocation": (I, [P, I, P, P, P]),
        "kv4_rope_table": (I, [ctypes.POINTER(kv4_rope_config), P, P]),
        "kv4_rope": (I, [ropep, I, I, I, I, P, I, LL, P, I, LL, i32p, P, I, LL, P, I, LL, P]),
        "kv4_append_rope": (I, [P, I, I, ropep, P, I, LL, P, I, LL, P, I, LL, i32p, i32p, i32p, i32p, I, P, I, LL, P]),
        "kv4_decode_shared_workspace_bytes": (I, [P, I, I, ctypes.POINTER(S)]),
        "kv4_decode_attn_shared": (I, [P, I, I, P, I, i32p, I, i32p, I, i32p, i32p, I, P, I, P, P, S, P]),
        "kv4_gather": (I, [P, I, I, i32p, i32p, i32p, i32p, I, P, P, I, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


lib = _load()


def status_string(status: int) -> str:
    return lib.kv4_status_string(status).decode()


def _check(fn: str, status: int) -> None:
    if status != KV4_OK:
        raise KV4Error(fn, status)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor expected")
    return t.data_ptr()


# A call's checks are a large part of a small call's time: sizes and strides are read once, devices as
# integers, and the current stream as a raw handle where torch offers it.
def _rows(t, shape, what: str):
    """(pointer, kv4_dtype, elements between tokens) of a tensor of shape [T][heads][D] whose heads are
    contiguous in a token."""
    if not t.is_cuda or len(shape) != 3:
        raise ValueError(f"{what}: device tensor [T][heads][D] expected")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what}: float32, bfloat16 or float16 expected, got {t.dtype}")
    T, H, D = shape
    st, sh, sd = t.stride()
    if (sd != 1 and D > 1) or (sh != D and H > 1):
        raise ValueError(f"{what}: the heads of a token must be contiguous")
    return t.data_ptr(), code, st if T > 1 else H * D


def _i32(t, what: str):
    if t is None:
        return None
    if t.dtype is not torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what}: contiguous int32 device tensor expected, got {t.dtype} on {t.device}")
    return t.data_ptr()


def _on_current_device(*tensors) -> None:
    """The library launches on the current device."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensor on {t.device}, but the current device is cuda:{dev}")


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_NO_STREAM = contextlib.nullcontext()


def _on_stream(stream):
    """Context in which torch allocates for work on the stream (the current one: None)."""
    if stream is None:
        return _NO_STREAM
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _new(shape, dtype, device, stream):
    """Tensor that a call on the stream writes.  It belongs to that stream, so that its memory has no work of
    another one pending; the current stream may read it too (once it has waited for the call) before it
    is used again."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on_stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


_DTYPES = {torch.float32: KV4_F32, torch.bfloat16: KV4_BF16, torch.float16: KV4_F16}


def dtype_code(t: torch.Tensor) -> int:
    return _DTYPES[t.dtype]


# ------------------------------------------------------------------------ C entry points

def kv4_query_sizes(cfg: kv4_config) -> tuple[int, int]:
    pool, side = ctypes.c_size_t(), ctypes.c_size_t()
    _check("kv4_query_sizes", lib.kv4_query_sizes(ctypes.byref(cfg), ctypes.byref(pool), ctypes.byref(side)))
    return pool.value, side.value


def kv4_cache_init(cfg: kv4_config, page_pool, side_cache) -> int:
    h = ctypes.c_void_p()
    _check("kv4_cache_init", lib.kv4_cache_init(ctypes.byref(cfg), _ptr(page_pool), _ptr(side_cache), ctypes.byref(h)))
    return h.value


def kv4_cache_destroy(handle: int) -> None:
    lib.kv4_cache_destroy(handle)


def kv4_append(handle, layer, T, K, k_dtype, V, v_dtype, seq_slot, pos, lens_after, page_table, stride, stream=None):
    _check("kv4_append", lib.kv4_append(handle, layer, T, _ptr(K), k_dtype, _ptr(V), v_dtype, _ptr(seq_slot), _ptr(pos),
                                        _ptr(lens_after), _ptr(page_table), stride, _stream(stream)))


def kv4_decode_workspace_bytes(handle, B) -> int:
    n = ctypes.c_size_t()
    _check("kv4_decode_workspace_bytes", lib.kv4_decode_workspace_bytes(handle, B, ctypes.byref(n)))
    return n.value


def kv4_decode_attn(handle, layer, B, q, q_dtype, page_table, stride, lens, max_len_hint, out, lse, workspace,
                    ws_bytes, stream=None):
    _check("kv4_decode_attn", lib.kv4_decode_attn(handle, layer, B, _ptr(q), q_dtype, _ptr(page_table), stride,
                                                  _ptr(lens), max_len_hint, _ptr(out), _ptr(lse), _ptr(workspace),
                                                  ws_bytes, _stream(stream)))


def kv4_decode_attn_static(handle, layer, B, q, q_dtype, page_table, stride, lens, max_len_hint, out, lse,
                           stream=None):
    """kv4_decode_attn without a workspace argument, for callers that cannot allocate device
    memory: the split partials use the library's static per-GPU scratch array
    (KV4_STATIC_SCRATCH_BYTES = 16 MiB); larger batches are rejected with KV4_ERR_WORKSPACE.
    Calls that overlap on one GPU share that array and must not run concurrently."""
    _check("kv4_decode_attn_static", lib.kv4_decode_attn_static(handle, layer, B, _ptr(q), q_dtype, _ptr(page_table),
                                                                stride, _ptr(lens), max_len_hint, _ptr(out), _ptr(lse),
                                                                _stream(stream)))


KV4_STATIC_SCRATCH_BYTES = 16 << 20


def kv4_set_rotation_signs(handle, sign_bits):
    """Randomised-sign rotation: sign_bits is a sequence of uint32 words (bit d negates dim d before
    the Hadamard), or None to clear it.  Set before the first append."""
    if sign_bits is None:
        _check("kv4_set_rotation_signs", lib.kv4_set_rotation_signs(handle, None))
        return
    arr = (ctypes.c_uint32 * 4)(*[int(x) & 0xFFFFFFFF for x in list(sign_bits)[:4]])
    _check("kv4_set_rotation_signs", lib.kv4_set_rotation_signs(handle, ctypes.cast(arr, ctypes.c_void_p)))


def kv4_set_value_rotation(handle, enable: bool):
    """Store values rotated like the keys; outputs are rotated back.  Set before the first append."""
    _check("kv4_set_value_rotation", lib.kv4_set_value_rotation(handle, 1 if enable else 0))


def kv4_set_decode_overlap(handle, enable: bool):
    """With enable, the decode kernel builds its schedule from lens and page_table while the
    preceding kernel on the stream runs (they must not be written by that kernel)."""
    _check("kv4_set_decode_overlap", lib.kv4_set_decode_overlap(handle, 1 if enable else 0))


def kv4_debug_mixed_row_copies(handle, enable: bool):
    """Test hook (mixed bit-width keys): padded key rows by one bulk copy per row instead of the
    tensor copy, the path taken when the driver's tensor-map encoder is not available."""
    _check("kv4_debug_mixed_row_copies", lib.kv4_debug_mixed_row_copies(handle, 1 if enable else 0))


def kv4_debug_force_wait_timeout(handle, enable: bool):
    """Test hook: with enable, the decode's bounded waits are made to run out (1 ms limit), so the
    device-side failure path runs and KV4_DEVERR_WAIT_LIMIT is reported.  Off by default."""
    _check("kv4_debug_force_wait_timeout", lib.kv4_debug_force_wait_timeout(handle, 1 if enable else 0))


def kv4_allocate_key_bits(handle, layer, T, K, k_dtype, stream=None):
    """Mixed bit-width keys: score the T keys K [T][Hkv][D] per RoPE block and allocate the layer's
    key bits on the device."""
    _check("kv4_allocate_key_bits", lib.kv4_allocate_key_bits(handle, layer, T, _ptr(K), k_dtype, _stream(stream)))


def kv4_set_key_allocation(handle, layer, widths, sigma, stream=None):
    """Mixed bit-width keys: set a layer's allocation from host arrays widths uint8 [Hkv][D/2] and
    sigma float32 [Hkv][D/2] (NumPy)."""
    import numpy as np
    w = np.ascontiguousarray(widths, np.uint8)
    sg = np.ascontiguousarray(sigma, np.float32)
    _check("kv4_set_key_allocation", lib.kv4_set_key_allocation(handle, layer, w.ctypes.data_as(ctypes.c_void_p),
                                                                sg.ctypes.data_as(ctypes.c_void_p), _stream(stream)))


def kv4_get_key_allocation(handle, layer, Hkv, D, stream=None):
    """Mixed bit-width keys: (widths uint8 [Hkv][D/2], sigma float32 [Hkv][D/2]) of a layer."""
    import numpy as np
    w = np.zeros((Hkv, D // 2), np.uint8)
    sg = np.zeros((Hkv, D // 2), np.float32)
    _check("kv4_get_key_allocation", lib.kv4_get_key_allocation(handle, layer, w.ctypes.data_as(ctypes.c_void_p),
                                                                sg.ctypes.data_as(ctypes.c_void_p), _stream(stream)))
    return w, sg


def kv4_rope_table(cfg: kv4_rope_config, table, stream=None):
    """Write the cos/sin table fp32 [max_pos][rotary_dim / 2][2] of a rotary configuration."""
    _check("kv4_rope_table", lib.kv4_rope_table(ctypes.byref(cfg), _ptr(table), _stream(stream)))


def kv4_rope(params: kv4_rope_params, q, k, pos, q_out, k_out, stream=None):
    """Norm and rotate T tokens' queries [T][Hq][D] and keys [T][Hkv][D] (either may be None)."""
    if q is None and k is None:
        raise ValueError("q or k expected")
    rows, heads, tokens, size = [], [], None, None
    for src, dst, what in ((q, q_out, "q"), (k, k_out, "k")):
        if src is None:
            if dst is not None:
                raise ValueError(f"{what}_out without {what}")
            rows += (None, 0, 0), (None, 0, 0)
            heads.append(0)
            continue
        shape = src.shape
        if dst is None or dst.shape != shape:
            raise ValueError(f"{what}_out: the shape of its input expected")
        rows += _rows(src, shape, what), _rows(dst, shape, what + "_out")
        if tokens is not None and (tokens != shape[0] or size != shape[2]):
            raise ValueError("q and k differ in tokens or head size")
        tokens, _, size = shape
        heads.append(shape[1])
    if pos.numel() != tokens:
        raise ValueError("pos: one position per token expected")
    _on_current_device(q, k, pos, q_out, k_out)
    _check("kv4_rope", lib.kv4_rope(ctypes.byref(params), tokens, heads[0], heads[1], size, *rows[0], *rows[2],
                                    _i32(pos, "pos"), *rows[1], *rows[3], _stream(stream)))


def kv4_append_rope(handle, layer, params: kv4_rope_params, q, K, V, seq_slot, pos, lens_after, page_table, stride,
                    q_out, stream=None):
    """Append keys and values [T][Hkv][D], the keys normed and rotated on the way; q_out receives the
    normed and rotated queries (q and q_out None: append only)."""
    T, shape = seq_slot.numel(), K.shape
    if q is None:
        rq = ro = (None, 0, 0)
        if q_out is not None:
            raise ValueError("q_out without q")
    else:
        qs = q.shape
        if q_out is None or q_out.shape != qs or qs[0] != T:
            raise ValueError("q and q_out of one shape, with the tokens of seq_slot, expected")
        rq, ro = _rows(q, qs, "q"), _rows(q_out, qs, "q_out")
    if pos.numel() != T or shape[0] != T or shape != V.shape:
        raise ValueError("q, K, V, seq_slot and pos must have the same tokens")
    _on_current_device(q, K, V, seq_slot, pos, lens_after, page_table, q_out)
    _check("kv4_append_rope", lib.kv4_append_rope(handle, layer, T, ctypes.byref(params), *rq, *_rows(K, shape, "K"),
                                                  *_rows(V, shape, "V"), _i32(seq_slot, "seq_slot"), _i32(pos, "pos"),
                                                  _i32(lens_after, "lens_after"), _i32(page_table, "page_table"), stride,
                                                  *ro, _stream(stream)))


def kv4_gather(handle, layer, T, seq_slot, pos, lens, page_table, stride, K_out, V_out, out_dtype, stream=None):
    """Read T cached positions back as dense keys and values [T][Hkv][D] in their original basis."""
    _on_current_device(seq_slot, pos, lens, page_table, K_out, V_out)
    _check("kv4_gather", lib.kv4_gather(handle, layer, T, _i32(seq_slot, "seq_slot"), _i32(pos, "pos"), _i32(lens, "lens"),
                                        _i32(page_table, "page_table"), stride, _ptr(K_out), _ptr(V_out), out_dtype,
                                        _stream(stream)))


def kv4_decode_shared_workspace_bytes(handle, B, n_groups) -> int:
    n = ctypes.c_size_t()
    _check("kv4_decode_shared_workspace_bytes", lib.kv4_decode_shared_workspace_bytes(handle, B, n_groups, ctypes.byref(n)))
    return n.value


def kv4_decode_attn_shared(handle, layer, B, q, q_dtype, page_table, stride, lens, n_groups, group_start, prefix_len,
                           max_len_hint, out, out_dtype, lse, workspace, ws_bytes, stream=None):
    """kv4_decode_attn for groups of batch rows that share a prefix, each read once per group."""
    _on_current_device(q, page_table, lens, group_start, prefix_len, out, lse, workspace)
    _check("kv4_decode_attn_shared", lib.kv4_decode_attn_shared(
        handle, layer, B, _ptr(q), q_dtype, _i32(page_table, "page_table"), stride, _i32(lens, "lens"), n_groups,
        _i32(group_start, "group_start"), _i32(prefix_len, "prefix_len"), max_len_hint, _ptr(out), out_dtype, _ptr(lse),
        _ptr(workspace), ws_bytes, _stream(stream)))


def kv4_bf16_query_sizes(cfg: kv4_config) -> int:
    pool = ctypes.c_size_t()
    _check("kv4_bf16_query_sizes", lib.kv4_bf16_query_sizes(ctypes.byref(cfg), ctypes.byref(pool)))
    return pool.value


def kv4_bf16_cache_init(cfg: kv4_config, page_pool) -> int:
    h = ctypes.c_void_p()
    _check("kv4_bf16_cache_init", lib.kv4_bf16_cache_init(ctypes.byref(cfg), _ptr(page_pool), ctypes.byref(h)))
    return h.value


def kv4_bf16_append(handle, layer, T, K, k_dtype, V, v_dtype, seq_slot, pos, page_table, stride, stream=None):
    _check("kv4_bf16_append", lib.kv4_bf16_append(handle, layer, T, _ptr(K), k_dtype, _ptr(V), v_dtype, _ptr(seq_slot),
                                                  _ptr(pos), _ptr(page_table), stride, _stream(stream)))


def kv4_bf16_decode_workspace_bytes(handle, B) -> int:
    n = ctypes.c_size_t()
    _check("kv4_bf16_decode_workspace_bytes", lib.kv4_bf16_decode_workspace_bytes(handle, B, ctypes.byref(n)))
    return n.value


def kv4_bf16_decode_attn(handle, layer, B, q, q_dtype, page_table, stride, lens, max_len_hint, out, lse, workspace,
                         ws_bytes, stream=None):
    _check("kv4_bf16_decode_attn", lib.kv4_bf16_decode_attn(handle, layer, B, _ptr(q), q_dtype, _ptr(page_table), stride,
                                                            _ptr(lens), max_len_hint, _ptr(out), _ptr(lse),
                                                            _ptr(workspace), ws_bytes, _stream(stream)))


def kv4_get_device_error() -> int:
    v = ctypes.c_uint32()
    _check("kv4_get_device_error", lib.kv4_get_device_error(ctypes.byref(v)))
    return v.value


def kv4_launch_count() -> int:
    return int(lib.kv4_launch_count())


def kv4_version() -> int:
    return int(lib.kv4_version())


# ------------------------------------------------------------------------ conveniences

@dataclass
class Geometry:
    num_layers: int
    num_q_heads: int
    num_kv_heads: int
    head_dim: int
    page_size: int
    num_sinks: int
    recent_window: int
    hadamard_block: int
    max_seqs: int
    max_pages: int
    value_format: int = KV4_VALUES_INT4
    key_bits: int = 0      # KV4_KEYS_MIXED only
    value_bits: int = 0    # KV4_KEYS_MIXED only

    def c(self) -> kv4_config:
        return kv4_config(self.num_layers, self.num_q_heads, self.num_kv_heads, self.head_dim, self.page_size,
                          self.num_sinks, self.recent_window, self.hadamard_block, self.max_seqs, self.max_pages,
                          self.value_format, self.key_bits, self.value_bits)

    def page_bytes(self) -> int:
        """Bytes of one page (all KV heads) of one layer."""
        D, P, H = self.head_dim, self.page_size, self.num_kv_heads
        if self.value_format == KV4_KEYS_MIXED:
            return H * P * ((self.key_bits + self.value_bits) * D // 8 + 8)
        return H * P * (D // 2 + 4 + 2 * D if self.value_format == KV4_VALUES_BF16 else D + 8)


@dataclass
class RopeGeometry:
    rotary_dim: int
    max_pos: int
    layout: int = KV4_ROPE_HALF
    base: float = 10000.0
    scaling: int = KV4_ROPE_SCALE_NONE
    factor: float = 1.0
    original_max_pos: int = 0
    low_freq_factor: float = 1.0
    high_freq_factor: float = 4.0
    beta_fast: float = 32.0
    beta_slow: float = 1.0
    attention_factor: float = 0.0

    def c(self) -> kv4_rope_config:
        return kv4_rope_config(self.rotary_dim, self.max_pos, self.scaling, self.original_max_pos, self.base, self.factor,
                               self.low_freq_factor, self.high_freq_factor, self.beta_fast, self.beta_slow,
                               self.attention_factor)


class Rope:
    """A rotary embedding with its torch-allocated table and the per-head norm weights (None: no
    norm); the weights are [head_dim] tensors of one type that the caller keeps."""

    def __init__(self, geo: RopeGeometry, q_weight=None, k_weight=None, eps: float = 1e-6, device="cuda", stream=None):
        for w in (q_weight, k_weight):
            if w is not None and (w.dim() != 1 or not w.is_contiguous() or w.dtype not in _DTYPES):
                raise ValueError("norm weights: contiguous [head_dim] tensors expected")
        if q_weight is not None and k_weight is not None and (q_weight.dtype, q_weight.shape) != (k_weight.dtype, k_weight.shape):
            raise ValueError("norm weights: one type and size expected")
        self.geo, self.q_weight, self.k_weight, self.eps = geo, q_weight, k_weight, eps
        self.cfg = geo.c()
        self.table = _new((max(geo.max_pos, 0), max(geo.rotary_dim, 0) // 2, 2), torch.float32, device, stream)
        self.build(stream)
        w = q_weight if q_weight is not None else k_weight
        self.params = kv4_rope_params(self.table.data_ptr(), geo.max_pos, geo.rotary_dim, geo.layout,
                                      dtype_code(w) if w is not None else KV4_F32, _ptr(q_weight), _ptr(k_weight), eps)

    def build(self, stream=None) -> torch.Tensor:
        """(Re)write the table on the stream; other streams must wait for it."""
        _on_current_device(self.table, self.q_weight, self.k_weight)
        kv4_rope_table(self.cfg, self.table, stream)
        return self.table

    def check_head_dim(self, D: int) -> None:
        _on_current_device(self.table)
        for w in (self.q_weight, self.k_weight):
            if w is not None and w.numel() != D:
                raise ValueError(f"norm weights of {w.numel()} elements for heads of {D}")

    def apply(self, q, k, pos, q_out=None, k_out=None, stream=None):
        """Normed and rotated (q, k); new tensors of the inputs' types unless outputs are given."""
        x = q if q is not None else k
        if x is not None:
            self.check_head_dim(x.shape[-1])
        if q is not None and q_out is None:
            q_out = _new(q.shape, q.dtype, q.device, stream)
        if k is not None and k_out is None:
            k_out = _new(k.shape, k.dtype, k.device, stream)
        kv4_rope(self.params, q, k, pos, q_out, k_out, stream)
        return q_out, k_out


class _Workspaces:
    """Device buffers of the calls that are given none: one for each stream, since calls on one stream do
    not overlap, grown by half at least when a call needs more (so that a batch whose shape changes every
    step settles on one).  During a capture a call gets a buffer from the graph's own memory instead: it
    lives as long as the graph, whatever later calls need."""

    def __init__(self):
        self._bufs = {}  # stream -> (what the last call asked for, its buffer)

    def get(self, size, args, device, stream=None) -> torch.Tensor:
        """A buffer of at least size(*args) bytes for work on the stream."""
        if stream is not None:
            with _on_stream(stream):
                return self.get(size, args, device)
        if torch.cuda.is_current_stream_capturing():
            return torch.empty(size(*args), dtype=torch.uint8, device=device)
        key = _stream(None)
        last, buf = self._bufs.get(key, (None, None))
        if last == (size, args):
            return buf
        n = size(*args)
        if buf is None or buf.numel() < n:
            n = n if buf is None else max(n, buf.numel() * 3 // 2)
            self._bufs.pop(key, None)
            del buf
            buf = torch.empty(n, dtype=torch.uint8, device=device)
        self._bufs[key] = (size, args), buf
        return buf

    def clear(self) -> None:
        self._bufs.clear()


class _RopeCacheMixin:
    """kv4_append_rope and kv4_gather of a cache object (both kinds of handle)."""

    def append_rope(self, layer, rope: Rope, q, K, V, seq_slot, pos, lens_after, page_table, q_out=None, stream=None):
        """Append K and V [T][Hkv][D], the keys normed and rotated; returns the normed and rotated
        queries (None when q is None).  lens_after is not read by a BF16 or mixed-key cache."""
        g = self.geo
        rope.check_head_dim(g.head_dim)
        if K.shape[1:] != (g.num_kv_heads, g.head_dim) or (q is not None and q.shape[1:] != (g.num_q_heads, g.head_dim)):
            raise ValueError("q [T][Hq][D] and K, V [T][Hkv][D] of the cache's geometry expected")
        if q is not None and q_out is None:
            q_out = _new(q.shape, q.dtype, q.device, stream)
        kv4_append_rope(self.handle, layer, rope.params, q, K, V, seq_slot, pos, lens_after, page_table,
                        page_table.size(1), q_out, stream)
        return q_out

    def gather(self, layer, seq_slot, pos, page_table, lens=None, dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
        """Cached positions as dense (K, V) [T][Hkv][D] in their original basis."""
        T = seq_slot.numel()
        if pos.numel() != T:
            raise ValueError("one position per seq_slot expected")
        shape = (T, self.geo.num_kv_heads, self.geo.head_dim)
        k_out = _new(shape, dtype, pos.device, stream) if k_out is None else k_out
        v_out = _new(shape, dtype, pos.device, stream) if v_out is None else v_out
        if k_out.shape != shape or v_out.shape != shape or k_out.dtype != v_out.dtype:
            raise ValueError("k_out and v_out [T][Hkv][D] of one type expected")
        kv4_gather(self.handle, layer, T, seq_slot, pos, lens, page_table, page_table.size(1), k_out, v_out,
                   dtype_code(k_out), stream)
        return k_out, v_out


class Cache(_RopeCacheMixin):
    """INT4 cache with torch-allocated page pool and side cache (uint8 tensors)."""

    def __init__(self, geo: Geometry, device="cuda", fill: int | None = None):
        self.geo = geo
        self.cfg = geo.c()
        pool_b, side_b = kv4_query_sizes(self.cfg)
        self.pool = torch.empty(max(pool_b, 16), dtype=torch.uint8, device=device)
        self.side = torch.empty(max(side_b, 16), dtype=torch.uint8, device=device)
        if fill is not None:
            self.pool.fill_(fill)
            self.side.fill_(fill)
        self.handle = kv4_cache_init(self.cfg, self.pool, self.side)
        self._ws = _Workspaces()

    def layer_views(self, layer: int):
        """(pages of the layer, side cache of the layer) as uint8 views."""
        pool_b, side_b = kv4_query_sizes(self.cfg)
        pl, sl = self.geo.page_bytes() * self.geo.max_pages, side_b // self.geo.num_layers
        return self.pool[layer * pl:(layer + 1) * pl], self.side[layer * sl:(layer + 1) * sl]

    def allocate_key_bits(self, layer, K, stream=None):
        """Mixed bit-width keys: allocate the layer's key bits from keys K [T][Hkv][D]."""
        kv4_allocate_key_bits(self.handle, layer, int(K.shape[0]), K, dtype_code(K), stream)

    def key_allocation(self, layer):
        return kv4_get_key_allocation(self.handle, layer, self.geo.num_kv_heads, self.geo.head_dim)

    def append(self, layer, K, V, seq_slot, pos, lens_after, page_table, stream=None):
        kv4_append(self.handle, layer, int(seq_slot.numel()), K, dtype_code(K), V, dtype_code(V), seq_slot, pos,
                   lens_after, page_table, int(page_table.shape[1]), stream)

    def workspace(self, B: int, stream=None) -> torch.Tensor:
        """The cache's workspace for calls on the stream; it may be larger than the call needs."""
        return self._ws.get(kv4_decode_workspace_bytes, (self.handle, B), self.pool.device, stream)

    def decode(self, layer, q, page_table, lens, out=None, lse=None, max_len_hint=0, workspace=None, stream=None):
        B = int(lens.numel())
        if out is None:
            out = _new((B, self.geo.num_q_heads, self.geo.head_dim), torch.float32, q.device, stream)
        ws = workspace if workspace is not None else self.workspace(B, stream)
        kv4_decode_attn(self.handle, layer, B, q, dtype_code(q), page_table, int(page_table.shape[1]), lens,
                        max_len_hint, out, lse, ws, ws.numel(), stream)
        return out

    def shared_workspace(self, B: int, n_groups: int, stream=None) -> torch.Tensor:
        """The cache's workspace for calls on the stream; it may be larger than the call needs."""
        return self._ws.get(kv4_decode_shared_workspace_bytes, (self.handle, B, n_groups), self.pool.device, stream)

    def decode_shared(self, layer, q, page_table, lens, group_start, prefix_len, out=None, lse=None, max_len_hint=0,
                      workspace=None, stream=None):
        """Decode of a batch whose row groups [group_start[i], group_start[i + 1]) share their first
        prefix_len[i] positions (their whole pages; the rest is read as each row's own); out has q's type
        unless given."""
        B, n = lens.numel(), prefix_len.numel()
        shape = (B, self.geo.num_q_heads, self.geo.head_dim)
        if q.shape != shape or page_table.size(0) < B:
            raise ValueError("q [B][Hq][D] and a page-table row per sequence expected")
        if group_start.numel() != n + 1:
            raise ValueError("group_start: one entry more than prefix_len expected")
        if out is None:
            out = _new(shape, q.dtype, q.device, stream)
        elif out.shape != shape:
            raise ValueError("out [B][Hq][D] expected")
        if lse is not None and (lse.shape != shape[:2] or lse.dtype is not torch.float32):
            raise ValueError("lse float32 [B][Hq] expected")
        if workspace is None:
            workspace = self.shared_workspace(B, n, stream)
        elif workspace.dtype is not torch.uint8:
            raise ValueError("workspace: uint8 tensor expected")
        kv4_decode_attn_shared(self.handle, layer, B, q, dtype_code(q), page_table, page_table.size(1), lens, n,
                               group_start, prefix_len, max_len_hint, out, dtype_code(out), lse, workspace,
                               workspace.numel(), stream)
        return out

    def close(self):
        self._ws.clear()
        if self.handle:
            kv4_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class BF16Cache(_RopeCacheMixin):
    """BF16-KV baseline cache (same page table conventions, bf16 K and V in the pages)."""

    def __init__(self, geo: Geometry, device="cuda"):
        self.geo = geo
        self.cfg = geo.c()
        self.pool = torch.empty(max(kv4_bf16_query_sizes(self.cfg), 16), dtype=torch.uint8, device=device)
        self.handle = kv4_bf16_cache_init(self.cfg, self.pool)
        self._ws = _Workspaces()

    def append(self, layer, K, V, seq_slot, pos, page_table, stream=None):
        kv4_bf16_append(self.handle, layer, int(seq_slot.numel()), K, dtype_code(K), V, dtype_code(V), seq_slot, pos,
                        page_table, int(page_table.shape[1]), stream)

    def workspace(self, B: int, stream=None) -> torch.Tensor:
        """The cache's workspace for calls on the stream; it may be larger than the call needs."""
        return self._ws.get(kv4_bf16_decode_workspace_bytes, (self.handle, B), self.pool.device, stream)

    def decode(self, layer, q, page_table, lens, out=None, lse=None, max_len_hint=0, workspace=None, stream=None):
        B = int(lens.numel())
        if out is None:
            out = _new((B, self.geo.num_q_heads, self.geo.head_dim), torch.float32, q.device, stream)
        ws = workspace if workspace is not None else self.workspace(B, stream)
        kv4_bf16_decode_attn(self.handle, layer, B, q, dtype_code(q), page_table, int(page_table.shape[1]), lens,
                             max_len_hint, out, lse, ws, ws.numel(), stream)
        return out

    def close(self):
        self._ws.clear()
        if self.handle:
            kv4_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
