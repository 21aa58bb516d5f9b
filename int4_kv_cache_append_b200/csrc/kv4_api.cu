// kv4_api.cu -- the C ABI of libkv4.so (declared in include/kv4.h): argument validation on the
// host, grid sizing from the SM count, and the launches.  No device memory is allocated here
// except the library's one static per-device error word.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <new>
#include <vector>

#include "../../include/kv4.h"
#include "kv4_internal.h"

namespace {

__device__ uint32_t g_kv4_device_error;

constexpr int kMaxDevices = 64;
std::mutex g_mu;
uint32_t* g_err_ptr[kMaxDevices] = {};
int g_sm_count[kMaxDevices] = {};
std::atomic<uint64_t> g_launches{0};

enum Format { FMT_INT4 = 1, FMT_BF16 = 2, FMT_MIXED = 3 };

}  // namespace

struct kv4_cache {
  kv4_config cfg;
  int format;
  uint8_t* pool;
  uint8_t* side;
  size_t page_bytes;       // one page, all KV heads
  size_t pool_layer_bytes;
  size_t side_slot_bytes;  // one sequence slot, all KV heads
  size_t side_layer_bytes;
  int nt8;
  int overlap;        // kv4_set_decode_overlap
  uint32_t signs[4];  // kv4_set_rotation_signs
  int rotate_v;       // kv4_set_value_rotation
  int stall_test;     // kv4_debug_force_wait_timeout
  int mixed_rows;     // kv4_debug_mixed_row_copies
  // mixed bit-width keys: per-layer block-allocation records after the pages, and which layers
  // have one
  uint8_t* alloc_base;
  size_t alloc_layer_bytes;
  std::vector<uint8_t> allocated;
};

namespace kv4 {
void note_launches(int n) { g_launches.fetch_add(static_cast<uint64_t>(n), std::memory_order_relaxed); }
}  // namespace kv4

namespace {

bool device_info(uint32_t** err, int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_err_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_kv4_device_error) != cudaSuccess) return false;
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return false;
    g_err_ptr[dev] = static_cast<uint32_t*>(p);
    g_sm_count[dev] = n;
  }
  if (err) *err = g_err_ptr[dev];
  if (sms) *sms = g_sm_count[dev];
  return true;
}

bool pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

kv4_status check_config(const kv4_config* c) {
  if (!c) return KV4_ERR_INVALID_ARG;
  if (c->num_layers <= 0 || c->num_q_heads <= 0 || c->num_kv_heads <= 0 || c->max_seqs <= 0 || c->max_pages <= 0 ||
      c->page_size <= 0 || c->num_sinks < 0 || c->recent_window < 0 || c->head_dim <= 0 || c->hadamard_block <= 0)
    return KV4_ERR_INVALID_ARG;
  if (c->num_q_heads % c->num_kv_heads) return KV4_ERR_INVALID_ARG;
  const int G = c->num_q_heads / c->num_kv_heads;
  if (G != 1 && G != 2 && G != 4) return KV4_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return KV4_ERR_UNSUPPORTED;
  if (c->page_size % 16) return KV4_ERR_UNSUPPORTED;
  if (!pow2(c->hadamard_block) || c->head_dim % c->hadamard_block) return KV4_ERR_INVALID_ARG;
  if (c->num_sinks > (1 << 20) || c->recent_window > (1 << 20)) return KV4_ERR_UNSUPPORTED;
  if (c->value_format != KV4_VALUES_INT4 && c->value_format != KV4_VALUES_BF16 && c->value_format != KV4_KEYS_MIXED)
    return KV4_ERR_INVALID_ARG;
  if (c->value_format == KV4_KEYS_MIXED) {
    // the mixed bit-width key cache has no side cache and no rotation
    if (c->num_sinks != 0 || c->recent_window != 0 || c->hadamard_block != 1) return KV4_ERR_INVALID_ARG;
    if (c->key_bits < 1 || c->key_bits > 8) return KV4_ERR_INVALID_ARG;
    if (c->value_bits != 2 && c->value_bits != 3 && c->value_bits != 4 && c->value_bits != 8) return KV4_ERR_UNSUPPORTED;
  }
  return KV4_OK;
}

size_t mixed_alloc_layer_bytes(const kv4_config* c) {
  return static_cast<size_t>(c->num_kv_heads) * kv4::mixed_alloc_record_bytes(c->head_dim);
}

void sizes(const kv4_config* c, size_t* page_bytes, size_t* side_slot, int* nt8) {
  const size_t D = static_cast<size_t>(c->head_dim);
  if (c->value_format == KV4_KEYS_MIXED) {
    *page_bytes = static_cast<size_t>(c->num_kv_heads) * static_cast<size_t>(c->page_size) *
                  (static_cast<size_t>(c->key_bits + c->value_bits) * D / 8 + 8);
    *nt8 = 0;
    *side_slot = 0;
    return;
  }
  const bool vbf = c->value_format == KV4_VALUES_BF16;
  *page_bytes = static_cast<size_t>(c->num_kv_heads) * static_cast<size_t>(c->page_size) * (vbf ? D / 2 + 4 + 2 * D : D + 8);
  *nt8 = (c->num_sinks + c->recent_window + 15) / 16;
  *side_slot = static_cast<size_t>(c->num_kv_heads) * static_cast<size_t>(*nt8) * 16u * (vbf ? 3 * D + 2 : 2 * D + 4);
}

kv4_status dtype_ok_kv(kv4_dtype d) { return (d == KV4_F32 || d == KV4_BF16) ? KV4_OK : KV4_ERR_INVALID_ARG; }
kv4_status dtype_ok_q(kv4_dtype d) {
  return (d == KV4_F32 || d == KV4_BF16 || d == KV4_F16) ? KV4_OK : KV4_ERR_INVALID_ARG;
}

size_t align16(size_t x) { return (x + 15) & ~static_cast<size_t>(15); }

int decode_ctas_full(const kv4_cache* c, int sms) {
  if (c->format == FMT_INT4) return kv4::decode_ctas_per_sm() * sms;
  if (c->format == FMT_MIXED)
    return kv4::mixed_decode_ctas_per_sm(c->cfg.head_dim, c->cfg.num_q_heads / c->cfg.num_kv_heads, c->cfg.value_bits,
                                         c->cfg.key_bits) * sms;
  return sms;
}

int warps_per_cta(int format) {
  return format == FMT_INT4 ? kv4::decode_warps_per_cta()
                            : (format == FMT_MIXED ? kv4::mixed_decode_warps_per_cta() : kv4::bf16_decode_warps_per_cta());
}

// Workspace: per (sequence, KV head) a 16-byte record of where its partials are (max_seqs * Hkv
// records, INT4 format), then the split partials, one row group of G rows of (o[D], m, l) padded
// to D + 4 floats per possible partial index (warps of the grid + 2 * B * Hkv segments).
size_t meta_bytes(const kv4_cache* c) {
  return c->format == FMT_INT4 ? static_cast<size_t>(c->cfg.max_seqs) * c->cfg.num_kv_heads * 16 : 0;
}

size_t workspace_for(const kv4_cache* c, int B, int ctas) {
  const int G = c->cfg.num_q_heads / c->cfg.num_kv_heads;
  const int warps = ctas * warps_per_cta(c->format);
  const size_t segs = static_cast<size_t>(B) * c->cfg.num_kv_heads * (c->format == FMT_INT4 ? 2 : 1);
  return meta_bytes(c) + align16((static_cast<size_t>(warps) + segs) * G * (c->cfg.head_dim + 4) * sizeof(float));
}

// The format the INT4-cache entry points serve for this handle: the INT4 cache or the mixed
// bit-width key cache (a BF16 baseline handle maps to FMT_INT4 and is then rejected).
int own_format(const kv4_cache* c) { return (c && c->format == FMT_MIXED) ? FMT_MIXED : FMT_INT4; }

// Everything of AppendArgs that comes from the cache, the layer and the token lists.
kv4::AppendArgs cache_args(const kv4_cache* c, int layer, int T, const int32_t* seq_slot, const int32_t* pos,
                           const int32_t* lens_after, const int32_t* page_table, int stride, uint32_t* err) {
  const bool int4 = c->format == FMT_INT4;
  kv4::AppendArgs a{};
  a.pool = c->pool + static_cast<size_t>(layer) * c->pool_layer_bytes;
  a.side = c->side ? c->side + static_cast<size_t>(layer) * c->side_layer_bytes : nullptr;
  a.seq_slot = seq_slot;
  a.pos = pos;
  a.lens_after = lens_after;
  a.page_table = page_table;
  a.stride = stride;
  a.T = T;
  a.Hkv = c->cfg.num_kv_heads;
  a.P = c->cfg.page_size;
  a.p_shift = pow2(a.P) ? __builtin_ctz(static_cast<unsigned>(a.P)) : -1;
  a.s = int4 ? c->cfg.num_sinks : 0;
  a.w = int4 ? c->cfg.recent_window : 0;
  a.h = int4 ? c->cfg.hadamard_block : 1;
  a.max_seqs = c->cfg.max_seqs;
  a.max_pages = c->cfg.max_pages;
  a.nt8 = c->nt8;
  a.page_bytes = c->page_bytes;
  a.side_slot_bytes = c->side_slot_bytes;
  for (int i = 0; i < 4; ++i) a.signs[i] = int4 ? c->signs[i] : 0u;
  a.rotate_v = int4 ? c->rotate_v : 0;
  a.vbf = (int4 && c->cfg.value_format == KV4_VALUES_BF16) ? 1 : 0;
  if (c->format == FMT_MIXED) {
    a.alloc = c->alloc_base + static_cast<size_t>(layer) * c->alloc_layer_bytes;
    a.kbits = c->cfg.key_bits;
    a.vbits = c->cfg.value_bits;
  }
  a.err = err;
  return a;
}

kv4_status append_common(kv4_cache* c, int fmt, int layer, int T, const void* K, kv4_dtype kd, const void* V,
                         kv4_dtype vd, const int32_t* seq_slot, const int32_t* pos, const int32_t* lens_after,
                         const int32_t* page_table, int stride, void* stream) {
  if (!c || c->format != fmt) return KV4_ERR_INVALID_ARG;
  if (layer < 0 || layer >= c->cfg.num_layers || T < 0 || stride <= 0) return KV4_ERR_INVALID_ARG;
  if (T == 0) return KV4_OK;
  if (!K || !V || !seq_slot || !pos || !page_table || (fmt == FMT_INT4 && !lens_after)) return KV4_ERR_INVALID_ARG;
  if (fmt == FMT_MIXED && !c->allocated[layer]) return KV4_ERR_NO_ALLOCATION;
  if (dtype_ok_kv(kd) != KV4_OK || dtype_ok_kv(vd) != KV4_OK) return KV4_ERR_INVALID_ARG;
  if (!aligned(K, kd == KV4_F32 ? 16 : 8) || !aligned(V, vd == KV4_F32 ? 16 : 8)) return KV4_ERR_INVALID_ARG;
  if (static_cast<long long>(T) * c->cfg.num_kv_heads > (1LL << 30)) return KV4_ERR_UNSUPPORTED;
  uint32_t* err = nullptr;
  if (!device_info(&err, nullptr)) return KV4_ERR_CUDA;
  kv4::AppendArgs a = cache_args(c, layer, T, seq_slot, pos, lens_after, page_table, stride, err);
  a.K = K;
  a.V = V;
  a.k_dtype = kd;
  a.v_dtype = vd;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = fmt == FMT_INT4    ? kv4::launch_append_int4(a, c->cfg.head_dim, st)
                        : fmt == FMT_MIXED ? kv4::launch_append_mixed(a, c->cfg.head_dim, st)
                                           : kv4::launch_append_bf16(a, c->cfg.head_dim, st);
  return e == cudaSuccess ? KV4_OK : KV4_ERR_CUDA;
}

// Rows of D-element heads, `stride` elements apart: the kernels move four elements at a time.
bool rows_ok(const void* p, kv4_dtype d, int64_t stride, int64_t row) {
  return p && dtype_ok_q(d) == KV4_OK && aligned(p, d == KV4_F32 ? 16 : 8) && stride >= row && stride % 4 == 0;
}

kv4_status check_rope(const kv4_rope_params* r, int D) {
  if (!r || !r->table || !aligned(r->table, 16) || r->max_pos <= 0 || !(r->eps >= 0.f) || !std::isfinite(r->eps))
    return KV4_ERR_INVALID_ARG;
  if (r->layout != KV4_ROPE_HALF && r->layout != KV4_ROPE_INTERLEAVED) return KV4_ERR_INVALID_ARG;
  if (r->rotary_dim <= 0 || r->rotary_dim > D) return KV4_ERR_INVALID_ARG;
  if (r->rotary_dim % 8) return KV4_ERR_UNSUPPORTED;
  if (r->q_weight || r->k_weight) {
    if (dtype_ok_q(r->weight_dtype) != KV4_OK) return KV4_ERR_INVALID_ARG;
    const size_t al = r->weight_dtype == KV4_F32 ? 16 : 8;
    if (!aligned(r->q_weight, al) || !aligned(r->k_weight, al)) return KV4_ERR_INVALID_ARG;
  }
  return KV4_OK;
}

kv4::RopeArgs rope_args(const kv4_rope_params* r, uint32_t* err) {
  kv4::RopeArgs a{};
  a.table = r->table;
  a.max_pos = r->max_pos;
  a.R = r->rotary_dim;
  a.layout = r->layout;
  a.qw = r->q_weight;
  a.kw = r->k_weight;
  a.w_dtype = r->weight_dtype;
  a.eps = r->eps;
  a.err = err;
  return a;
}

// Warps of the rotary kernels are counted in 32 bits.
constexpr long long kMaxVectors = 1LL << 26;

// What kv4_decode_attn_shared adds.
struct SharedPrefix {
  int n_groups;
  const int32_t* group_start;
  const int32_t* prefix_len;
  int out_dtype;
};

// Its workspace after the decode's own: the prefix records, the own-tile list, the prefix partials.
size_t shared_rows_bytes(const kv4_cache* c, int B) {
  return static_cast<size_t>(B) * c->cfg.num_kv_heads * 16 + align16(static_cast<size_t>(B) * 4);
}
size_t shared_part_bytes(const kv4_cache* c, int B, int n_groups, int sms) {
  const size_t G = static_cast<size_t>(c->cfg.num_q_heads / c->cfg.num_kv_heads), rb = static_cast<size_t>(kv4::shared_row_block());
  const size_t segs = static_cast<size_t>(c->cfg.num_kv_heads) * (static_cast<size_t>(n_groups) + static_cast<size_t>(B) * G / rb);
  return (static_cast<size_t>(sms) + segs) * rb * (static_cast<size_t>(c->cfg.head_dim) + 4) * sizeof(float);
}

kv4_status decode_common(kv4_cache* c, int fmt, int layer, int B, const void* q, kv4_dtype qd,
                         const int32_t* page_table, int stride, const int32_t* lens, int max_len_hint, float* out,
                         float* lse, void* ws, size_t ws_bytes, void* stream, const SharedPrefix* sp = nullptr) {
  if (!c || c->format != fmt) return KV4_ERR_INVALID_ARG;
  if (layer < 0 || layer >= c->cfg.num_layers || B < 0 || B > c->cfg.max_seqs || stride <= 0 || max_len_hint < 0)
    return KV4_ERR_INVALID_ARG;
  if (B == 0) return KV4_OK;
  if (!q || !page_table || !lens || !out) return KV4_ERR_INVALID_ARG;
  if (dtype_ok_q(qd) != KV4_OK) return KV4_ERR_INVALID_ARG;
  if (!aligned(q, qd == KV4_F32 ? 4 : 2) || !aligned(out, 16)) return KV4_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 16)) return KV4_ERR_WORKSPACE;
  if (fmt == FMT_MIXED && !c->allocated[layer]) return KV4_ERR_NO_ALLOCATION;
  uint32_t* err = nullptr;
  int sms = 0;
  if (!device_info(&err, &sms)) return KV4_ERR_CUDA;
  const int full = decode_ctas_full(c, sms);
  int ctas = full;
  if (max_len_hint > 0) {
    // Enough CTAs that each warp gets at least ~16 slots of the hinted upper bound.
    const long long tiles = (static_cast<long long>(max_len_hint) + 15) / 16;
    const long long slots = static_cast<long long>(B) * c->cfg.num_kv_heads * (tiles + (fmt == FMT_INT4 ? 2LL * c->nt8 : 0));
    const int warps = warps_per_cta(fmt);
    long long want = (slots + 16LL * warps - 1) / (16LL * warps);
    if (want < 1) want = 1;
    if (want < ctas) ctas = static_cast<int>(want);
  }
  const size_t own_ws = workspace_for(c, B, ctas);
  if (ws_bytes < own_ws + (sp ? shared_rows_bytes(c, B) + shared_part_bytes(c, B, sp->n_groups, sms) : 0)) return KV4_ERR_WORKSPACE;
  {
    // work units are counted in 32 bits on the device: bound the worst case (every sequence at
    // the page-table capacity)
    const long long tiles = (static_cast<long long>(stride) * c->cfg.page_size + 15) / 16;
    const long long units = static_cast<long long>(B) * c->cfg.num_kv_heads * (tiles + 2LL * c->nt8);
    if (units >= (1LL << 31)) return KV4_ERR_UNSUPPORTED;
    // so are the prefix kernel's: every segment at the page-table capacity
    if (sp && (sp->n_groups + static_cast<long long>(B)) * c->cfg.num_kv_heads * (tiles / 8 + 2) >= (1LL << 31)) return KV4_ERR_UNSUPPORTED;
  }
  kv4::DecodeArgs a{};
  a.pool = c->pool + static_cast<size_t>(layer) * c->pool_layer_bytes;
  a.side = c->side ? c->side + static_cast<size_t>(layer) * c->side_layer_bytes : nullptr;
  a.q = q;
  a.q_dtype = qd;
  a.page_table = page_table;
  a.stride = stride;
  a.lens = lens;
  a.B = B;
  a.Hq = c->cfg.num_q_heads;
  a.Hkv = c->cfg.num_kv_heads;
  a.P = c->cfg.page_size;
  a.s = fmt == FMT_INT4 ? c->cfg.num_sinks : 0;
  a.w = fmt == FMT_INT4 ? c->cfg.recent_window : 0;
  a.h = fmt == FMT_INT4 ? c->cfg.hadamard_block : 1;
  a.max_pages = c->cfg.max_pages;
  a.nt8 = c->nt8;
  a.smw = a.w > 0 ? a.s % a.w : 0;
  a.page_bytes = c->page_bytes;
  a.side_slot_bytes = c->side_slot_bytes;
  a.meta = static_cast<unsigned int*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + meta_bytes(c));
  a.out = out;
  a.lse = lse;
  a.qscale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(c->cfg.head_dim)));
  a.err = err;
  a.early = (fmt == FMT_INT4 && c->overlap) ? 1 : 0;
  for (int i = 0; i < 4; ++i) a.signs[i] = c->signs[i];
  a.rotate_v = fmt == FMT_INT4 ? c->rotate_v : 0;
  a.vbf = (fmt == FMT_INT4 && c->cfg.value_format == KV4_VALUES_BF16) ? 1 : 0;
  const int tpp = c->cfg.page_size / 16;
  a.tp_shift = pow2(tpp) ? __builtin_ctz(static_cast<unsigned>(tpp)) : -1;
  // The wait-limit test runs every warp's first wait out after 1 ms; the normal limit is 2 s.
  a.stall_test = ((fmt == FMT_INT4 || fmt == FMT_MIXED) && c->stall_test) ? 1 : 0;
  a.wait_ns = a.stall_test ? 1000000ull : 2000000000ull;
  if (fmt == FMT_MIXED) {
    a.alloc = c->alloc_base + static_cast<size_t>(layer) * c->alloc_layer_bytes;
    a.kbits = c->cfg.key_bits;
    a.vbits = c->cfg.value_bits;
  }
  const int G = c->cfg.num_q_heads / c->cfg.num_kv_heads;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (sp) {
    uint8_t* rows = static_cast<uint8_t*>(ws) + own_ws;
    a.n_groups = sp->n_groups;
    a.group_start = sp->group_start;
    a.prefix_len = sp->prefix_len;
    a.out_dtype = sp->out_dtype;
    a.PW = sms;
    a.early = 0;  // its first kernel writes what the decode's schedule reads
    a.pmeta = reinterpret_cast<uint4*>(rows);
    a.own = reinterpret_cast<int*>(rows + static_cast<size_t>(B) * c->cfg.num_kv_heads * 16);
    a.ppart = reinterpret_cast<float*>(rows + shared_rows_bytes(c, B));
    return kv4::launch_decode_shared(a, c->cfg.head_dim, G, ctas, st) == cudaSuccess ? KV4_OK : KV4_ERR_CUDA;
  }
  const cudaError_t e = fmt == FMT_INT4    ? kv4::launch_decode_int4(a, c->cfg.head_dim, G, ctas, st)
                        : fmt == FMT_MIXED ? kv4::launch_decode_mixed(a, c->cfg.head_dim, G, ctas, st, c->mixed_rows != 0)
                                           : kv4::launch_decode_bf16(a, c->cfg.head_dim, G, ctas, st);
  return e == cudaSuccess ? KV4_OK : KV4_ERR_CUDA;
}

}  // namespace

extern "C" {

kv4_status kv4_query_sizes(const kv4_config* cfg, size_t* page_pool_bytes, size_t* side_cache_bytes) {
  const kv4_status st = check_config(cfg);
  if (st != KV4_OK) return st;
  size_t pb, ss;
  int nt8;
  sizes(cfg, &pb, &ss, &nt8);
  if (page_pool_bytes)
    *page_pool_bytes = static_cast<size_t>(cfg->num_layers) * cfg->max_pages * pb +
                       (cfg->value_format == KV4_KEYS_MIXED ? static_cast<size_t>(cfg->num_layers) * mixed_alloc_layer_bytes(cfg) : 0);
  if (side_cache_bytes) *side_cache_bytes = static_cast<size_t>(cfg->num_layers) * cfg->max_seqs * ss;
  return KV4_OK;
}

kv4_status kv4_cache_init(const kv4_config* cfg, void* page_pool, void* side_cache, kv4_cache** out) {
  const kv4_status st = check_config(cfg);
  if (st != KV4_OK) return st;
  if (!out || !page_pool || !aligned(page_pool, 16)) return KV4_ERR_INVALID_ARG;
  const bool need_side = cfg->num_sinks + cfg->recent_window > 0;
  if (need_side && (!side_cache || !aligned(side_cache, 16))) return KV4_ERR_INVALID_ARG;
  kv4_cache* c = new (std::nothrow) kv4_cache();
  if (!c) return KV4_ERR_INVALID_ARG;
  c->cfg = *cfg;
  c->format = cfg->value_format == KV4_KEYS_MIXED ? FMT_MIXED : FMT_INT4;
  c->pool = static_cast<uint8_t*>(page_pool);
  c->side = need_side ? static_cast<uint8_t*>(side_cache) : nullptr;
  sizes(cfg, &c->page_bytes, &c->side_slot_bytes, &c->nt8);
  c->pool_layer_bytes = c->page_bytes * static_cast<size_t>(cfg->max_pages);
  c->side_layer_bytes = c->side_slot_bytes * static_cast<size_t>(cfg->max_seqs);
  if (c->format == FMT_MIXED) {
    c->alloc_base = c->pool + c->pool_layer_bytes * static_cast<size_t>(cfg->num_layers);
    c->alloc_layer_bytes = mixed_alloc_layer_bytes(cfg);
    try {
      c->allocated.assign(static_cast<size_t>(cfg->num_layers), 0);
    } catch (...) {
      delete c;
      return KV4_ERR_INVALID_ARG;
    }
  }
  *out = c;
  return KV4_OK;
}

void kv4_cache_destroy(kv4_cache* cache) { delete cache; }

kv4_status kv4_append(kv4_cache* cache, int layer, int T, const void* K, kv4_dtype k_dtype, const void* V,
                      kv4_dtype v_dtype, const int32_t* seq_slot, const int32_t* pos, const int32_t* lens_after,
                      const int32_t* page_table, int stride, void* stream) {
  return append_common(cache, own_format(cache), layer, T, K, k_dtype, V, v_dtype, seq_slot, pos, lens_after, page_table,
                       stride, stream);
}

kv4_status kv4_decode_workspace_bytes(const kv4_cache* cache, int B, size_t* bytes) {
  if (!cache || own_format(cache) != cache->format || B < 0 || !bytes) return KV4_ERR_INVALID_ARG;
  int sms = 0;
  if (!device_info(nullptr, &sms)) return KV4_ERR_CUDA;
  *bytes = workspace_for(cache, B, decode_ctas_full(cache, sms));
  return KV4_OK;
}

kv4_status kv4_decode_attn(kv4_cache* cache, int layer, int B, const void* q, kv4_dtype q_dtype,
                           const int32_t* page_table, int stride, const int32_t* lens, int max_len_hint, float* out,
                           float* lse, void* workspace, size_t ws_bytes, void* stream) {
  return decode_common(cache, own_format(cache), layer, B, q, q_dtype, page_table, stride, lens, max_len_hint, out,
                       lse, workspace, ws_bytes, stream);
}

kv4_status kv4_decode_shared_workspace_bytes(const kv4_cache* cache, int B, int n_groups, size_t* bytes) {
  if (!cache || cache->format != FMT_INT4 || B < 0 || n_groups < 0 || !bytes) return KV4_ERR_INVALID_ARG;
  if (cache->cfg.value_format != KV4_VALUES_INT4) return KV4_ERR_UNSUPPORTED;
  int sms = 0;
  if (!device_info(nullptr, &sms)) return KV4_ERR_CUDA;
  *bytes = workspace_for(cache, B, decode_ctas_full(cache, sms)) + shared_rows_bytes(cache, B) + shared_part_bytes(cache, B, n_groups, sms);
  return KV4_OK;
}

kv4_status kv4_decode_attn_shared(kv4_cache* cache, int layer, int B, const void* q, kv4_dtype q_dtype,
                                  const int32_t* page_table, int stride, const int32_t* lens, int n_groups,
                                  const int32_t* group_start, const int32_t* prefix_len, int max_len_hint, void* out,
                                  kv4_dtype out_dtype, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  if (!cache || cache->format != FMT_INT4 || n_groups < 0 || n_groups > (1 << 20) || dtype_ok_q(out_dtype) != KV4_OK)
    return KV4_ERR_INVALID_ARG;
  if (cache->cfg.value_format != KV4_VALUES_INT4) return KV4_ERR_UNSUPPORTED;
  if (B > 0 && n_groups > 0 && (!group_start || !prefix_len)) return KV4_ERR_INVALID_ARG;
  const SharedPrefix sp{n_groups, group_start, prefix_len, out_dtype};
  return decode_common(cache, FMT_INT4, layer, B, q, q_dtype, page_table, stride, lens, max_len_hint, static_cast<float*>(out),
                       lse, workspace, ws_bytes, stream, &sp);
}

// No-allocation decode: the split-K partials go to this file-scope device array instead of a
// caller workspace.  In host code the name is only a stand-in, so its device address is looked
// up per device (cudaGetSymbolAddress, with that device current) and passed to the kernels.
static __device__ __align__(256) unsigned char g_kv4_static_scratch[KV4_STATIC_SCRATCH_BYTES];
static void* g_static_scratch_ptr[kMaxDevices] = {};

// First use on a device: look up the array's address (with that device current).
static bool static_scratch_address(void** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_static_scratch_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_kv4_static_scratch) != cudaSuccess || !p) return false;
    g_static_scratch_ptr[dev] = p;
  }
  *out = g_static_scratch_ptr[dev];
  return true;
}

kv4_status kv4_set_rotation_signs(kv4_cache* cache, const uint32_t* sign_bits) {
  if (!cache || cache->format != FMT_INT4) return KV4_ERR_INVALID_ARG;
  const int words = (cache->cfg.head_dim + 31) / 32;
  for (int i = 0; i < 4; ++i) cache->signs[i] = (sign_bits && i < words) ? sign_bits[i] : 0u;
  return KV4_OK;
}

kv4_status kv4_set_value_rotation(kv4_cache* cache, int enable) {
  if (!cache || cache->format != FMT_INT4) return KV4_ERR_INVALID_ARG;
  if (enable && cache->cfg.value_format == KV4_VALUES_BF16) return KV4_ERR_INVALID_ARG;
  cache->rotate_v = enable ? 1 : 0;
  return KV4_OK;
}

kv4_status kv4_set_decode_overlap(kv4_cache* cache, int enable) {
  if (!cache || cache->format != FMT_INT4) return KV4_ERR_INVALID_ARG;
  cache->overlap = enable ? 1 : 0;
  return KV4_OK;
}

kv4_status kv4_debug_force_wait_timeout(kv4_cache* cache, int enable) {
  if (!cache || (cache->format != FMT_INT4 && cache->format != FMT_MIXED)) return KV4_ERR_INVALID_ARG;
  cache->stall_test = enable ? 1 : 0;
  return KV4_OK;
}

kv4_status kv4_debug_mixed_row_copies(kv4_cache* cache, int enable) {
  if (!cache || cache->format != FMT_MIXED) return KV4_ERR_INVALID_ARG;
  cache->mixed_rows = enable ? 1 : 0;
  return KV4_OK;
}

kv4_status kv4_allocate_key_bits(kv4_cache* cache, int layer, int T, const void* K, kv4_dtype k_dtype, void* stream) {
  if (!cache || cache->format != FMT_MIXED || layer < 0 || layer >= cache->cfg.num_layers || T < 0)
    return KV4_ERR_INVALID_ARG;
  if (T > 0 && (!K || dtype_ok_q(k_dtype) != KV4_OK || !aligned(K, k_dtype == KV4_F32 ? 4 : 2))) return KV4_ERR_INVALID_ARG;
  if (!device_info(nullptr, nullptr)) return KV4_ERR_CUDA;
  kv4::ScoreArgs a{};
  a.K = K;
  a.k_dtype = k_dtype;
  a.T = T;
  a.Hkv = cache->cfg.num_kv_heads;
  a.kbits = cache->cfg.key_bits;
  a.alloc = cache->alloc_base + static_cast<size_t>(layer) * cache->alloc_layer_bytes;
  if (kv4::launch_mixed_score(a, cache->cfg.head_dim, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return KV4_ERR_CUDA;
  cache->allocated[layer] = 1;
  return KV4_OK;
}

kv4_status kv4_set_key_allocation(kv4_cache* cache, int layer, const uint8_t* widths, const float* sigma, void* stream) {
  if (!cache || cache->format != FMT_MIXED || layer < 0 || layer >= cache->cfg.num_layers || !widths || !sigma)
    return KV4_ERR_INVALID_ARG;
  const int Hkv = cache->cfg.num_kv_heads, NB = cache->cfg.head_dim / 2;
  const size_t rec = kv4::mixed_alloc_record_bytes(cache->cfg.head_dim);
  std::vector<uint8_t> host;
  try {
    host.assign(cache->alloc_layer_bytes, 0);
  } catch (...) {
    return KV4_ERR_INVALID_ARG;
  }
  for (int g = 0; g < Hkv; ++g) {
    int sum = 0;
    for (int b = 0; b < NB; ++b) {
      const uint8_t w = widths[static_cast<size_t>(g) * NB + b];
      const float sg = sigma[static_cast<size_t>(g) * NB + b];
      if (w > 8 || !(sg > 0.f) || !std::isfinite(sg)) return KV4_ERR_INVALID_ARG;
      sum += w;
      std::memcpy(host.data() + g * rec + 4 * static_cast<size_t>(b), &sg, 4);
      host[g * rec + 4 * static_cast<size_t>(NB) + b] = w;
    }
    if (sum != cache->cfg.key_bits * NB) return KV4_ERR_INVALID_ARG;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(cache->alloc_base + static_cast<size_t>(layer) * cache->alloc_layer_bytes, host.data(), host.size(),
                      cudaMemcpyHostToDevice, st) != cudaSuccess)
    return KV4_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return KV4_ERR_CUDA;  // host buffer freed on return
  cache->allocated[layer] = 1;
  return KV4_OK;
}

kv4_status kv4_get_key_allocation(kv4_cache* cache, int layer, uint8_t* widths, float* sigma, void* stream) {
  if (!cache || cache->format != FMT_MIXED || layer < 0 || layer >= cache->cfg.num_layers || !widths || !sigma)
    return KV4_ERR_INVALID_ARG;
  if (!cache->allocated[layer]) return KV4_ERR_NO_ALLOCATION;
  const int Hkv = cache->cfg.num_kv_heads, NB = cache->cfg.head_dim / 2;
  const size_t rec = kv4::mixed_alloc_record_bytes(cache->cfg.head_dim);
  std::vector<uint8_t> host;
  try {
    host.assign(cache->alloc_layer_bytes, 0);
  } catch (...) {
    return KV4_ERR_INVALID_ARG;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(host.data(), cache->alloc_base + static_cast<size_t>(layer) * cache->alloc_layer_bytes, host.size(),
                      cudaMemcpyDeviceToHost, st) != cudaSuccess)
    return KV4_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return KV4_ERR_CUDA;
  for (int g = 0; g < Hkv; ++g)
    for (int b = 0; b < NB; ++b) {
      std::memcpy(&sigma[static_cast<size_t>(g) * NB + b], host.data() + g * rec + 4 * static_cast<size_t>(b), 4);
      widths[static_cast<size_t>(g) * NB + b] = host[g * rec + 4 * static_cast<size_t>(NB) + b];
    }
  return KV4_OK;
}

kv4_status kv4_decode_attn_static(kv4_cache* cache, int layer, int B, const void* q, kv4_dtype q_dtype,
                                  const int32_t* page_table, int stride, const int32_t* lens, int max_len_hint,
                                  float* out, float* lse, void* stream) {
  if (!cache || own_format(cache) != cache->format || B < 0 || B > cache->cfg.max_seqs) return KV4_ERR_INVALID_ARG;
  if (B == 0) return KV4_OK;
  int sms = 0;
  if (!device_info(nullptr, &sms)) return KV4_ERR_CUDA;
  if (workspace_for(cache, B, decode_ctas_full(cache, sms)) > KV4_STATIC_SCRATCH_BYTES) return KV4_ERR_WORKSPACE;
  void* scratch = nullptr;
  if (!static_scratch_address(&scratch)) return KV4_ERR_CUDA;
  return decode_common(cache, cache->format, layer, B, q, q_dtype, page_table, stride, lens, max_len_hint, out, lse,
                       scratch, KV4_STATIC_SCRATCH_BYTES, stream);
}

kv4_status kv4_bf16_query_sizes(const kv4_config* cfg, size_t* page_pool_bytes) {
  const kv4_status st = check_config(cfg);
  if (st != KV4_OK) return st;
  if (page_pool_bytes)
    *page_pool_bytes = static_cast<size_t>(cfg->num_layers) * cfg->max_pages * cfg->num_kv_heads * cfg->page_size * 4 *
                       static_cast<size_t>(cfg->head_dim);
  return KV4_OK;
}

kv4_status kv4_bf16_cache_init(const kv4_config* cfg, void* page_pool, kv4_cache** out) {
  const kv4_status st = check_config(cfg);
  if (st != KV4_OK) return st;
  if (!out || !page_pool || !aligned(page_pool, 16)) return KV4_ERR_INVALID_ARG;
  kv4_cache* c = new (std::nothrow) kv4_cache();
  if (!c) return KV4_ERR_INVALID_ARG;
  c->cfg = *cfg;
  c->cfg.value_format = KV4_VALUES_INT4;  // the baseline pool stores K and V in bf16 whatever the field says
  c->format = FMT_BF16;
  c->pool = static_cast<uint8_t*>(page_pool);
  c->side = nullptr;
  c->page_bytes = static_cast<size_t>(cfg->num_kv_heads) * cfg->page_size * 4 * static_cast<size_t>(cfg->head_dim);
  c->pool_layer_bytes = c->page_bytes * static_cast<size_t>(cfg->max_pages);
  c->side_slot_bytes = 0;
  c->side_layer_bytes = 0;
  c->nt8 = 0;
  *out = c;
  return KV4_OK;
}

kv4_status kv4_bf16_append(kv4_cache* cache, int layer, int T, const void* K, kv4_dtype k_dtype, const void* V,
                           kv4_dtype v_dtype, const int32_t* seq_slot, const int32_t* pos, const int32_t* page_table,
                           int stride, void* stream) {
  return append_common(cache, FMT_BF16, layer, T, K, k_dtype, V, v_dtype, seq_slot, pos, nullptr, page_table, stride,
                       stream);
}

kv4_status kv4_bf16_decode_workspace_bytes(const kv4_cache* cache, int B, size_t* bytes) {
  if (!cache || cache->format != FMT_BF16 || B < 0 || !bytes) return KV4_ERR_INVALID_ARG;
  int sms = 0;
  if (!device_info(nullptr, &sms)) return KV4_ERR_CUDA;
  *bytes = workspace_for(cache, B, decode_ctas_full(cache, sms));
  return KV4_OK;
}

kv4_status kv4_bf16_decode_attn(kv4_cache* cache, int layer, int B, const void* q, kv4_dtype q_dtype,
                                const int32_t* page_table, int stride, const int32_t* lens, int max_len_hint,
                                float* out, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  return decode_common(cache, FMT_BF16, layer, B, q, q_dtype, page_table, stride, lens, max_len_hint, out, lse,
                       workspace, ws_bytes, stream);
}

// Frequencies of a rotary configuration as turns per position; false when a parameter is out of range.
static bool rope_frequencies(const kv4_rope_config* c, double* turns, double* mult) {
  constexpr double kTwoPi = 6.283185307179586476925;
  auto positive = [](double x) { return x > 0.0 && std::isfinite(x); };
  const int R = c->rotary_dim, n = R / 2;
  const double f = c->factor, L = static_cast<double>(c->original_max_pos);
  if (!(c->base > 1.0) || !std::isfinite(c->base) || !std::isfinite(c->attention_factor) || c->attention_factor < 0.0) return false;
  if (c->scaling != KV4_ROPE_SCALE_NONE && !positive(f)) return false;
  *mult = c->attention_factor > 0.0 ? c->attention_factor : 1.0;
  const double base = c->scaling == KV4_ROPE_SCALE_NTK ? c->base * std::pow(f, static_cast<double>(R) / (R - 2)) : c->base;
  if (!(base > 0.0) || !std::isfinite(base)) return false;
  double low = 0.0, high = 1.0;
  if (c->scaling == KV4_ROPE_SCALE_YARN) {
    if (c->original_max_pos <= 0 || !positive(c->beta_slow) || !positive(c->beta_fast) || c->beta_fast <= c->beta_slow) return false;
    // pair index at which a pair turns `beta` times over the trained length
    auto index = [&](double beta) { return R * std::log(L / (beta * kTwoPi)) / (2.0 * std::log(c->base)); };
    low = std::fmax(std::floor(index(c->beta_fast)), 0.0);
    high = std::fmin(std::ceil(index(c->beta_slow)), R - 1.0);
    if (!(high > low)) high = low + 0.001;
    if (c->attention_factor == 0.0 && f > 1.0) *mult = 0.1 * std::log(f) + 1.0;
  }
  if (c->scaling == KV4_ROPE_SCALE_BANDS &&
      (c->original_max_pos <= 0 || !positive(c->low_freq_factor) || !positive(c->high_freq_factor) ||
       c->high_freq_factor <= c->low_freq_factor))
    return false;
  for (int i = 0; i < n; ++i) {
    double w = std::pow(base, -2.0 * i / R);
    double keep = 1.0;  // share of the unscaled frequency
    switch (c->scaling) {
      case KV4_ROPE_SCALE_NONE:
      case KV4_ROPE_SCALE_NTK: break;
      case KV4_ROPE_SCALE_LINEAR: keep = 0.0; break;
      case KV4_ROPE_SCALE_YARN: keep = 1.0 - std::fmin(std::fmax((i - low) / (high - low), 0.0), 1.0); break;
      case KV4_ROPE_SCALE_BANDS:
        keep = std::fmin(std::fmax((L * w / kTwoPi - c->low_freq_factor) / (c->high_freq_factor - c->low_freq_factor), 0.0), 1.0);
        break;
      default: return false;
    }
    if (keep < 1.0) w = keep * w + (1.0 - keep) * w / f;
    turns[i] = w / kTwoPi;
  }
  return true;
}

kv4_status kv4_rope_table(const kv4_rope_config* cfg, float* table, void* stream) {
  if (!cfg || !table || !aligned(table, 16) || cfg->max_pos <= 0 || cfg->rotary_dim <= 0) return KV4_ERR_INVALID_ARG;
  if (cfg->rotary_dim % 8 || cfg->rotary_dim > 128) return KV4_ERR_UNSUPPORTED;
  kv4::RopeTableArgs a{};
  if (!rope_frequencies(cfg, a.turns, &a.mult)) return KV4_ERR_INVALID_ARG;
  a.table = reinterpret_cast<float2*>(table);
  a.max_pos = cfg->max_pos;
  a.R = cfg->rotary_dim;
  return kv4::launch_rope_table(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KV4_OK : KV4_ERR_CUDA;
}

kv4_status kv4_rope(const kv4_rope_params* rope, int T, int Hq, int Hkv, int D, const void* q, kv4_dtype q_dtype,
                    int64_t q_stride, const void* k, kv4_dtype k_dtype, int64_t k_stride, const int32_t* pos, void* q_out,
                    kv4_dtype q_out_dtype, int64_t q_out_stride, void* k_out, kv4_dtype k_out_dtype, int64_t k_out_stride,
                    void* stream) {
  if (T < 0 || Hq < 0 || Hkv < 0) return KV4_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return KV4_ERR_UNSUPPORTED;
  const kv4_status st = check_rope(rope, D);
  if (st != KV4_OK) return st;
  if (T == 0 || Hq + Hkv == 0) return KV4_OK;
  if (!pos) return KV4_ERR_INVALID_ARG;
  if (Hq > (1 << 20) || Hkv > (1 << 20) || static_cast<long long>(T) * (Hq + Hkv) > kMaxVectors) return KV4_ERR_UNSUPPORTED;
  const int64_t qr = static_cast<int64_t>(Hq) * D, kr = static_cast<int64_t>(Hkv) * D;
  if (Hq && (!rows_ok(q, q_dtype, q_stride, qr) || !rows_ok(q_out, q_out_dtype, q_out_stride, qr))) return KV4_ERR_INVALID_ARG;
  if (Hkv && (!rows_ok(k, k_dtype, k_stride, kr) || !rows_ok(k_out, k_out_dtype, k_out_stride, kr))) return KV4_ERR_INVALID_ARG;
  if (Hq && q == q_out && (q_dtype != q_out_dtype || q_stride != q_out_stride)) return KV4_ERR_INVALID_ARG;
  if (Hkv && k == k_out && (k_dtype != k_out_dtype || k_stride != k_out_stride)) return KV4_ERR_INVALID_ARG;
  uint32_t* err = nullptr;
  if (!device_info(&err, nullptr)) return KV4_ERR_CUDA;
  kv4::RopeArgs a = rope_args(rope, err);
  a.q = q;
  a.q_dtype = q_dtype;
  a.q_stride = q_stride;
  a.k = k;
  a.k_dtype = k_dtype;
  a.k_stride = k_stride;
  a.q_out = q_out;
  a.q_out_dtype = q_out_dtype;
  a.q_out_stride = q_out_stride;
  a.k_out = k_out;
  a.k_out_dtype = k_out_dtype;
  a.k_out_stride = k_out_stride;
  a.pos = pos;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  return kv4::launch_rope(a, D, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KV4_OK : KV4_ERR_CUDA;
}

kv4_status kv4_append_rope(kv4_cache* cache, int layer, int T, const kv4_rope_params* rope, const void* q,
                           kv4_dtype q_dtype, int64_t q_stride, const void* K, kv4_dtype k_dtype, int64_t k_stride,
                           const void* V, kv4_dtype v_dtype, int64_t v_stride, const int32_t* seq_slot, const int32_t* pos,
                           const int32_t* lens_after, const int32_t* page_table, int stride, void* q_out,
                           kv4_dtype q_out_dtype, int64_t q_out_stride, void* stream) {
  if (!cache || layer < 0 || layer >= cache->cfg.num_layers || T < 0 || stride <= 0) return KV4_ERR_INVALID_ARG;
  const int D = cache->cfg.head_dim, Hq = q ? cache->cfg.num_q_heads : 0, Hkv = cache->cfg.num_kv_heads;
  const kv4_status st = check_rope(rope, D);
  if (st != KV4_OK) return st;
  if (T == 0) return KV4_OK;
  if (!seq_slot || !pos || !page_table || (cache->format == FMT_INT4 && !lens_after)) return KV4_ERR_INVALID_ARG;
  if (cache->format == FMT_MIXED && !cache->allocated[layer]) return KV4_ERR_NO_ALLOCATION;
  const int64_t qr = static_cast<int64_t>(Hq) * D, kr = static_cast<int64_t>(Hkv) * D;
  if (!rows_ok(K, k_dtype, k_stride, kr) || !rows_ok(V, v_dtype, v_stride, kr)) return KV4_ERR_INVALID_ARG;
  if (q && (!rows_ok(q, q_dtype, q_stride, qr) || !rows_ok(q_out, q_out_dtype, q_out_stride, qr))) return KV4_ERR_INVALID_ARG;
  if (q && q == q_out && (q_dtype != q_out_dtype || q_stride != q_out_stride)) return KV4_ERR_INVALID_ARG;
  if (static_cast<long long>(T) * (Hq + 2LL * Hkv) > kMaxVectors) return KV4_ERR_UNSUPPORTED;
  uint32_t* err = nullptr;
  if (!device_info(&err, nullptr)) return KV4_ERR_CUDA;
  const kv4::AppendArgs a = cache_args(cache, layer, T, seq_slot, pos, lens_after, page_table, stride, err);
  kv4::RopeArgs r = rope_args(rope, err);
  r.q = q;
  r.q_dtype = q_dtype;
  r.q_stride = q_stride;
  r.k = K;
  r.k_dtype = k_dtype;
  r.k_stride = k_stride;
  r.v = V;
  r.v_dtype = v_dtype;
  r.v_stride = v_stride;
  r.q_out = q_out;
  r.q_out_dtype = q_out_dtype;
  r.q_out_stride = q_out_stride;
  r.T = T;
  r.Hq = Hq;
  r.Hkv = Hkv;
  const cudaError_t e = kv4::launch_append_rope(r, a, D, cache->format == FMT_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KV4_OK : KV4_ERR_CUDA;
}

kv4_status kv4_gather(kv4_cache* cache, int layer, int T, const int32_t* seq_slot, const int32_t* pos, const int32_t* lens,
                      const int32_t* page_table, int stride, void* K_out, void* V_out, kv4_dtype out_dtype, void* stream) {
  if (!cache || layer < 0 || layer >= cache->cfg.num_layers || T < 0 || stride <= 0 || dtype_ok_q(out_dtype) != KV4_OK)
    return KV4_ERR_INVALID_ARG;
  if (T == 0 || (!K_out && !V_out)) return KV4_OK;
  if (!seq_slot || !pos || !page_table || !aligned(K_out, 16) || !aligned(V_out, 16)) return KV4_ERR_INVALID_ARG;
  if (cache->format == FMT_MIXED && !cache->allocated[layer]) return KV4_ERR_NO_ALLOCATION;
  if (static_cast<long long>(T) * cache->cfg.num_kv_heads > kMaxVectors) return KV4_ERR_UNSUPPORTED;
  uint32_t* err = nullptr;
  if (!device_info(&err, nullptr)) return KV4_ERR_CUDA;
  const kv4::AppendArgs a = cache_args(cache, layer, T, seq_slot, pos, lens, page_table, stride, err);
  const cudaError_t e = kv4::launch_gather(a, cache->cfg.head_dim, cache->format == FMT_BF16, K_out, V_out, out_dtype,
                                           static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KV4_OK : KV4_ERR_CUDA;
}

kv4_status kv4_get_device_error(uint32_t* bits) {
  if (!bits) return KV4_ERR_INVALID_ARG;
  if (!device_info(nullptr, nullptr)) return KV4_ERR_CUDA;
  if (cudaDeviceSynchronize() != cudaSuccess) return KV4_ERR_CUDA;
  uint32_t v = 0;
  if (cudaMemcpyFromSymbol(&v, g_kv4_device_error, sizeof(v)) != cudaSuccess) return KV4_ERR_CUDA;
  const uint32_t zero = 0;
  if (cudaMemcpyToSymbol(g_kv4_device_error, &zero, sizeof(zero)) != cudaSuccess) return KV4_ERR_CUDA;
  *bits = v;
  return KV4_OK;
}

uint64_t kv4_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

const char* kv4_status_string(kv4_status s) {
  switch (s) {
    case KV4_OK: return "ok";
    case KV4_ERR_INVALID_ARG: return "invalid argument";
    case KV4_ERR_UNSUPPORTED: return "unsupported geometry";
    case KV4_ERR_WORKSPACE: return "workspace missing or too small";
    case KV4_ERR_CUDA: return "CUDA error";
    case KV4_ERR_DEVICE: return "device-side guard fired";
    case KV4_ERR_NO_ALLOCATION: return "layer has no key bit allocation";
  }
  return "unknown status";
}

int kv4_version(void) { return 100; }

}  // extern "C"
