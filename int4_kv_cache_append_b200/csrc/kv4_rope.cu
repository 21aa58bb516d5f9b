// kv4_rope.cu -- rotary positions up to the cache: the cos/sin table, the per-head norm and rotation
// of queries and keys (kv4_rope), the same fused with the append of any cache format
// (kv4_append_rope), and the cache read back as dense keys and values (kv4_gather).
//
// Mathematics.  Pair i of a head at position p turns by the angle p f_i:
//   (a, b) -> (a cos - b sin, b cos + a sin),
// (a, b) = elements (i, i + R/2) (KV4_ROPE_HALF) or (2i, 2i + 1) (KV4_ROPE_INTERLEAVED) of the first
// R elements; the others pass.  Before it, with a weight, x_j -> x_j r w_j, r = 1 / sqrt(mean x^2 + eps).
// Every step is fixed so that the codes an append writes do not depend on the launch: the sum of
// squares is taken in fp64 (exact for bf16 inputs of any one scale, so its order does not show),
// r is its fp64 value rounded once to fp32, and the products and sums after it are single fp32
// operations (no contraction).  The rotated key enters the cache's encoder in fp32: it is rounded
// to no 16-bit type on the way.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4_device.cuh"
#include "kv4_internal.h"
#include "kv4_layout.cuh"
#include "kv4_mixed_encode.cuh"
#include "kv4_quant.cuh"

namespace kv4 {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarpsPerBlock = kThreads / 32;

// Four consecutive elements of any of the three types.
__device__ __forceinline__ void load4_any(const void* base, int dtype, long long i, float (&x)[4]) {
  if (dtype == KV4_F32) {
    load4<float>(base, static_cast<size_t>(i), x);
  } else if (dtype == KV4_BF16) {
    load4<__nv_bfloat16>(base, static_cast<size_t>(i), x);
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(reinterpret_cast<const __half*>(base) + i);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
  }
}

__device__ __forceinline__ void store4_any(void* base, int dtype, long long i, const float (&x)[4]) {
  if (dtype == KV4_F32) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + i) = make_float4(x[0], x[1], x[2], x[3]);
  } else if (dtype == KV4_BF16) {
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(base) + i) =
        make_uint2(pack_bf2(__float2bfloat16_rn(x[0]), __float2bfloat16_rn(x[1])),
                   pack_bf2(__float2bfloat16_rn(x[2]), __float2bfloat16_rn(x[3])));
  } else {
    const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(reinterpret_cast<__half*>(base) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

// ------------------------------------------------------------------ the table

// Thread (pair i, run of kRun positions): the run's first angle by one fp64 sincospi of the turns
// p f / 2 pi reduced exactly, then one fp64 complex product per position (relative error at most
// kRun 2^-52, far below the fp32 rounding of the entries).  Four fp64 multiply-adds an entry instead
// of a sine and a cosine keep the kernel on the memory's side: it writes 8 bytes an entry.
constexpr int kRun = 32;

__device__ __forceinline__ void turn(double p, double g, double* c, double* s) {
  const double hi = p * g;
  const double lo = fma(p, g, -hi);
  sincospi(2.0 * ((hi - rint(hi)) + lo), s, c);
}

__global__ void __launch_bounds__(kThreads) rope_table_kernel(RopeTableArgs a) {
  const int npair = a.R / 2;
  const long long id = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const int i = static_cast<int>(id % npair);
  const long long p0 = id / npair * kRun;
  if (p0 >= a.max_pos) return;
  const double g = a.turns[i];
  double c, s, dc, ds;
  turn(static_cast<double>(p0), g, &c, &s);
  turn(1.0, g, &dc, &ds);
  c *= a.mult;
  s *= a.mult;
  const int n = static_cast<int>(min(static_cast<long long>(kRun), a.max_pos - p0));
  float2* out = a.table + p0 * npair + i;
  for (int k = 0; k < n; ++k) {
    out[static_cast<long long>(k) * npair] = make_float2(static_cast<float>(c), static_cast<float>(s));
    const double cn = fma(c, dc, -s * ds);
    s = fma(s, dc, c * ds);
    c = cn;
  }
}

// ------------------------------------------------------------------ norm and rotation of one vector

// A warp holds one head vector, lane l elements 4l..4l+3 (lanes < D/4).
template <int D>
struct Rotation {
  float c[4], s[4];  // of the lane's elements; s carries the sign of the partner's term
  int src;           // lane of the half layout's partner
  bool on;           // the lane's elements are among the first R
  bool half;

  __device__ __forceinline__ void load(const RopeArgs& a, int pos, int lane) {
    const int R = a.R;
    half = a.layout == KV4_ROPE_HALF;
    on = 4 * lane < R;
    src = lane;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[j] = 1.f;
      s[j] = 0.f;
    }
    if (!on) return;
    const float* row = a.table + static_cast<size_t>(pos) * R;
    if (half) {
      const bool first = 8 * lane < R;
      src = first ? lane + R / 8 : lane - R / 8;
      const float4* t = reinterpret_cast<const float4*>(row + 2 * (first ? 4 * lane : 4 * lane - R / 2));
      const float4 u = __ldg(t), v = __ldg(t + 1);
      const float sg = first ? -1.f : 1.f;
      c[0] = u.x; s[0] = sg * u.y; c[1] = u.z; s[1] = sg * u.w;
      c[2] = v.x; s[2] = sg * v.y; c[3] = v.z; s[3] = sg * v.w;
    } else {
      const float4 u = __ldg(reinterpret_cast<const float4*>(row + 4 * lane));
      c[0] = c[1] = u.x; s[0] = -u.y; s[1] = u.y;
      c[2] = c[3] = u.z; s[2] = -u.w; s[3] = u.w;
    }
  }

  __device__ __forceinline__ void apply(float (&x)[4]) const {
    float o[4];
    if (half) {
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = __shfl_sync(FULL, x[j], src);
    } else {
      o[0] = x[1];
      o[1] = x[0];
      o[2] = x[3];
      o[3] = x[2];
    }
    if (on) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = __fadd_rn(__fmul_rn(x[j], c[j]), __fmul_rn(o[j], s[j]));
    }
  }
};

// 1 / sqrt(ms) rounded to fp32: the hardware's fp32 estimate and one Newton step in fp64 (relative
// error below 1e-13 before the rounding).  ms below or above the fp32 range goes by the fp64 root.
__device__ __forceinline__ float rsqrt_rn(double ms) {
  const float f = static_cast<float>(ms);
  if (f > 1e-37f && f < 1e37f) {
    const double y = static_cast<double>(rsqrtf(f));
    return static_cast<float>(y * fma(-0.5 * ms * y, y, 1.5));
  }
  return static_cast<float>(1.0 / sqrt(ms));
}

// x r w over the warp's D elements.
template <int D>
__device__ __forceinline__ void head_norm(float (&x)[4], const float (&w)[4], double eps) {
  double ss = 0.0;
#pragma unroll
  for (int j = 0; j < 4; ++j) ss = fma(static_cast<double>(x[j]), static_cast<double>(x[j]), ss);
#pragma unroll
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
  const float r = rsqrt_rn(ss * (1.0 / D) + eps);
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = __fmul_rn(__fmul_rn(x[j], r), w[j]);
}

template <int D>
__device__ __forceinline__ void load_weight(const void* w, int dtype, int lane, float (&x)[4]) {
  x[0] = x[1] = x[2] = x[3] = 1.f;
  if (w && lane < D / 4) load4_any(w, dtype, 4 * lane, x);
}

// n (<= kBatch) consecutive vectors, read before the first is worked on: norm, rotation, out.
constexpr int kBatch = 4;
template <int D>
__device__ __forceinline__ void rope_vectors(const RopeArgs& a, const Rotation<D>& rot, const float (&w)[4], bool norm,
                                             const void* in, int in_dt, long long i0, void* out, int out_dt, long long o0,
                                             int n, int lane) {
  const bool act = lane < D / 4;
  float x[kBatch][4];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0.f;
    if (act && u < n) load4_any(in, in_dt, i0 + u * D + 4 * lane, x[u]);
  }
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    if (u >= n) break;
    if (norm) head_norm<D>(x[u], w, a.eps);
    rot.apply(x[u]);
    if (act) store4_any(out, out_dt, o0 + u * D + 4 * lane, x[u]);
  }
}

// ------------------------------------------------------------------ kv4_rope

// Warp (token, run of hpw heads): queries first, then keys.
template <int D>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a, int hpw) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int nq = (a.Hq + hpw - 1) / hpw, nk = (a.Hkv + hpw - 1) / hpw;
  const int gw = static_cast<int>((blockIdx.x * static_cast<unsigned>(kThreads) + threadIdx.x) >> 5);
  const int t = gw / (nq + nk), c = gw - t * (nq + nk);
  if (t >= a.T) return;
  const int pos = a.pos[t];
  if (pos < 0 || pos >= a.max_pos) {
    if (pos != -1 && lane == 0) atomicOr(a.err, KV4_DEVERR_LENGTH);
    return;
  }
  const bool is_q = c < nq;
  const int h0 = (is_q ? c : c - nq) * hpw, h1 = min(h0 + hpw, is_q ? a.Hq : a.Hkv);
  const void* weight = is_q ? a.qw : a.kw;
  Rotation<D> rot;
  rot.load(a, pos, lane);
  float w[4];
  load_weight<D>(weight, a.w_dtype, lane, w);
  const void* in = is_q ? a.q : a.k;
  void* out = is_q ? a.q_out : a.k_out;
  const int idt = is_q ? a.q_dtype : a.k_dtype, odt = is_q ? a.q_out_dtype : a.k_out_dtype;
  const long long i0 = t * (is_q ? a.q_stride : a.k_stride), o0 = t * (is_q ? a.q_out_stride : a.k_out_stride);
  for (int h = h0; h < h1; h += kBatch)
    rope_vectors<D>(a, rot, w, weight != nullptr, in, idt, i0 + h * D, out, odt, o0 + h * D, min(kBatch, h1 - h), lane);
}

// ------------------------------------------------------------------ kv4_append_rope

enum PoolFormat { POOL_INT4, POOL_VBF, POOL_MIXED, POOL_BF16 };

// Where a token's rows go: page and tile of its position (false: the token is left out).
struct Place {
  int b, pos, page;
};

__device__ __forceinline__ bool place_of(const AppendArgs& a, int t, int lane, Place& p) {
  p.b = a.seq_slot[t];
  p.pos = a.pos[t];
  if (p.b == -1) return false;  // a padding row
  if (p.b < 0 || p.b >= a.max_seqs || p.pos < 0 || p.pos / a.P >= a.stride) {
    if (lane == 0) atomicOr(a.err, KV4_DEVERR_LENGTH);
    return false;
  }
  p.page = a.page_table[static_cast<size_t>(p.b) * a.stride + p.pos / a.P];
  if (p.page < 0 || p.page >= a.max_pages) {
    if (lane == 0) atomicOr(a.err, KV4_DEVERR_PAGE_RANGE);
    return false;
  }
  return true;
}

template <int D, int FMT>
constexpr int kPosBytes = FMT == POOL_VBF ? D / 2 + 4 + 2 * D : FMT == POOL_BF16 ? 4 * D : D + 8;

template <int D, int FMT>
__device__ __forceinline__ uint8_t* tile_of(const AppendArgs& a, const Place& p, int g) {
  constexpr int PB = kPosBytes<D, FMT>;
  return a.pool + static_cast<size_t>(p.page) * a.page_bytes + static_cast<size_t>(g) * a.P * PB +
         static_cast<size_t>((p.pos % a.P) >> 4) * (16 * PB);
}

template <int D, int FMT>
__device__ __forceinline__ uint8_t* side_tile_of(const AppendArgs& a, int b, int g, int row) {
  constexpr int T8 = FMT == POOL_VBF ? Geo<D>::T8V : Geo<D>::T8B;
  return a.side + static_cast<size_t>(b) * a.side_slot_bytes + static_cast<size_t>(g) * a.nt8 * T8 +
         static_cast<size_t>(row >> 4) * T8;
}

// The key of one (token, KV head), normed and rotated, into the page and the side row (-1: none).
template <int D, int FMT>
__device__ __forceinline__ void put_key(const AppendArgs& a, const Place& p, int g, int row, int lane, float (&k)[4]) {
  const bool act = lane < D / 4;
  uint8_t* tile = tile_of<D, FMT>(a, p, g);
  const int r = p.pos & 15;  // pages are multiples of 16 positions
  if constexpr (FMT == POOL_BF16) {
    if (act)
      *reinterpret_cast<uint2*>(kbf_unit<D>(tile, r, lane)) =
          make_uint2(pack_bf2(__float2bfloat16_rn(k[0]), __float2bfloat16_rn(k[1])),
                     pack_bf2(__float2bfloat16_rn(k[2]), __float2bfloat16_rn(k[3])));
  } else {
    flip_signs4(k, lane, a.signs);
    hadamard4(k, lane, a.h);
    uint32_t sz;
    bool bad;
    const uint32_t kc = quant_int4(k, act, &sz, &bad);
    if (act) store_k4<D>(tile, r, lane, kc);
    if (lane == 0) *reinterpret_cast<uint32_t*>(tile + (FMT == POOL_VBF ? 8 * D : 16 * D) + 4 * r) = sz;
    bool bad8 = false;
    if (row >= 0) {
      uint8_t* t8 = side_tile_of<D, FMT>(a, p.b, g, row);
      uint16_t sc;
      const uint32_t k8 = quant_int8(k, act, &sc, &bad8);
      if (act) *k8_word<D>(t8, row & 15, lane) = k8;
      if (lane == 0) *reinterpret_cast<uint16_t*>(t8 + 16 * D + 2 * (row & 15)) = sc;
    }
    if (lane == 0 && (bad || bad8)) atomicOr(a.err, KV4_DEVERR_RANGE);
  }
}

template <int D, int FMT>
__device__ __forceinline__ void put_value(const AppendArgs& a, const Place& p, int g, int row, int lane, float (&v)[4]) {
  const bool act = lane < D / 4;
  uint8_t* tile = tile_of<D, FMT>(a, p, g);
  const int r = p.pos & 15;
  if constexpr (FMT == POOL_BF16) {
    if (act) store_vbf<D>(tile + 32 * D, r, lane, v);
  } else if constexpr (FMT == POOL_VBF) {
    if (act) store_vbf<D>(tile + Geo<D>::VBO, r, lane, v);
    if (act && row >= 0) store_vbf<D>(side_tile_of<D, FMT>(a, p.b, g, row) + Geo<D>::VB8O, row & 15, lane, v);
  } else {
    if (a.rotate_v) {
      flip_signs4(v, lane, a.signs);
      hadamard4(v, lane, a.h);
    }
    uint32_t sz;
    bool bad, bad8 = false;
    const uint32_t vc = quant_int4(v, act, &sz, &bad);
    if (act) *v4_chunk<D>(tile, r, lane) = static_cast<uint16_t>(vc);
    if (lane == 0) *reinterpret_cast<uint32_t*>(tile + 16 * D + 64 + 4 * r) = sz;
    if (row >= 0) {
      uint8_t* vb = side_tile_of<D, FMT>(a, p.b, g, row) + Geo<D>::H8B;
      uint16_t sc;
      const uint32_t v8 = quant_int8(v, act, &sc, &bad8);
      if (act) {
#pragma unroll
        for (int i = 0; i < 4; ++i) vb[v8_offset<D>(row & 15, 4 * lane + i)] = static_cast<uint8_t>(v8 >> (8 * i));
      }
      if (lane == 0) *reinterpret_cast<uint16_t*>(vb + 16 * D + 2 * (row & 15)) = sc;
    }
    if (lane == 0 && (bad || bad8)) atomicOr(a.err, KV4_DEVERR_RANGE);
  }
}

// Warp (token, item): items are runs of hpw query heads, then the KV heads' keys, then their values
// (mixed bit-width keys: key and value of a KV head together, they share a row record).
template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) append_rope_kernel(RopeArgs q, AppendArgs a, int hpw) {
  constexpr int NI = D / 32;
  __shared__ uint32_t rows[FMT == POOL_MIXED ? kWarpsPerBlock : 1][2][kMixedRowWords<D>];
  __shared__ float xs[FMT == POOL_MIXED ? kWarpsPerBlock : 1][D];
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const bool act = lane < D / 4;
  const int nq = (q.Hq + hpw - 1) / hpw, per = nq + (FMT == POOL_MIXED ? a.Hkv : 2 * a.Hkv);
  const int gw = static_cast<int>((blockIdx.x * static_cast<unsigned>(kThreads) + threadIdx.x) >> 5);
  const int t = gw / per, c = gw - t * per;
  if (t >= a.T) return;
  Place p;
  if (!place_of(a, t, lane, p)) return;
  if (p.pos >= q.max_pos) {
    if (lane == 0) atomicOr(a.err, KV4_DEVERR_LENGTH);
    return;
  }
  Rotation<D> rot;
  float w[4];
  if (c < nq) {
    rot.load(q, p.pos, lane);
    load_weight<D>(q.qw, q.w_dtype, lane, w);
    const int h1 = min((c + 1) * hpw, q.Hq);
    for (int h = c * hpw; h < h1; h += kBatch)
      rope_vectors<D>(q, rot, w, q.qw != nullptr, q.q, q.q_dtype, t * q.q_stride + h * D, q.q_out, q.q_out_dtype,
                      t * q.q_out_stride + h * D, min(kBatch, h1 - h), lane);
    return;
  }
  const bool is_k = FMT == POOL_MIXED || c < nq + a.Hkv;
  const int g = is_k ? c - nq : c - nq - a.Hkv;
  const int row = FMT <= POOL_VBF ? side_row(p.pos, a.s, a.w, a.w > 0 && p.pos >= a.s ? a.lens_after[p.b] : 0) : -1;
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if (is_k) {
    if (act) load4_any(q.k, q.k_dtype, t * q.k_stride + g * D + 4 * lane, x);
    rot.load(q, p.pos, lane);
    load_weight<D>(q.kw, q.w_dtype, lane, w);
    if (q.kw) head_norm<D>(x, w, q.eps);
    rot.apply(x);
    if constexpr (FMT == POOL_MIXED) {
      // the encoder's lanes hold coordinates l + 32 i
      const int warp = threadIdx.x >> 5;
      float k[NI], v[NI];
      if (act) *reinterpret_cast<float4*>(&xs[warp][4 * lane]) = make_float4(x[0], x[1], x[2], x[3]);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        k[i] = xs[warp][lane + 32 * i];
        v[i] = load_elem(q.v, q.v_dtype, static_cast<size_t>(t * q.v_stride + g * D + lane + 32 * i));
      }
      mixed_encode_store<D>(a, g, p.page, p.pos, lane, k, v, rows[warp][0], rows[warp][1]);
    } else {
      put_key<D, FMT>(a, p, g, row, lane, x);
    }
  } else if constexpr (FMT != POOL_MIXED) {
    if (act) load4_any(q.v, q.v_dtype, t * q.v_stride + g * D + 4 * lane, x);
    put_value<D, FMT>(a, p, g, row, lane, x);
  }
}

// ------------------------------------------------------------------ kv4_gather

// Inverse of the stored rotation: diag(s) H x / h.
template <int D>
__device__ __forceinline__ void unrotate4(const AppendArgs& a, int lane, float (&x)[4]) {
  if (a.h > 1) {
    hadamard4(x, lane, a.h);
    const float ih = 1.f / static_cast<float>(a.h);  // a power of two: exact
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] *= ih;
  }
  flip_signs4(x, lane, a.signs);
}

__device__ __forceinline__ float2 scale_zero(const uint8_t* p) {
  const uint32_t sz = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__half2float(__ushort_as_half(static_cast<unsigned short>(sz & 0xffffu))),
                     __half2float(__ushort_as_half(static_cast<unsigned short>(sz >> 16))));
}

// Codes of `w` bits at bit `o` of a row of 32-bit words.
__device__ __forceinline__ uint32_t get_bits(const uint32_t* row, int o, int w) {
  if (w == 0) return 0u;
  const int wi = o >> 5, sh = o & 31;
  uint32_t x = row[wi] >> sh;
  if (sh + w > 32) x |= row[wi + 1] << (32 - sh);
  return x & ((1u << w) - 1u);
}

template <int D>
__device__ __forceinline__ void read_vbf(const uint8_t* vblock, int r, int lane, float (&x)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    x[j] = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(vblock + vbf_offset<D>(r, 4 * lane + j)));
}

// Key (or value) of one (token, KV head) as fp32, in its original basis.
template <int D, int FMT>
__device__ __forceinline__ void read_key(const AppendArgs& a, const Place& p, int g, int row, int lane, float (&x)[4]) {
  const bool act = lane < D / 4;
  if constexpr (FMT == POOL_MIXED) {
    const int KR = a.kbits * D / 8, VR = a.vbits * D / 8, pp = p.pos % a.P, rr = pp & 15;
    const uint8_t* slice = a.pool + static_cast<size_t>(p.page) * a.page_bytes +
                           static_cast<size_t>(g) * static_cast<size_t>(a.P) * (KR + VR + 8) +
                           static_cast<size_t>(pp >> 4) * 16 * (KR + VR + 8);
    const float ks = scale_zero(slice + 16 * (KR + VR) + 8 * rr).x;
    const float* sig = rec_sigma<D>(a.alloc, g);
    const uint8_t* wid = rec_width<D>(a.alloc, g);
    int w[4] = {0, 0, 0, 0}, sum = 0;
    if (act) {
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += w[j] = wid[(4 * lane + j) % (D / 2)];
    }
    int o = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(FULL, o, d);
      if (lane >= d) o += y;
    }
    o -= sum;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(slice + static_cast<size_t>(rr) * KR);
    if (act) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t c = get_bits(src, o, w[j]);
        o += w[j];
        const float mid = __fadd_rn(static_cast<float>(2u * c + 1u) * (1.f / static_cast<float>(1 << w[j])), -1.f);
        x[j] = w[j] ? __fmul_rn(__fmul_rn(ks, sig[(4 * lane + j) % (D / 2)]), mid) : 0.f;
      }
    }
  } else {
    if (row >= 0) {
      const uint8_t* t8 = side_tile_of<D, FMT>(a, p.b, g, row);
      const float sc = __half2float(*reinterpret_cast<const __half*>(t8 + 16 * D + 2 * (row & 15)));
      if (act) {
        const uint32_t c = *k8_word<D>(const_cast<uint8_t*>(t8), row & 15, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = sc * static_cast<float>(static_cast<int8_t>(c >> (8 * j)));
      }
    } else {
      uint8_t* tile = tile_of<D, FMT>(a, p, g);
      const int r = p.pos & 15;
      if constexpr (FMT == POOL_BF16) {
        if (act) load4<__nv_bfloat16>(kbf_unit<D>(tile, r, lane), 0, x);
      } else {
        const float2 sz = scale_zero(tile + (FMT == POOL_VBF ? 8 * D : 16 * D) + 4 * r);
        if (act) {
          const uint32_t* wd = k4_words<D>(tile, r & 7, lane);
          const int sh = 16 * (lane & 1) + 4 * (r >> 3);
          const uint32_t e = wd[0] >> sh, o = wd[1] >> sh;
          x[0] = fmaf(sz.x, static_cast<float>(e & 15u), sz.y);
          x[1] = fmaf(sz.x, static_cast<float>(o & 15u), sz.y);
          x[2] = fmaf(sz.x, static_cast<float>((e >> 8) & 15u), sz.y);
          x[3] = fmaf(sz.x, static_cast<float>((o >> 8) & 15u), sz.y);
        }
      }
    }
    if constexpr (FMT != POOL_BF16) unrotate4<D>(a, lane, x);
  }
}

template <int D, int FMT>
__device__ __forceinline__ void read_value(const AppendArgs& a, const Place& p, int g, int row, int lane, float (&x)[4]) {
  const bool act = lane < D / 4;
  if constexpr (FMT == POOL_MIXED) {
    const int KR = a.kbits * D / 8, VR = a.vbits * D / 8, pp = p.pos % a.P, rr = pp & 15;
    const uint8_t* slice = a.pool + static_cast<size_t>(p.page) * a.page_bytes +
                           static_cast<size_t>(g) * static_cast<size_t>(a.P) * (KR + VR + 8) +
                           static_cast<size_t>(pp >> 4) * 16 * (KR + VR + 8);
    const float2 zr = scale_zero(slice + 16 * (KR + VR) + 8 * rr + 4);  // zero, range
    const float step = __fdiv_rn(zr.y, static_cast<float>((1 << a.vbits) - 1));
    const uint32_t* src = reinterpret_cast<const uint32_t*>(slice + 16 * static_cast<size_t>(KR) + static_cast<size_t>(rr) * VR);
    if (act) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[j] = fmaf(step, static_cast<float>(get_bits(src, (4 * lane + j) * a.vbits, a.vbits)), zr.x);
    }
  } else if (FMT != POOL_BF16 && row >= 0) {
    const uint8_t* t8 = side_tile_of<D, FMT>(a, p.b, g, row);
    if constexpr (FMT == POOL_VBF) {
      if (act) read_vbf<D>(t8 + Geo<D>::VB8O, row & 15, lane, x);
    } else {
      const uint8_t* vb = t8 + Geo<D>::H8B;
      const float sc = __half2float(*reinterpret_cast<const __half*>(vb + 16 * D + 2 * (row & 15)));
      if (act) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = sc * static_cast<float>(static_cast<int8_t>(vb[v8_offset<D>(row & 15, 4 * lane + j)]));
      }
    }
  } else {
    uint8_t* tile = tile_of<D, FMT>(a, p, g);
    const int r = p.pos & 15;
    if constexpr (FMT == POOL_BF16) {
      if (act) read_vbf<D>(tile + 32 * D, r, lane, x);
    } else if constexpr (FMT == POOL_VBF) {
      if (act) read_vbf<D>(tile + Geo<D>::VBO, r, lane, x);
    } else {
      const float2 sz = scale_zero(tile + 16 * D + 64 + 4 * r);
      if (act) {
        const uint32_t c = *v4_chunk<D>(tile, r, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = fmaf(sz.x, static_cast<float>((c >> (4 * j)) & 15u), sz.y);
      }
    }
  }
  if (FMT == POOL_INT4 && a.rotate_v) unrotate4<D>(a, lane, x);
}

// Warp (token, KV head).
template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) gather_kernel(AppendArgs a, void* k_out, void* v_out, int dtype) {
  const int lane = threadIdx.x & 31;
  const int gw = static_cast<int>((blockIdx.x * static_cast<unsigned>(kThreads) + threadIdx.x) >> 5);
  const int t = gw / a.Hkv, g = gw - t * a.Hkv;
  if (t >= a.T) return;
  Place p;
  if (!place_of(a, t, lane, p)) return;
  int row = -1;
  if (a.lens_after) {
    const int L = a.lens_after[p.b];
    if (p.pos >= L) {
      if (lane == 0) atomicOr(a.err, KV4_DEVERR_LENGTH);
      return;
    }
    if (FMT <= POOL_VBF) row = side_row(p.pos, a.s, a.w, L);
  }
  const long long o = (static_cast<long long>(t) * a.Hkv + g) * D + 4 * lane;
  float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
  if (k_out) read_key<D, FMT>(a, p, g, row, lane, x);
  if (v_out) read_value<D, FMT>(a, p, g, row, lane, y);
  if (lane < D / 4) {
    if (k_out) store4_any(k_out, dtype, o, x);
    if (v_out) store4_any(v_out, dtype, o, y);
  }
}

unsigned blocks_for(long long warps) { return static_cast<unsigned>((warps + kWarpsPerBlock - 1) / kWarpsPerBlock); }

// Query heads a warp takes: one while the launch has fewer warps than the GPU holds (the latency
// counts), a batch of four loads in flight otherwise.
int heads_per_warp(long long vectors) { return vectors > 148LL * 64 ? kBatch : 1; }

}  // namespace

cudaError_t launch_rope_table(const RopeTableArgs& a, cudaStream_t st) {
  const long long threads = (a.max_pos + kRun - 1) / kRun * (a.R / 2);
  note_launches(1);
  rope_table_kernel<<<static_cast<unsigned>((threads + kThreads - 1) / kThreads), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_rope(const RopeArgs& a, int D, cudaStream_t st) {
  const int hpw = heads_per_warp(static_cast<long long>(a.T) * (a.Hq + a.Hkv));
  const unsigned grid = blocks_for(static_cast<long long>(a.T) * ((a.Hq + hpw - 1) / hpw + (a.Hkv + hpw - 1) / hpw));
  note_launches(1);
  if (D == 128) rope_kernel<128><<<grid, kThreads, 0, st>>>(a, hpw);
  else rope_kernel<64><<<grid, kThreads, 0, st>>>(a, hpw);
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_append_rope_d(const RopeArgs& q, const AppendArgs& a, int format, cudaStream_t st) {
  const int hpw = heads_per_warp(static_cast<long long>(a.T) * (q.Hq + 2 * a.Hkv));
  const int per = (q.Hq + hpw - 1) / hpw + (format == POOL_MIXED ? a.Hkv : 2 * a.Hkv);
  const unsigned grid = blocks_for(static_cast<long long>(a.T) * per);
  note_launches(1);
  switch (format) {
    case POOL_INT4: append_rope_kernel<D, POOL_INT4><<<grid, kThreads, 0, st>>>(q, a, hpw); break;
    case POOL_VBF: append_rope_kernel<D, POOL_VBF><<<grid, kThreads, 0, st>>>(q, a, hpw); break;
    case POOL_MIXED: append_rope_kernel<D, POOL_MIXED><<<grid, kThreads, 0, st>>>(q, a, hpw); break;
    default: append_rope_kernel<D, POOL_BF16><<<grid, kThreads, 0, st>>>(q, a, hpw); break;
  }
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_gather_d(const AppendArgs& a, int format, void* k_out, void* v_out, int dtype, cudaStream_t st) {
  const unsigned grid = blocks_for(static_cast<long long>(a.T) * a.Hkv);
  note_launches(1);
  switch (format) {
    case POOL_INT4: gather_kernel<D, POOL_INT4><<<grid, kThreads, 0, st>>>(a, k_out, v_out, dtype); break;
    case POOL_VBF: gather_kernel<D, POOL_VBF><<<grid, kThreads, 0, st>>>(a, k_out, v_out, dtype); break;
    case POOL_MIXED: gather_kernel<D, POOL_MIXED><<<grid, kThreads, 0, st>>>(a, k_out, v_out, dtype); break;
    default: gather_kernel<D, POOL_BF16><<<grid, kThreads, 0, st>>>(a, k_out, v_out, dtype); break;
  }
  return cudaGetLastError();
}

static int pool_format(const AppendArgs& a, bool bf16_pool) {
  return bf16_pool ? POOL_BF16 : a.alloc ? POOL_MIXED : a.vbf ? POOL_VBF : POOL_INT4;
}

cudaError_t launch_append_rope(const RopeArgs& q, const AppendArgs& a, int D, bool bf16_pool, cudaStream_t st) {
  const int f = pool_format(a, bf16_pool);
  return D == 128 ? launch_append_rope_d<128>(q, a, f, st) : launch_append_rope_d<64>(q, a, f, st);
}

cudaError_t launch_gather(const AppendArgs& a, int D, bool bf16_pool, void* k_out, void* v_out, int dtype, cudaStream_t st) {
  const int f = pool_format(a, bf16_pool);
  return D == 128 ? launch_gather_d<128>(a, f, k_out, v_out, dtype, st) : launch_gather_d<64>(a, f, k_out, v_out, dtype, st);
}

}  // namespace kv4
