// kv4_rope.cu -- rotary positions up to the cache: the cos/sin table, the per-head norm and rotation
// of queries and keys (kv4_rope), the same fused with the append of any cache format
// (kv4_append_rope), and the cache read back as dense keys and values (kv4_gather).
//
// Mathematics.  Pair i of a head at position p turns by the angle p f_i:
//   (a, b) -> (a cos - b sin, b cos + a sin),
// (a, b) = elements (i, i + R/2) (KV4_ROPE_HALF) or (2i, 2i + 1) (KV4_ROPE_INTERLEAVED) of the first
// R elements; the others pass.  Before it, with a weight, x_j -> x_j r w_j, r = 1 / sqrt(mean x^2 + eps).
// Every step is a single fp32 operation in a fixed order (no contraction; the sum of squares is a
// binary tree over the elements, the root IEEE-rounded), so that the codes an append writes do not
// depend on the launch.  A sum in fp64 was 550 cycles of dependent latency a vector and the kernel's
// bound (160 us for what the tree does in 131).  The rotated key enters the cache's encoder in fp32: it
// is rounded to no 16-bit type on the way.
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

// Eight consecutive elements of any of the three types (16-bit: one 16-byte access).
__device__ __forceinline__ void load8(const void* base, int dtype, long long i, float (&x)[8]) {
  if (dtype == KV4_F32) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + i);
    const float4 u = p[0], v = p[1];
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    return;
  }
  const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + i;
  uint32_t w[4];
  if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else {  // rows of a fused projection may start on 8 bytes
    const uint2 u = *reinterpret_cast<const uint2*>(p), v = *reinterpret_cast<const uint2*>(p + 4);
    w[0] = u.x; w[1] = u.y; w[2] = v.x; w[3] = v.y;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (dtype == KV4_BF16) {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      x[2 * j] = f.x;
      x[2 * j + 1] = f.y;
    }
  }
}

__device__ __forceinline__ void store8(void* base, int dtype, long long i, const float (&x)[8]) {
  if (dtype == KV4_F32) {
    float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + i);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (dtype == KV4_BF16) {
      w[j] = pack_bf2_rn(x[2 * j], x[2 * j + 1]);
    } else {
      const __half2 h = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  uint16_t* p = reinterpret_cast<uint16_t*>(base) + i;
  if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(p + 4) = make_uint2(w[2], w[3]);
  }
}

// ------------------------------------------------------------------ the table

// Thread (pair i, run of kRun positions): the run's first angle by one fp64 sincospi of the turns
// p f / 2 pi reduced exactly, then one fp64 complex product per position.  Absolute errors before the
// rounding to fp32: 2^-50 p f by the turns (at most 7 fp64 roundings), 2^-45 by the products (each below
// 7 2^-53).  Four fp64 multiply-adds an entry instead
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

// D / 8 lanes hold one head vector, lane gl of the group elements 8 gl..8 gl + 7; a warp takes kPerWarp
// vectors (heads of one token) at once: sixteen bytes a lane and half the shuffles of a vector spread
// over the whole warp (the norm and rotation of 16383 tokens: 207 -> 160 us).
template <int D>
constexpr int kLanes = D / 8;
template <int D>
constexpr int kPerWarp = 32 / kLanes<D>;

template <int D>
struct Rotation {
  float c[8], s[8];   // of the lane's elements; s carries the sign of the partner's term
  int src_lo, src_hi; // lanes of the half layout's partners of elements 0..3 and 4..7
  bool on;            // the lane's elements are among the first R
  bool half, cross;   // half layout; its partner is four elements off (R / 2 not a multiple of 8)

  __device__ __forceinline__ void load(const RopeArgs& a, int pos, int lane) {
    const int R = a.R, gl = lane % kLanes<D>, base = lane - gl;
    half = a.layout == KV4_ROPE_HALF;
    cross = ((R / 2) & 7) != 0;
    on = 8 * gl < R;
    src_lo = src_hi = lane;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = 1.f;
      s[j] = 0.f;
    }
    if (!on) return;
    const float* row = a.table + static_cast<size_t>(pos) * R;
    if (half) {
      const int m = R / 16;
      const bool f0 = 16 * gl < R, f1 = 16 * gl + 8 < R;  // elements 0..3 and 4..7 are in the first half
      src_lo = base + (f0 ? gl + m : gl - m - (cross ? 1 : 0));
      src_hi = base + (f1 ? gl + m + (cross ? 1 : 0) : gl - m);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const bool first = q ? f1 : f0;
        const int i = 8 * gl + 4 * q;
        const float4* t = reinterpret_cast<const float4*>(row + 2 * (first ? i : i - R / 2));
        const float4 u = __ldg(t), v = __ldg(t + 1);
        const float sg = first ? -1.f : 1.f;
        c[4 * q] = u.x; s[4 * q] = sg * u.y; c[4 * q + 1] = u.z; s[4 * q + 1] = sg * u.w;
        c[4 * q + 2] = v.x; s[4 * q + 2] = sg * v.y; c[4 * q + 3] = v.z; s[4 * q + 3] = sg * v.w;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(row + 8 * gl + 4 * q));
        c[4 * q] = c[4 * q + 1] = u.x; s[4 * q] = -u.y; s[4 * q + 1] = u.y;
        c[4 * q + 2] = c[4 * q + 3] = u.z; s[4 * q + 2] = -u.w; s[4 * q + 3] = u.w;
      }
    }
  }

  __device__ __forceinline__ void apply(float (&x)[8]) const {
    float o[8];
    if (!half) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = x[j ^ 1];
    } else if (!cross) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = __shfl_sync(FULL, x[j], j < 4 ? src_lo : src_hi);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = __shfl_sync(FULL, x[j ^ 4], j < 4 ? src_lo : src_hi);
    }
    if (on) {
      // (as packed pairs the products and the sum were fused, against their .rn)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __fadd_rn(__fmul_rn(x[j], c[j]), __fmul_rn(o[j], s[j]));
    }
  }
};

// x r w over the group's D elements.  The squares are summed as a binary tree over the elements in
// order (neighbours first), in the lane and then across the group.
template <int D>
__device__ __forceinline__ void head_norm(float (&x)[8], const float (&w)[8], float eps) {
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; j += 2) unpack2(mul2(pack2(x[j], x[j + 1]), pack2(x[j], x[j + 1])), s[j], s[j + 1]);
  float ss = __fadd_rn(__fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3])), __fadd_rn(__fadd_rn(s[4], s[5]), __fadd_rn(s[6], s[7])));
#pragma unroll
  for (int o = 1; o < kLanes<D>; o <<= 1) ss = __fadd_rn(ss, __shfl_xor_sync(FULL, ss, o));
  const float r = __frsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.0f / D), eps));
  const uint64_t r2 = pack2(r, r);
#pragma unroll
  for (int j = 0; j < 8; j += 2) unpack2(mul2(mul2(pack2(x[j], x[j + 1]), r2), pack2(w[j], w[j + 1])), x[j], x[j + 1]);
}

template <int D>
__device__ __forceinline__ void load_weight(const void* w, int dtype, int lane, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = 1.f;
  if (w) load8(w, dtype, 8 * (lane % kLanes<D>), x);
}

// Eight 16-bit elements to and from fp32.
__device__ __forceinline__ void widen8(const uint4& u, bool bf16, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (bf16) {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      x[2 * j] = f.x;
      x[2 * j + 1] = f.y;
    }
  }
}
__device__ __forceinline__ uint4 narrow8(const float (&x)[8], bool bf16) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (bf16) {
      w[j] = pack_bf2_rn(x[2 * j], x[2 * j + 1]);
    } else {
      const __half2 h = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Both sides 16-bit with 16-byte rows (what a projection's output is).
__host__ __device__ inline bool rows16(const void* in, int in_dt, long long in_stride, const void* out, int out_dt, long long out_stride) {
  return in_dt != KV4_F32 && out_dt != KV4_F32 && ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15) == 0 &&
         ((in_stride | out_stride) & 7) == 0;
}

// Heads h0.. (below h1) of one token: norm, rotation, out.  fast (rows16): the loads of BATCH warp
// passes of kPerWarp heads are issued before the first is worked on.  kv4_rope takes four (64 bytes a
// lane in flight; 16383 tokens of 32 + 8 heads: 131 us with one, 111 with four).  The append takes
// two, for its registers.
constexpr int kRunPasses = 8;  // passes of a warp when there are many heads
template <int D, int BATCH>
__device__ __forceinline__ void rope_heads(const RopeArgs& a, const Rotation<D>& rot, const float (&w)[8], bool norm, const void* in,
                                           int in_dt, long long i0, void* out, int out_dt, long long o0, int h0, int h1, bool fast, int lane) {
  const int mine = lane / kLanes<D>, e = 8 * (lane % kLanes<D>);
  if (fast) {
    const uint16_t* src = reinterpret_cast<const uint16_t*>(in) + i0 + e;
    uint16_t* dst = reinterpret_cast<uint16_t*>(out) + o0 + e;
    const bool bi = in_dt == KV4_BF16, bo = out_dt == KV4_BF16;
    for (int h = h0 + mine; h - mine < h1; h += BATCH * kPerWarp<D>) {
      uint4 raw[BATCH];
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        const int k = h + u * kPerWarp<D>;
        raw[u] = k < h1 ? __ldcs(reinterpret_cast<const uint4*>(src + k * D)) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        const int k = h + u * kPerWarp<D>;
        if (k - mine >= h1) break;
        float x[8];
        widen8(raw[u], bi, x);
        if (norm) head_norm<D>(x, w, a.eps);
        rot.apply(x);
        if (k < h1) *reinterpret_cast<uint4*>(dst + k * D) = narrow8(x, bo);
      }
    }
    return;
  }
#pragma unroll 1
  for (int h = h0 + mine; h - mine < h1; h += kPerWarp<D>) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0.f;
    if (h < h1) load8(in, in_dt, i0 + h * D + e, x);
    if (norm) head_norm<D>(x, w, a.eps);
    rot.apply(x);
    if (h < h1) store8(out, out_dt, o0 + h * D + e, x);
  }
}

// ------------------------------------------------------------------ kv4_rope

// Warp (token, run of hpw heads): queries first, then keys.  Four blocks an SM (64 registers, 128
// bytes a thread spilled) hide more of the loads' latency than three (80): 97 -> 92 us for 16383 tokens of 32 + 8
// heads in bf16, 3.7 TB/s of the 6.55 a copy reaches.  What is left is issue (66 M warp
// instructions, 2.7 a cycle an SM, are 59 us at four a cycle, above the 52 of the bytes) and latency: types,
// layout and norm are branches at run time around arrays held in registers, and a norm's tree, its root
// and its products depend on one another.
template <int D>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(RopeArgs a, int hpw) {
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
  float w[8];
  load_weight<D>(weight, a.w_dtype, lane, w);
  rope_heads<D, 4>(a, rot, w, weight != nullptr, is_q ? a.q : a.k, is_q ? a.q_dtype : a.k_dtype, t * (is_q ? a.q_stride : a.k_stride),
                is_q ? a.q_out : a.k_out, is_q ? a.q_out_dtype : a.k_out_dtype, t * (is_q ? a.q_out_stride : a.k_out_stride), h0, h1,
                is_q ? a.q_fast : a.k_fast, lane);
}

// ------------------------------------------------------------------ kv4_append_rope

enum PoolFormat { POOL_INT4, POOL_VBF, POOL_MIXED, POOL_BF16 };

// Where a token's rows go: page and tile of its position (false: the token is left out).
struct Place {
  int b, pos, page;
};

// Page-table column of a position, and the position in its page: by shift where P is a power of two.
__device__ __forceinline__ int page_of(const AppendArgs& a, int pos) { return a.p_shift >= 0 ? pos >> a.p_shift : pos / a.P; }
__device__ __forceinline__ int in_page(const AppendArgs& a, int pos) { return a.p_shift >= 0 ? pos & (a.P - 1) : pos % a.P; }

__device__ __forceinline__ bool place_of(const AppendArgs& a, int t, int lane, Place& p) {
  p.b = a.seq_slot[t];
  p.pos = a.pos[t];
  if (p.b == -1) return false;  // a padding row
  if (p.b < 0 || p.b >= a.max_seqs || p.pos < 0 || page_of(a, p.pos) >= a.stride) {
    if (lane == 0) atomicOr(a.err, KV4_DEVERR_LENGTH);
    return false;
  }
  p.page = a.page_table[static_cast<size_t>(p.b) * a.stride + page_of(a, p.pos)];
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
         static_cast<size_t>(in_page(a, p.pos) >> 4) * (16 * PB);
}

template <int D, int FMT>
__device__ __forceinline__ uint8_t* side_tile_of(const AppendArgs& a, int b, int g, int row) {
  constexpr int T8 = FMT == POOL_VBF ? Geo<D>::T8V : Geo<D>::T8B;
  return a.side + static_cast<size_t>(b) * a.side_slot_bytes + static_cast<size_t>(g) * a.nt8 * T8 +
         static_cast<size_t>(row >> 4) * T8;
}

// The key of one (token, KV head), normed and rotated, into the page and the side row (-1: none), by its
// lane group; act: the group has a head (the others take part in the shuffles).
template <int D, int FMT>
__device__ __forceinline__ void put_key(const AppendArgs& a, const Place& p, int g, int row, int gl, bool act, float (&k)[8]) {
  uint8_t* tile = tile_of<D, FMT>(a, p, g);
  const int r = p.pos & 15;  // pages are multiples of 16 positions
  if constexpr (FMT == POOL_BF16) {
    if (act) {
      // both 4-element halves of the lane are in one 16-byte unit
      uint4 w;
      w.x = pack_bf2_rn(k[0], k[1]);
      w.y = pack_bf2_rn(k[2], k[3]);
      w.z = pack_bf2_rn(k[4], k[5]);
      w.w = pack_bf2_rn(k[6], k[7]);
      *reinterpret_cast<uint4*>(kbf_unit<D>(tile, r, 2 * gl)) = w;
    }
  } else {
    flip_signs8(k, gl, a.signs);
    hadamard8(k, gl, a.h);
    uint32_t sz;
    bool bad, bad8 = false;
    const uint32_t kc = quant_int4_8<D>(k, &sz, &bad);
    if (act) {
      store_k4_8<D>(tile, r, gl, kc);
      if (gl == 0) *reinterpret_cast<uint32_t*>(tile + (FMT == POOL_VBF ? 8 * D : 16 * D) + 4 * r) = sz;
    }
    if (row >= 0) {
      uint16_t sc;
      const uint2 k8 = quant_int8_8<D>(k, &sc, &bad8);
      if (act) {
        uint8_t* t8 = side_tile_of<D, FMT>(a, p.b, g, row);
        *reinterpret_cast<uint2*>(k8_word<D>(t8, row & 15, 2 * gl)) = k8;
        if (gl == 0) *reinterpret_cast<uint16_t*>(t8 + 16 * D + 2 * (row & 15)) = sc;
      }
    }
    if (act && gl == 0 && (bad || bad8)) atomicOr(a.err, KV4_DEVERR_RANGE);
  }
}

template <int D, int FMT>
__device__ __forceinline__ void put_value(const AppendArgs& a, const Place& p, int g, int row, int gl, bool act, float (&v)[8]) {
  uint8_t* tile = tile_of<D, FMT>(a, p, g);
  const int r = p.pos & 15;
  if constexpr (FMT == POOL_BF16) {
    if (act) store_vbf_8<D>(tile + 32 * D, r, gl, v);
  } else if constexpr (FMT == POOL_VBF) {
    if (act) store_vbf_8<D>(tile + Geo<D>::VBO, r, gl, v);
    if (act && row >= 0) store_vbf_8<D>(side_tile_of<D, FMT>(a, p.b, g, row) + Geo<D>::VB8O, row & 15, gl, v);
  } else {
    if (a.rotate_v) {
      flip_signs8(v, gl, a.signs);
      hadamard8(v, gl, a.h);
    }
    uint32_t sz;
    bool bad, bad8 = false;
    const uint32_t vc = quant_int4_8<D>(v, &sz, &bad);
    if (act) {
      *v4_chunk<D>(tile, r, 2 * gl) = static_cast<uint16_t>(vc);
      *v4_chunk<D>(tile, r, 2 * gl + 1) = static_cast<uint16_t>(vc >> 16);
      if (gl == 0) *reinterpret_cast<uint32_t*>(tile + 16 * D + 64 + 4 * r) = sz;
    }
    if (row >= 0) {
      uint16_t sc;
      const uint2 v8 = quant_int8_8<D>(v, &sc, &bad8);
      if (act) {
        uint8_t* vb = side_tile_of<D, FMT>(a, p.b, g, row) + Geo<D>::H8B;
#pragma unroll
        for (int e = 0; e < 8; ++e) vb[v8_offset<D>(row & 15, 8 * gl + e)] = static_cast<uint8_t>((e < 4 ? v8.x : v8.y) >> (8 * (e & 3)));
        if (gl == 0) *reinterpret_cast<uint16_t*>(vb + 16 * D + 2 * (row & 15)) = sc;
      }
    }
    if (act && gl == 0 && (bad || bad8)) atomicOr(a.err, KV4_DEVERR_RANGE);
  }
}

// Warp (token, item): items are runs of hpw query heads, then passes of kPerWarp KV heads: the key and
// the value of each together with `joint` (one prologue and both loads in flight; many tokens), else
// keys and values apart (few tokens: the latency counts).  Mixed bit-width keys: one KV head an item,
// key and value share a record.  Four blocks an SM, as in rope_kernel: an encoder is a chain of
// shuffles, a division and the codes' packing, and more warps hide more of it (14460 tokens of 32 + 8
// heads: 181 us with three, 169 with four, 175 with five and their spills; 161 with four and two query
// loads in flight instead of four; 2.3 instructions a cycle).
template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 4) append_rope_kernel(RopeArgs q, AppendArgs a, int hpw, bool joint) {
  constexpr int NI = D / 32, HP = FMT == POOL_MIXED ? 1 : kPerWarp<D>;
  __shared__ uint32_t rows[FMT == POOL_MIXED ? kWarpsPerBlock : 1][2][kMixedRowWords<D>];
  __shared__ float xs[FMT == POOL_MIXED ? kWarpsPerBlock : 1][D];
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, gl = lane % kLanes<D>, mine = lane / kLanes<D>;
  const int nq = (q.Hq + hpw - 1) / hpw, nkv = (a.Hkv + HP - 1) / HP, per = nq + (FMT == POOL_MIXED || joint ? nkv : 2 * nkv);
  const int gw = static_cast<int>((blockIdx.x * static_cast<unsigned>(kThreads) + threadIdx.x) >> 5);
  const int t = gw / per, c = gw - t * per;
  if (t >= a.T) return;
  Place p;
  if (!place_of(a, t, lane, p)) return;
  if (p.pos >= q.max_pos) {
    if (lane == 0) atomicOr(a.err, KV4_DEVERR_LENGTH);
    return;
  }
  if (c < nq) {
    Rotation<D> rot;
    float w[8];
    rot.load(q, p.pos, lane);
    load_weight<D>(q.qw, q.w_dtype, lane, w);
    rope_heads<D, 2>(q, rot, w, q.qw != nullptr, q.q, q.q_dtype, t * q.q_stride, q.q_out, q.q_out_dtype, t * q.q_out_stride, c * hpw,
                  min((c + 1) * hpw, q.Hq), q.q_fast, lane);
    return;
  }
  const bool is_k = FMT == POOL_MIXED || c < nq + nkv, is_v = FMT != POOL_MIXED && (joint || !is_k);
  const int g0 = (is_k ? c - nq : c - nq - nkv) * HP, g = FMT == POOL_MIXED ? g0 : min(g0 + mine, a.Hkv - 1);
  const bool act = FMT == POOL_MIXED ? mine == 0 : g0 + mine < a.Hkv;
  const int row = FMT <= POOL_VBF ? side_row(p.pos, a.s, a.w, a.w > 0 && p.pos >= a.s ? a.lens_after[p.b] : 0) : -1;
  float x[8], v[8];
  if (is_v) load8(q.v, q.v_dtype, t * q.v_stride + g * D + 8 * gl, v);
  if (is_k) {
    load8(q.k, q.k_dtype, t * q.k_stride + g * D + 8 * gl, x);
    if (q.kw) {
      float w[8];
      load_weight<D>(q.kw, q.w_dtype, lane, w);
      head_norm<D>(x, w, q.eps);
    }
    {
      Rotation<D> rot;
      rot.load(q, p.pos, lane);
      rot.apply(x);
    }
    if constexpr (FMT == POOL_MIXED) {
      // the encoder's lanes hold coordinates l + 32 i
      const int warp = threadIdx.x >> 5;
      float k[NI], vv[NI];
#pragma unroll
      for (int i = 0; i < NI; ++i) vv[i] = load_elem(q.v, q.v_dtype, static_cast<size_t>(t * q.v_stride + g * D + lane + 32 * i));
      if (act) {
        *reinterpret_cast<float4*>(&xs[warp][8 * gl]) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(&xs[warp][8 * gl + 4]) = make_float4(x[4], x[5], x[6], x[7]);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NI; ++i) k[i] = xs[warp][lane + 32 * i];
      mixed_encode_store<D>(a, g, p.page, p.pos, lane, k, vv, rows[warp][0], rows[warp][1]);
    } else {
      put_key<D, FMT>(a, p, g, row, gl, act, x);
    }
  }
  if constexpr (FMT != POOL_MIXED) {
    if (is_v) put_value<D, FMT>(a, p, g, row, gl, act, v);
  }
}

// ------------------------------------------------------------------ kv4_gather

// Inverse of the stored rotation: diag(s) H x / h.
__device__ __forceinline__ void unrotate8(const AppendArgs& a, int gl, float (&x)[8]) {
  if (a.h > 1) {
    hadamard8(x, gl, a.h);
    const float ih = 1.f / static_cast<float>(a.h);  // a power of two: exact
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= ih;
  }
  flip_signs8(x, gl, a.signs);
}

__device__ __forceinline__ float2 scale_zero(const uint8_t* p) {
  const uint32_t sz = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__half2float(__ushort_as_half(static_cast<unsigned short>(sz & 0xffffu))),
                     __half2float(__ushort_as_half(static_cast<unsigned short>(sz >> 16))));
}

// c < 2^23 as a float, exactly, off the conversion pipe.
__device__ __forceinline__ float small_float(uint32_t c) { return __uint_as_float(c | 0x4B000000u) - 8388608.f; }

// Codes of `w` bits at bit `o` of a row of 32-bit words.
__device__ __forceinline__ uint32_t get_bits(const uint32_t* row, int o, int w) {
  if (w == 0) return 0u;
  const int wi = o >> 5, sh = o & 31;
  uint32_t x = row[wi] >> sh;
  if (sh + w > 32) x |= row[wi + 1] << (32 - sh);
  return x & ((1u << w) - 1u);
}

template <int D>
__device__ __forceinline__ void read_vbf(const uint8_t* vblock, int r, int gl, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    x[j] = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(vblock + vbf_offset<D>(r, 8 * gl + j)));
}

// Slice of a mixed-key page tile that holds the position.
template <int D>
__device__ __forceinline__ const uint8_t* slice_of(const AppendArgs& a, const Place& p, int g, int KR, int VR) {
  return a.pool + static_cast<size_t>(p.page) * a.page_bytes + static_cast<size_t>(g) * static_cast<size_t>(a.P) * (KR + VR + 8) +
         static_cast<size_t>(in_page(a, p.pos) >> 4) * 16 * (KR + VR + 8);
}

// Key of one (token, KV head) as fp32 in its original basis, by its lane group.
template <int D, int FMT>
__device__ __forceinline__ void read_key(const AppendArgs& a, const Place& p, int g, int row, int gl, float (&x)[8]) {
  const int r = p.pos & 15;
  if constexpr (FMT == POOL_MIXED) {
    const int KR = a.kbits * D / 8, VR = a.vbits * D / 8;
    const uint8_t* slice = slice_of<D>(a, p, g, KR, VR);
    const float ks = scale_zero(slice + 16 * (KR + VR) + 8 * r).x;
    const float* sig = rec_sigma<D>(a.alloc, g);
    const uint2 wb = *reinterpret_cast<const uint2*>(rec_width<D>(a.alloc, g) + (8 * gl) % (D / 2));
    int w[8], sum = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += w[j] = static_cast<int>(((j < 4 ? wb.x : wb.y) >> (8 * (j & 3))) & 255u);
    int o = sum;
#pragma unroll
    for (int d = 1; d < kLanes<D>; d <<= 1) {
      const int y = __shfl_up_sync(FULL, o, d, kLanes<D>);
      if (gl >= d) o += y;
    }
    o -= sum;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(slice + static_cast<size_t>(r) * KR);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t c = get_bits(src, o, w[j]);
      o += w[j];
      const float mid = __fadd_rn(small_float(2u * c + 1u) * (1.f / static_cast<float>(1 << w[j])), -1.f);
      x[j] = w[j] ? __fmul_rn(__fmul_rn(ks, sig[(8 * gl + j) % (D / 2)]), mid) : 0.f;
    }
  } else if (FMT != POOL_BF16 && row >= 0) {
    uint8_t* t8 = side_tile_of<D, FMT>(a, p.b, g, row);
    const float sc = __half2float(*reinterpret_cast<const __half*>(t8 + 16 * D + 2 * (row & 15)));
    const uint2 c = *reinterpret_cast<const uint2*>(k8_word<D>(t8, row & 15, 2 * gl));
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = sc * static_cast<float>(static_cast<int8_t>((j < 4 ? c.x : c.y) >> (8 * (j & 3))));
    unrotate8(a, gl, x);
  } else {
    uint8_t* tile = tile_of<D, FMT>(a, p, g);
    if constexpr (FMT == POOL_BF16) {
      load8(kbf_unit<D>(tile, r, 2 * gl), KV4_BF16, 0, x);
    } else {
      const float2 sz = scale_zero(tile + (FMT == POOL_VBF ? 8 * D : 16 * D) + 4 * r);
      const uint2 w = *reinterpret_cast<const uint2*>(k4_group<D>(tile, r & 7, gl));
      const int sh = 4 * (r >> 3);
      const uint32_t even = w.x >> sh, odd = w.y >> sh;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = fmaf(sz.x, small_float((even >> (8 * j)) & 15u), sz.y);
        x[2 * j + 1] = fmaf(sz.x, small_float((odd >> (8 * j)) & 15u), sz.y);
      }
      unrotate8(a, gl, x);
    }
  }
}

template <int D, int FMT>
__device__ __forceinline__ void read_value(const AppendArgs& a, const Place& p, int g, int row, int gl, float (&x)[8]) {
  const int r = p.pos & 15;
  if constexpr (FMT == POOL_MIXED) {
    const int KR = a.kbits * D / 8, VR = a.vbits * D / 8;
    const uint8_t* slice = slice_of<D>(a, p, g, KR, VR);
    const float2 zr = scale_zero(slice + 16 * (KR + VR) + 8 * r + 4);  // zero, range
    const float step = __fdiv_rn(zr.y, static_cast<float>((1 << a.vbits) - 1));
    const uint32_t* src = reinterpret_cast<const uint32_t*>(slice + 16 * static_cast<size_t>(KR) + static_cast<size_t>(r) * VR);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = fmaf(step, small_float(get_bits(src, (8 * gl + j) * a.vbits, a.vbits)), zr.x);
  } else if (FMT != POOL_BF16 && row >= 0) {
    uint8_t* t8 = side_tile_of<D, FMT>(a, p.b, g, row);
    if constexpr (FMT == POOL_VBF) {
      read_vbf<D>(t8 + Geo<D>::VB8O, row & 15, gl, x);
    } else {
      const uint8_t* vb = t8 + Geo<D>::H8B;
      const float sc = __half2float(*reinterpret_cast<const __half*>(vb + 16 * D + 2 * (row & 15)));
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = sc * static_cast<float>(static_cast<int8_t>(vb[v8_offset<D>(row & 15, 8 * gl + j)]));
    }
  } else {
    uint8_t* tile = tile_of<D, FMT>(a, p, g);
    if constexpr (FMT == POOL_BF16) {
      read_vbf<D>(tile + 32 * D, r, gl, x);
    } else if constexpr (FMT == POOL_VBF) {
      read_vbf<D>(tile + Geo<D>::VBO, r, gl, x);
    } else {
      const float2 sz = scale_zero(tile + 16 * D + 64 + 4 * r);
      const uint32_t c = *v4_chunk<D>(tile, r, 2 * gl) | (static_cast<uint32_t>(*v4_chunk<D>(tile, r, 2 * gl + 1)) << 16);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = fmaf(sz.x, small_float((c >> (4 * j)) & 15u), sz.y);
    }
  }
  if (FMT == POOL_INT4 && a.rotate_v) unrotate8(a, gl, x);
}

// Warp (token, kPerWarp KV heads).  Bound by issue (2.9 instructions a cycle), so the warps in flight
// count: eight blocks an SM (32 registers) read 14460 positions of 8 heads back in 38 us, 40 registers in
// 41, and four passes a warp in a loop, a fifth of the instructions fewer but 64 registers, in 46.
template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 8) gather_kernel(AppendArgs a, void* k_out, void* v_out, int dtype) {
  const int lane = threadIdx.x & 31, gl = lane % kLanes<D>;
  const int per = (a.Hkv + kPerWarp<D> - 1) / kPerWarp<D>;
  const int gw = static_cast<int>((blockIdx.x * static_cast<unsigned>(kThreads) + threadIdx.x) >> 5);
  const int t = gw / per, g = (gw - t * per) * kPerWarp<D> + lane / kLanes<D>;
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
  const int gr = min(g, a.Hkv - 1);  // lanes without a head read the last one
  const long long o = (static_cast<long long>(t) * a.Hkv + g) * D + 8 * gl;
  float x[8], y[8];
  if (k_out) read_key<D, FMT>(a, p, gr, row, gl, x);
  if (v_out) read_value<D, FMT>(a, p, gr, row, gl, y);
  if (g < a.Hkv) {
    if (k_out) store8(k_out, dtype, o, x);
    if (v_out) store8(v_out, dtype, o, y);
  }
}

unsigned blocks_for(long long warps) { return static_cast<unsigned>((warps + kWarpsPerBlock - 1) / kWarpsPerBlock); }

// Few vectors: the launch has fewer warps than the GPU holds and the latency counts.
template <int D>
bool few(long long vectors) { return vectors <= 148LL * 64 * kPerWarp<D>; }

// Heads a warp takes: one pass when there are few, kRunPasses otherwise (their table row and weights are read once).
template <int D>
int heads_per_warp(long long vectors) { return few<D>(vectors) ? kPerWarp<D> : kRunPasses * kPerWarp<D>; }

}  // namespace

cudaError_t launch_rope_table(const RopeTableArgs& a, cudaStream_t st) {
  const long long threads = (a.max_pos + kRun - 1) / kRun * (a.R / 2);
  note_launches(1);
  rope_table_kernel<<<static_cast<unsigned>((threads + kThreads - 1) / kThreads), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <int D>
static void launch_rope_d(RopeArgs a, cudaStream_t st) {
  a.q_fast = rows16(a.q, a.q_dtype, a.q_stride, a.q_out, a.q_out_dtype, a.q_out_stride);
  a.k_fast = rows16(a.k, a.k_dtype, a.k_stride, a.k_out, a.k_out_dtype, a.k_out_stride);
  const int hpw = heads_per_warp<D>(static_cast<long long>(a.T) * (a.Hq + a.Hkv));
  const unsigned grid = blocks_for(static_cast<long long>(a.T) * ((a.Hq + hpw - 1) / hpw + (a.Hkv + hpw - 1) / hpw));
  rope_kernel<D><<<grid, kThreads, 0, st>>>(a, hpw);
}

cudaError_t launch_rope(const RopeArgs& a, int D, cudaStream_t st) {
  note_launches(1);
  if (D == 128) launch_rope_d<128>(a, st);
  else launch_rope_d<64>(a, st);
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_append_rope_d(RopeArgs q, const AppendArgs& a, int format, cudaStream_t st) {
  q.q_fast = rows16(q.q, q.q_dtype, q.q_stride, q.q_out, q.q_out_dtype, q.q_out_stride);
  const long long vectors = static_cast<long long>(a.T) * (q.Hq + 2 * a.Hkv);
  const int hpw = heads_per_warp<D>(vectors), passes = (a.Hkv + kPerWarp<D> - 1) / kPerWarp<D>;
  const bool joint = !few<D>(vectors);
  const int per = (q.Hq + hpw - 1) / hpw + (format == POOL_MIXED ? a.Hkv : joint ? passes : 2 * passes);
  const unsigned grid = blocks_for(static_cast<long long>(a.T) * per);
  note_launches(1);
  switch (format) {
    case POOL_INT4: append_rope_kernel<D, POOL_INT4><<<grid, kThreads, 0, st>>>(q, a, hpw, joint); break;
    case POOL_VBF: append_rope_kernel<D, POOL_VBF><<<grid, kThreads, 0, st>>>(q, a, hpw, joint); break;
    case POOL_MIXED: append_rope_kernel<D, POOL_MIXED><<<grid, kThreads, 0, st>>>(q, a, hpw, joint); break;
    default: append_rope_kernel<D, POOL_BF16><<<grid, kThreads, 0, st>>>(q, a, hpw, joint); break;
  }
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_gather_d(const AppendArgs& a, int format, void* k_out, void* v_out, int dtype, cudaStream_t st) {
  const unsigned grid = blocks_for(static_cast<long long>(a.T) * ((a.Hkv + kPerWarp<D> - 1) / kPerWarp<D>));
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
