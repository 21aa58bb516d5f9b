// kv4_quant.cuh -- the per-vector encoders of the append kernels and where their codes go in a page
// tile or a side-cache row.  kv4_append: a warp holds one head vector, lane l elements 4l..4l+3 (D =
// 128 uses all 32 lanes, D = 64 the first 16).  kv4_append_rope (the functions with an 8): D / 8 lanes
// hold one, lane l of the group elements 8l..8l+7, and a warp 2 or 4 vectors.  Bit-exact rules: the butterfly runs strides 1, 2, ...,
// h/2 in that order with plain fp32 add/sub (a + b, a - b); the quantiser uses IEEE fp32 sub/div,
// rint (ties to even) and directed fp16 conversions; min and max are taken as values (+0 for zero).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kv4_device.cuh"
#include "kv4_layout.cuh"

namespace kv4 {

constexpr unsigned kFullWarp = 0xffffffffu;
template <typename T>
__device__ __forceinline__ void load4(const void* base, size_t i, float (&x)[4]);

template <>
__device__ __forceinline__ void load4<float>(const void* base, size_t i, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + i);
  x[0] = v.x;
  x[1] = v.y;
  x[2] = v.z;
  x[3] = v.w;
}

template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(const void* base, size_t i, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(base) + i);
  x[0] = __uint_as_float(v.x << 16);
  x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16);
  x[3] = __uint_as_float(v.y & 0xffff0000u);
}

// The signs of the randomised-sign rotation: dims of set bits are negated (exact).
__device__ __forceinline__ void flip_signs4(float (&x)[4], int lane, const uint32_t (&signs)[4]) {
  const uint32_t sb = (signs[lane >> 3] >> (4 * (lane & 7))) & 15u;
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(__float_as_uint(x[e]) ^ (((sb >> e) & 1u) << 31));
}

// Sylvester block Hadamard on blocks of h over the warp's D elements (lane holds 4).
__device__ __forceinline__ void hadamard4(float (&x)[4], int lane, int h) {
  if (h >= 2) {
    float a = x[0], b = x[1];
    x[0] = __fadd_rn(a, b);
    x[1] = __fsub_rn(a, b);
    a = x[2];
    b = x[3];
    x[2] = __fadd_rn(a, b);
    x[3] = __fsub_rn(a, b);
  }
  if (h >= 4) {
    float a = x[0], b = x[2];
    x[0] = __fadd_rn(a, b);
    x[2] = __fsub_rn(a, b);
    a = x[1];
    b = x[3];
    x[1] = __fadd_rn(a, b);
    x[3] = __fsub_rn(a, b);
  }
  for (int st = 4; st < h; st <<= 1) {
    const int m = st >> 2;
    const bool upper = (lane & m) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float o = __shfl_xor_sync(kFullWarp, x[i], m);
      x[i] = upper ? __fsub_rn(o, x[i]) : __fadd_rn(x[i], o);
    }
  }
}

__device__ __forceinline__ float warp_min(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fminf(v, __shfl_xor_sync(kFullWarp, v, o));
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullWarp, v, o));
  return v;
}

// INT4 codes of the lane's 4 elements packed as elements 0..3 in bits 0..15 (4 bits each);
// *sz receives (fp16 scale bits) | (fp16 zero bits << 16).  A vector whose zero or scale is not a
// finite fp16 (values beyond the fp16 range) keeps those parameters, gets all-zero codes and sets
// *bad (warp-uniform: the parameters come from warp reductions).
__device__ __forceinline__ uint32_t quant_int4(const float (&x)[4], bool act, uint32_t* sz, bool* bad) {
  float mn = act ? fminf(fminf(x[0], x[1]), fminf(x[2], x[3])) : __int_as_float(0x7f800000);
  float mx = act ? fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) : __int_as_float(0xff800000);
  mn = __fadd_rn(warp_min(mn), 0.0f);
  mx = __fadd_rn(warp_max(mx), 0.0f);
  const __half zh = __float2half_rd(mn);
  const float zf = __half2float(zh);
  const float r = __fsub_rn(mx, zf);
  const __half sh = __float2half_ru(__fdiv_rn(r, 15.0f));
  const float sf = __half2float(sh);
  *bad = !(isfinite(zf) && isfinite(sf));
  uint32_t packed = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int c = 0;
    if (sf != 0.0f && !*bad) {
      c = static_cast<int>(rintf(__fdiv_rn(__fsub_rn(x[i], zf), sf)));
      c = min(max(c, 0), 15);
    }
    packed |= static_cast<uint32_t>(c) << (4 * i);
  }
  *sz = static_cast<uint32_t>(__half_as_ushort(sh)) | (static_cast<uint32_t>(__half_as_ushort(zh)) << 16);
  return packed;
}

// Symmetric INT8 codes of the lane's 4 elements (bytes 0..3), fp16 scale bits in *sc; a scale
// that is not a finite fp16 gives all-zero codes and sets *bad, as for INT4.
__device__ __forceinline__ uint32_t quant_int8(const float (&x)[4], bool act, uint16_t* sc, bool* bad) {
  float a = act ? fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))) : 0.0f;
  a = warp_max(a);
  const __half sh = __float2half_ru(__fdiv_rn(a, 127.0f));
  const float sf = __half2float(sh);
  *bad = !isfinite(sf);
  uint32_t packed = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int c = 0;
    if (sf != 0.0f && !*bad) {
      c = static_cast<int>(rintf(__fdiv_rn(x[i], sf)));
      c = min(max(c, -127), 127);
    }
    packed |= (static_cast<uint32_t>(c) & 0xffu) << (8 * i);
  }
  *sc = __half_as_ushort(sh);
  return packed;
}

// Offset of value element e of row r in a 16-row bf16 V block (the BF16 pool's V order).
template <int D>
__device__ __forceinline__ int vbf_offset(int r, int e) {
  using Gm = Geo<D>;
  const int p = r >> 1, half = p >> 2, pl = p & 3;
  const int gq = e / Gm::DG, m = e % Gm::DG, uu = m >> 2;
  return ((half * 8 + gq) * 4 + pl) * (D / 2) + ((uu ^ bf16_swz(D, pl, gq)) << 4) + (m & 3) * 4 + (r & 1) * 2;
}

// ------------------------------------------------------------------ stores

// INT4 key codes of row r (0..15) of a page tile: row r shares pair-row r % 8 with row r ^ 8 (low
// nibbles rows 0-7, high nibbles rows 8-15), so its nibbles are merged in with atomics (another
// token of the tile may be written by another warp of this launch).  Elements 4l, 4l+2 go to bytes
// 2(l&1), 2(l&1)+1 of word 0 of 8-byte group l/2, elements 4l+1, 4l+3 to the same bytes of word 1.
template <int D>
__device__ __forceinline__ uint32_t* k4_words(uint8_t* tile, int pr, int lane) {
  const int gb = 8 * (lane >> 1);                                    // group byte in the pair-row
  const int unit = (gb >> 4) ^ (D >= 128 ? (pr & 1) : 0);
  return reinterpret_cast<uint32_t*>(tile + pr * D + 16 * unit + (gb & 15));
}

template <int D>
__device__ __forceinline__ void store_k4(uint8_t* tile, int r, int lane, uint32_t kc) {
  uint32_t* w0 = k4_words<D>(tile, r & 7, lane);
  const int sh = 16 * (lane & 1) + 4 * (r >> 3);                     // bit of byte 2(l&1)
  const uint32_t e0 = kc & 15u, e1 = (kc >> 4) & 15u, e2 = (kc >> 8) & 15u, e3 = (kc >> 12) & 15u;
  const uint32_t clear = ~((0xFu << sh) | (0xFu << (sh + 8)));
  atomicAnd(w0, clear);
  atomicOr(w0, (e0 << sh) | (e2 << (sh + 8)));
  atomicAnd(w0 + 1, clear);
  atomicOr(w0 + 1, (e1 << sh) | (e3 << (sh + 8)));
}

// INT4 value codes of row r: the 16-bit chunk of quad Q = lane.
template <int D>
__device__ __forceinline__ uint16_t* v4_chunk(uint8_t* tile, int r, int lane) {
  using Gm = Geo<D>;
  const int Q = lane, p = r >> 1, half = p >> 2, pl = p & 3;
  const int off = ((half * 8 + Q / Gm::WPC) * 4 + pl) * Gm::CH + 4 * (Q % Gm::WPC) + 2 * (r & 1);
  return reinterpret_cast<uint16_t*>(tile + 8 * D + off);
}

// bf16 values (nearest even) of row r into a V block in the BF16 pool's order.
template <int D>
__device__ __forceinline__ void store_vbf(uint8_t* vblock, int r, int lane, const float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<__nv_bfloat16*>(vblock + vbf_offset<D>(r, 4 * lane + i)) = __float2bfloat16_rn(v[i]);
}

// INT8 key codes of side row r8 (0..15) of a side tile.
template <int D>
__device__ __forceinline__ uint32_t* k8_word(uint8_t* t8, int r8, int lane) {
  const int e = 4 * lane;
  return reinterpret_cast<uint32_t*>(t8 + r8 * D + 16 * ((e >> 4) ^ (r8 & 1)) + (e & 15));
}

// Byte of value element e of side row r8, from the value half of a side tile.
template <int D>
__device__ __forceinline__ int v8_offset(int r8, int e) {
  using Gm = Geo<D>;
  const int p = r8 >> 1, half = p >> 2, pl = p & 3, gq = e / Gm::DG, dd = e % Gm::DG;
  int bb = (dd >> 1) * 4 + (dd & 1) * 2 + (r8 & 1);
  if (Gm::CH8 >= 32) bb ^= 16 * (gq & 1);
  return ((half * 8 + gq) * 4 + pl) * Gm::CH8 + bb;
}

// Side row of an appended position: its sink or ring row, -1 when it is in neither region.
__device__ __forceinline__ int side_row(int pos, int s, int w, int len_after) {
  if (pos < s) return pos;
  return w > 0 && pos >= len_after - w ? s + pos % w : -1;
}

// bf16 keys of row r of a BF16 pool tile: element e in thread chunk c = e / EPT, unit u =
// (e % EPT) / 8 stored at u ^ sw.
template <int D>
__device__ __forceinline__ uint8_t* kbf_unit(uint8_t* tile, int r, int lane) {
  using Gm = Geo<D>;
  const int e = 4 * lane, c = e / Gm::EPT, u = (e % Gm::EPT) >> 3;
  return tile + r * 2 * D + c * 2 * Gm::EPT + ((u ^ bf16_swz(D, c, r)) << 4) + (e & 7) * 2;
}

// ------------------------------------------------------------------ eight elements a lane

// All D / 8 lanes of a vector's group hold the result of these.
template <int D>
__device__ __forceinline__ float group_min(float v) {
#pragma unroll
  for (int o = D / 16; o; o >>= 1) v = fminf(v, __shfl_xor_sync(kFullWarp, v, o));
  return v;
}
template <int D>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = D / 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullWarp, v, o));
  return v;
}

__device__ __forceinline__ void flip_signs8(float (&x)[8], int gl, const uint32_t (&signs)[4]) {
  if ((signs[0] | signs[1] | signs[2] | signs[3]) == 0u) return;
  const uint32_t sb = (signs[gl >> 2] >> (8 * (gl & 3))) & 255u;
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(__float_as_uint(x[e]) ^ (((sb >> e) & 1u) << 31));
}

// Sylvester block Hadamard on blocks of h, strides ascending, over the group's D elements.
__device__ __forceinline__ void hadamard8(float (&x)[8], int gl, int h) {
#pragma unroll
  for (int st = 1; st < 8; st <<= 1) {
    if (st >= h) return;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if ((e & st) == 0) {
        const float a = x[e], b = x[e + st];
        x[e] = __fadd_rn(a, b);
        x[e + st] = __fsub_rn(a, b);
      }
  }
  for (int st = 8; st < h; st <<= 1) {
    const int m = st >> 3;
    // the upper half of a pair gets o - x, the lower x + o: one rounding of o +- x either way
    const float sg = (gl & m) ? -1.f : 1.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __fmaf_rn(x[e], sg, __shfl_xor_sync(kFullWarp, x[e], m));
  }
}

// rint(a / s), the IEEE quotient rounded to an integer, in the low bits of the result (two's
// complement): adding 1.5 2^23 rounds to an integer and leaves it there.  q = a inv is within 128 2^-22
// of the quotient, so away from the middle between two integers it rounds to the same one; near the
// middle the division itself decides.
__device__ __forceinline__ uint32_t rint_div(float q, float a, float s) {
  constexpr float kRound = 12582912.f;
  float u = __fadd_rn(q, kRound);
  if (fabsf(q - __fsub_rn(u, kRound)) > 0.4999f) u = __fadd_rn(rintf(__fdiv_rn(a, s)), kRound);
  return __float_as_uint(u);
}

// INT4 codes of the lane's 8 elements, element e in bits 4e..4e+3; parameters and *bad as quant_int4.
template <int D>
__device__ __forceinline__ uint32_t quant_int4_8(const float (&x)[8], uint32_t* sz, bool* bad) {
  float mn = x[0], mx = x[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    mn = fminf(mn, x[e]);
    mx = fmaxf(mx, x[e]);
  }
  mn = __fadd_rn(group_min<D>(mn), 0.0f);
  mx = __fadd_rn(group_max<D>(mx), 0.0f);
  const __half zh = __float2half_rd(mn);
  const float zf = __half2float(zh);
  const __half sh = __float2half_ru(__fdiv_rn(__fsub_rn(mx, zf), 15.0f));
  const float sf = __half2float(sh);
  *bad = !(isfinite(zf) && isfinite(sf));
  *sz = static_cast<uint32_t>(__half_as_ushort(sh)) | (static_cast<uint32_t>(__half_as_ushort(zh)) << 16);
  if (sf == 0.0f || *bad) return 0u;
  const float inv = __frcp_rn(sf);
  uint32_t packed = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // zero <= x and the scale was rounded up: a code is at most 15; a NaN takes code 0
    const float d = __fsub_rn(x[e], zf);
    packed |= (rint_div(fmaxf(d * inv, 0.f), d, sf) & 15u) << (4 * e);
  }
  return packed;
}

// Symmetric INT8 codes, elements 0..3 in .x, 4..7 in .y.
template <int D>
__device__ __forceinline__ uint2 quant_int8_8(const float (&x)[8], uint16_t* sc, bool* bad) {
  float a = fabsf(x[0]);
#pragma unroll
  for (int e = 1; e < 8; ++e) a = fmaxf(a, fabsf(x[e]));
  a = group_max<D>(a);
  const __half sh = __float2half_ru(__fdiv_rn(a, 127.0f));
  const float sf = __half2float(sh);
  *bad = !isfinite(sf);
  *sc = __half_as_ushort(sh);
  if (sf == 0.0f || *bad) return make_uint2(0u, 0u);
  const float inv = __frcp_rn(sf);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float q = x[e] * inv;  // at most 127 in magnitude; a NaN takes code 0
    w[e >> 2] |= (rint_div(q == q ? q : 0.f, x[e], sf) & 0xffu) << (8 * (e & 3));
  }
  return make_uint2(w[0], w[1]);
}

// The lane's 8 key elements of pair-row pr are one 8-byte group (even elements, then odd ones), both rows'.
template <int D>
__device__ __forceinline__ unsigned long long* k4_group(uint8_t* tile, int pr, int gl) {
  const int unit = (gl >> 1) ^ (D >= 128 ? (pr & 1) : 0);
  return reinterpret_cast<unsigned long long*>(tile + pr * D + 16 * unit + 8 * (gl & 1));
}

// Nibbles 0, 2, 4, 6 of x to the low nibbles of 4 bytes.
__device__ __forceinline__ uint32_t spread_even(uint32_t x) {
  return (x & 0xFu) | (x & 0xF00u) | (x & 0xF0000u) | (x & 0xF000000u);
}

template <int D>
__device__ __forceinline__ void store_k4_8(uint8_t* tile, int r, int gl, uint32_t kc) {
  unsigned long long* w = k4_group<D>(tile, r & 7, gl);
  const unsigned long long codes = static_cast<unsigned long long>(spread_even(kc)) | (static_cast<unsigned long long>(spread_even(kc >> 4)) << 32);
  const int sh = 4 * (r >> 3);
  atomicAnd(w, ~(0x0F0F0F0F0F0F0F0Full << sh));
  atomicOr(w, codes << sh);
}

template <int D>
__device__ __forceinline__ void store_vbf_8(uint8_t* vblock, int r, int gl, const float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    *reinterpret_cast<__nv_bfloat16*>(vblock + vbf_offset<D>(r, 8 * gl + e)) = __float2bfloat16_rn(v[e]);
}

}  // namespace kv4
