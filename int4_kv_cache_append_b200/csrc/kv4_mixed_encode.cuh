// kv4_mixed_encode.cuh -- the encoder of the mixed bit-width key cache: one token's key (block
// scales and widths) and value (per-token affine), bit-packed into the page slot.  The format is
// described in kv4_mixed.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kv4_device.cuh"
#include "kv4_internal.h"

namespace kv4 {

__device__ __forceinline__ float load_elem(const void* base, int dtype, size_t i) {
  if (dtype == KV4_F32) return reinterpret_cast<const float*>(base)[i];
  if (dtype == KV4_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[i]);
  return __half2float(reinterpret_cast<const __half*>(base)[i]);
}

template <int D>
__device__ __forceinline__ const float* rec_sigma(const uint8_t* alloc, int g) {
  return reinterpret_cast<const float*>(alloc + static_cast<size_t>(g) * mixed_alloc_record_bytes(D));
}
template <int D>
__device__ __forceinline__ const uint8_t* rec_width(const uint8_t* alloc, int g) {
  return alloc + static_cast<size_t>(g) * mixed_alloc_record_bytes(D) + (D / 2) * 4;
}

// Add `code` (w bits) at bit `o` of a row held as 32-bit words in shared memory.
__device__ __forceinline__ void put_bits(uint32_t* row, int o, uint32_t code, int w) {
  if (w == 0) return;
  const int wi = o >> 5, sh = o & 31;
  atomicOr(&row[wi], code << sh);
  if (sh + w > 32) atomicOr(&row[wi + 1], code >> (32 - sh));
}

// A row of codes being built: up to 8 bits per coordinate and a guard word.
template <int D>
constexpr int kMixedRowWords = D / 4 + 1;

// Encode key k and value v of one (token, KV head) by one warp (lane l holds coordinates l + 32 i)
// and write them to position pos of page `page`.  krow and vrow are the warp's row buffers.
template <int D>
__device__ __forceinline__ void mixed_encode_store(const AppendArgs& a, int g, int page, int pos, int lane,
                                                   const float (&k)[D / 32], const float (&v)[D / 32], uint32_t* krow,
                                                   uint32_t* vrow) {
  constexpr int NB = D / 2, NI = D / 32, RW = kMixedRowWords<D>;
  const float* sig = rec_sigma<D>(a.alloc, g);
  const uint8_t* wid = rec_width<D>(a.alloc, g);
  float sg[NI];
  int w[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int j = lane + 32 * i;
    sg[i] = sig[j % NB];
    w[i] = wid[j % NB];
  }
  for (int i = lane; i < RW; i += 32) krow[i] = vrow[i] = 0u;

  // bit offsets of the lane's coordinates: exclusive prefix of the block widths (coordinate j is
  // block j mod D/2; the second half of the row starts after key_bits * D / 2 bits)
  int pre[NI];
  {
    int run = 0;
#pragma unroll
    for (int c = 0; c < NB / 32; ++c) {
      int x = w[c];  // block lane + 32 c is coordinate lane + 32 c
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      pre[c] = run + x - w[c];
      run += __shfl_sync(0xffffffffu, x, 31);
    }
#pragma unroll
    for (int i = NB / 32; i < NI; ++i) pre[i] = run + pre[i - NB / 32];
  }

  // key: one fp16 scale over the block-standardised coordinates that have bits
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < NI; ++i)
    if (w[i] > 0) m = fmaxf(m, __fdiv_rn(fabsf(k[i]), sg[i]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const __half ksh = __float2half_ru(m);
  const float sf = __half2float(ksh);
  const bool kbad = !isfinite(sf);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    uint32_t c = 0u;
    if (w[i] > 0 && sf != 0.f && !kbad) {
      const int top = (1 << w[i]) - 1;
      const float d = __fmul_rn(sg[i], sf);
      const float tq = __fdiv_rn(k[i], d);
      const float u = __fmul_rn(__fadd_rn(tq, 1.0f), static_cast<float>(1 << (w[i] - 1)));
      const float f = floorf(u);
      c = f < 0.f ? 0u : (f > static_cast<float>(top) ? static_cast<uint32_t>(top) : static_cast<uint32_t>(f));
    }
    put_bits(krow, pre[i], c, w[i]);
  }

  // value: per-token affine code at vbits
  float mn = v[0], mx = v[0];
#pragma unroll
  for (int i = 1; i < NI; ++i) {
    mn = fminf(mn, v[i]);
    mx = fmaxf(mx, v[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  mn = mn + 0.0f;
  mx = mx + 0.0f;
  const __half vzh = __float2half_rd(mn);
  const float zf = __half2float(vzh);
  const __half vrh = __float2half_ru(__fsub_rn(mx, zf));
  const float rf = __half2float(vrh);
  const bool vbad = !isfinite(zf) || !isfinite(rf);
  const int vtop = (1 << a.vbits) - 1;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    uint32_t c = 0u;
    if (rf != 0.f && !vbad) {
      const float step = __fdiv_rn(rf, static_cast<float>(vtop));
      const float r = rintf(__fdiv_rn(__fsub_rn(v[i], zf), step));
      c = r < 0.f ? 0u : (r > static_cast<float>(vtop) ? static_cast<uint32_t>(vtop) : static_cast<uint32_t>(r));
    }
    put_bits(vrow, (lane + 32 * i) * a.vbits, c, a.vbits);
  }
  if (lane == 0 && (kbad || vbad)) atomicOr(a.err, KV4_DEVERR_RANGE);
  __syncwarp();

  const int KR = a.kbits * D / 8, VR = a.vbits * D / 8, pp = pos % a.P, rr = pp & 15;
  // the position's 16-position slice: 16 key rows, 16 value rows, 16 records
  uint8_t* slice = a.pool + static_cast<size_t>(page) * a.page_bytes +
                   static_cast<size_t>(g) * static_cast<size_t>(a.P) * (KR + VR + 8) +
                   static_cast<size_t>(pp >> 4) * 16 * (KR + VR + 8);
  uint32_t* kdst = reinterpret_cast<uint32_t*>(slice + static_cast<size_t>(rr) * KR);
  uint32_t* vdst = reinterpret_cast<uint32_t*>(slice + 16 * static_cast<size_t>(KR) + static_cast<size_t>(rr) * VR);
  for (int i = lane; i < KR / 4; i += 32) kdst[i] = krow[i];
  for (int i = lane; i < VR / 4; i += 32) vdst[i] = vrow[i];
  if (lane == 0) {
    const unsigned long long rec =
        static_cast<unsigned long long>(__half_as_ushort(ksh)) |
        (static_cast<unsigned long long>(__half_as_ushort(vzh)) << 32) |
        (static_cast<unsigned long long>(__half_as_ushort(vrh)) << 48);
    *reinterpret_cast<unsigned long long*>(slice + 16 * static_cast<size_t>(KR + VR) + static_cast<size_t>(rr) * 8) = rec;
  }
}

}  // namespace kv4
