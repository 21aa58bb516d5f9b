// kv4_append.cu -- fused append: block-Hadamard rotation of K, per-token affine INT4
// quantisation of rotated K and of V, nibble packing into the page slot, INT8 routing of
// sink / recent positions into the side cache.  Plus the BF16 pool append of the baseline.
//
// Method: KV4-RL (ai.info summary), "Methodology in Plain English" paragraph 2 (one affine INT4
// group per token-head vector, FP16 scale and offset, keys Hadamard-rotated before
// quantisation) and paragraph 3 (INT8 side cache for the first s and last w positions);
// SAW-INT4 (gist.science summary), section 2 (block-diagonal rotation in blocks of h, fused with
// quantisation in one kernel).
//
// One warp per (token, KV head); the encoders and their bit-exact rules are in kv4_quant.cuh.
#include <cuda_bf16.h>

#include "kv4_device.cuh"
#include "kv4_internal.h"
#include "kv4_layout.cuh"
#include "kv4_quant.cuh"

namespace kv4 {
namespace {

constexpr int kAppendThreads = 256;

// VB: values kept as bf16 (KV4_VALUES_BF16) instead of INT4 / INT8.
template <int D, typename KT, typename VT, bool VB>
__global__ void __launch_bounds__(kAppendThreads) append_int4_kernel(AppendArgs a) {
  using Gm = Geo<D>;
  constexpr int PB = VB ? D / 2 + 4 + 2 * D : D + 8;  // bytes of one position of one head in a page
  constexpr int KPO = VB ? 8 * D : 16 * D;             // K parameters in a page tile
  constexpr int T8 = VB ? Gm::T8V : Gm::T8B;           // side tile
  pdl_launch_dependents();  // the decode kernel that follows may start its launch now
  const int gw = static_cast<int>((blockIdx.x * blockDim.x + threadIdx.x) >> 5);
  const int lane = threadIdx.x & 31;
  if (gw >= a.T * a.Hkv) return;
  const int t = gw / a.Hkv, g = gw - t * a.Hkv;
  // Three dependent round trips at most: {token's slot and position, its K and V} -> {page-table
  // entry, length after the call} -> stores.  K and V are read before the checks (every t < T is
  // a valid input row).
  const bool act = lane < D / 4;
  float k[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
  const size_t in0 = (static_cast<size_t>(t) * a.Hkv + g) * D + 4 * lane;
  if (act) {
    load4<KT>(a.K, in0, k);
    load4<VT>(a.V, in0, v);
  }
  const int b = a.seq_slot[t], pos = a.pos[t];
  if (b < 0 || b >= a.max_seqs || pos < 0 || pos / a.P >= a.stride) {
    if (lane == 0) atomicOr(a.err, KV4_DEVERR_LENGTH);
    return;
  }
  const int page = a.page_table[static_cast<size_t>(b) * a.stride + pos / a.P];
  const int len_after = a.w > 0 && pos >= a.s ? a.lens_after[b] : 0;
  if (page < 0 || page >= a.max_pages) {
    if (lane == 0) atomicOr(a.err, KV4_DEVERR_PAGE_RANGE);
    return;
  }
  flip_signs4(k, lane, a.signs);  // randomised-sign rotation
  hadamard4(k, lane, a.h);
  if (a.rotate_v) {  // value rotation: the same H diag(s) as the keys
    flip_signs4(v, lane, a.signs);
    hadamard4(v, lane, a.h);
  }

  const int pp = pos % a.P, r = pp & 15;
  uint8_t* tile = a.pool + static_cast<size_t>(page) * a.page_bytes + static_cast<size_t>(g) * a.P * PB +
                  static_cast<size_t>(pp >> 4) * (16 * PB);
  uint32_t ksz, vsz = 0;
  bool kbad, vbad = false;
  const uint32_t kc = quant_int4(k, act, &ksz, &kbad);
  uint32_t vc = 0;
  if constexpr (!VB) vc = quant_int4(v, act, &vsz, &vbad);
  if (lane == 0 && (kbad || vbad)) atomicOr(a.err, KV4_DEVERR_RANGE);
  if (act) {
    store_k4<D>(tile, r, lane, kc);
    if constexpr (VB)
      store_vbf<D>(tile + Gm::VBO, r, lane, v);
    else
      *v4_chunk<D>(tile, r, lane) = static_cast<uint16_t>(vc);
  }
  if (lane == 0) {
    *reinterpret_cast<uint32_t*>(tile + KPO + 4 * r) = ksz;
    if constexpr (!VB) *reinterpret_cast<uint32_t*>(tile + 16 * D + 64 + 4 * r) = vsz;
  }

  // INT8 side cache: sinks and the recent window (warp-uniform decision).
  const int row = side_row(pos, a.s, a.w, len_after);
  if (row < 0) return;
  uint8_t* t8 = a.side + static_cast<size_t>(b) * a.side_slot_bytes +
                static_cast<size_t>(g) * a.nt8 * T8 + static_cast<size_t>(row >> 4) * T8;
  const int r8 = row & 15;
  uint16_t ks, vs = 0;
  bool kbad8, vbad8 = false;
  const uint32_t k8 = quant_int8(k, act, &ks, &kbad8);
  uint32_t v8 = 0;
  if constexpr (!VB) v8 = quant_int8(v, act, &vs, &vbad8);
  if (lane == 0 && (kbad8 || vbad8)) atomicOr(a.err, KV4_DEVERR_RANGE);
  if (act) {
    *k8_word<D>(t8, r8, lane) = k8;
    if constexpr (VB) {
      store_vbf<D>(t8 + Gm::VB8O, r8, lane, v);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) t8[Gm::H8B + v8_offset<D>(r8, 4 * lane + i)] = static_cast<uint8_t>(v8 >> (8 * i));
    }
  }
  if (lane == 0) {
    *reinterpret_cast<uint16_t*>(t8 + 16 * D + 2 * r8) = ks;
    if constexpr (!VB) *reinterpret_cast<uint16_t*>(t8 + Gm::H8B + 16 * D + 2 * r8) = vs;
  }
}

// BF16 baseline pool append: K and V stored as bf16 (no rotation, no quantisation).
template <int D, typename KT, typename VT>
__global__ void __launch_bounds__(kAppendThreads) append_bf16_kernel(AppendArgs a) {
  using Gm = Geo<D>;
  const int gw = static_cast<int>((blockIdx.x * blockDim.x + threadIdx.x) >> 5);
  const int lane = threadIdx.x & 31;
  if (gw >= a.T * a.Hkv) return;
  const int t = gw / a.Hkv, g = gw - t * a.Hkv;
  const int b = a.seq_slot[t], pos = a.pos[t];
  if (b < 0 || b >= a.max_seqs || pos < 0 || pos / a.P >= a.stride) {
    if (lane == 0) atomicOr(a.err, KV4_DEVERR_LENGTH);
    return;
  }
  const int page = a.page_table[static_cast<size_t>(b) * a.stride + pos / a.P];
  if (page < 0 || page >= a.max_pages) {
    if (lane == 0) atomicOr(a.err, KV4_DEVERR_PAGE_RANGE);
    return;
  }
  if (lane >= D / 4) return;
  float k[4], v[4];
  const size_t in0 = (static_cast<size_t>(t) * a.Hkv + g) * D + 4 * lane;
  load4<KT>(a.K, in0, k);
  load4<VT>(a.V, in0, v);
  const int pp = pos % a.P, r = pp & 15;
  uint8_t* tile = a.pool + static_cast<size_t>(page) * a.page_bytes + static_cast<size_t>(g) * a.P * 4 * D +
                  static_cast<size_t>(pp >> 4) * Gm::TBF;
  uint2 kw;
  kw.x = pack_bf2(__float2bfloat16_rn(k[0]), __float2bfloat16_rn(k[1]));
  kw.y = pack_bf2(__float2bfloat16_rn(k[2]), __float2bfloat16_rn(k[3]));
  *reinterpret_cast<uint2*>(kbf_unit<D>(tile, r, lane)) = kw;
  store_vbf<D>(tile + 32 * D, r, lane, v);
}

#define KV4_APPEND_LAUNCH(KERN, KT, VT) KERN<D, KT, VT><<<grid, block, 0, st>>>(a)
#define KV4_APPEND_LAUNCH4(KT, VT)                                   \
  do {                                                               \
    if (a.vbf) append_int4_kernel<D, KT, VT, true><<<grid, block, 0, st>>>(a); \
    else append_int4_kernel<D, KT, VT, false><<<grid, block, 0, st>>>(a);      \
  } while (0)

template <int D, bool BF16_POOL>
cudaError_t dispatch_types(const AppendArgs& a, cudaStream_t st) {
  // 8-warp blocks: a block of this kernel keeps the following decode kernel's block (which needs a
  // whole SM) off its SM until it exits, but spreading the append over more SMs ends it sooner,
  // and that measured better for the whole step than fewer 32-warp blocks (0.0606 vs 0.0633 ms).
  const int warps = a.T * a.Hkv;
  const dim3 grid((warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32)), block(kAppendThreads);
  const bool kf = a.k_dtype == KV4_F32, vf = a.v_dtype == KV4_F32;
  if (BF16_POOL) {
    if (kf && vf) KV4_APPEND_LAUNCH(append_bf16_kernel, float, float);
    else if (kf) KV4_APPEND_LAUNCH(append_bf16_kernel, float, __nv_bfloat16);
    else if (vf) KV4_APPEND_LAUNCH(append_bf16_kernel, __nv_bfloat16, float);
    else KV4_APPEND_LAUNCH(append_bf16_kernel, __nv_bfloat16, __nv_bfloat16);
  } else {
    if (kf && vf) KV4_APPEND_LAUNCH4(float, float);
    else if (kf) KV4_APPEND_LAUNCH4(float, __nv_bfloat16);
    else if (vf) KV4_APPEND_LAUNCH4(__nv_bfloat16, float);
    else KV4_APPEND_LAUNCH4(__nv_bfloat16, __nv_bfloat16);
  }
  return cudaGetLastError();
}

#undef KV4_APPEND_LAUNCH
#undef KV4_APPEND_LAUNCH4

}  // namespace

cudaError_t launch_append_int4(const AppendArgs& a, int D, cudaStream_t st) {
  if (a.T <= 0) return cudaSuccess;
  note_launches(1);
  return D == 128 ? dispatch_types<128, false>(a, st) : dispatch_types<64, false>(a, st);
}

cudaError_t launch_append_bf16(const AppendArgs& a, int D, cudaStream_t st) {
  if (a.T <= 0) return cudaSuccess;
  note_launches(1);
  return D == 128 ? dispatch_types<128, true>(a, st) : dispatch_types<64, true>(a, st);
}

}  // namespace kv4
