// kv4_decode.cu -- kv4_decode_attn on the INT4 cache: the split-K kernel (kv4_decode_kernel.cuh) and the
// LSE merge of its partials.
#include "kv4_decode_kernel.cuh"

namespace kv4 {
namespace {

// ------------------------------------------------------------------ LSE merge kernel

// Merge of the partials of (sequence b, query head j): MW warps per (b, j), MW chosen on the host
// so that a warp has at most kMergeBatch partials (MW = 1: four (b, j) per CTA of 4 warps; else one
// (b, j) per CTA of MW warps).  The decode kernel left, per (b, g), where the n partials are
// (meta); warp w of the MW merges head j % G of partials [w n / MW, (w+1) n / MW) in one pass of
// batches of kMergeBatch rows, each batch one round trip.  With MW > 1, warp 0 combines the
// warps' (M, L, o) through shared memory.  (b, g) with at most one partial, and sequences of
// length 0 (record of zeros), were written by the decode kernel.  Launched as a programmatic
// dependent of the decode kernel: griddepcontrol.wait orders every read of its results after its
// completion.
constexpr int kMergeThreads = 128;
constexpr int kMergeBatch = 16;

template <int D, int G, int MW>
__global__ void __launch_bounds__(MW == 1 ? kMergeThreads : 32 * MW) merge_int4_kernel(const DecodeArgs a) {
  constexpr int PER = D / 32;
  constexpr int kInFlight = kMergeBatch;
  constexpr int RS = kPartRow<D>;
  using VecT = typename std::conditional<PER == 4, float4, float2>::type;
  __shared__ float smo[MW][D];
  __shared__ float smM[MW], smL[MW];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = MW == 1 ? 0 : warp;                       // warp within the item
  const int item = MW == 1 ? blockIdx.x * (kMergeThreads / 32) + warp : blockIdx.x;
  if (item >= a.B * a.Hq) return;
  const int b = item / a.Hq, j = item - b * a.Hq;
  const int g = j / G, hd = j - g * G;
  pdl_wait();
  const uint4 mt = *reinterpret_cast<const uint4*>(a.meta + 4 * (b * a.Hkv + g));
  {
    // A record whose partial rows fall outside the workspace can only be left over from a decode
    // that stopped early (a wait that ran out): report it and write no output from it.
    const unsigned long long rows = static_cast<unsigned long long>(a.W) + 2ull * a.B * a.Hkv;
    const unsigned long long sid8 = 2ull * (b * a.Hkv + g);
    const bool bad8 = mt.z && static_cast<unsigned long long>(mt.x) + mt.z + sid8 > rows;
    const bool bad4 = mt.w && static_cast<unsigned long long>(mt.y) + mt.w + sid8 + 1ull > rows;
    if (bad8 || bad4 || mt.z > rows || mt.w > rows) {
      if (lane == 0 && sub == 0) atomicOr(a.err, KV4_DEVERR_RECORD);
      return;
    }
  }
  const int n8p = static_cast<int>(mt.z), n = static_cast<int>(mt.z + mt.w);
  if (n == 0 || (n == 1 && !a.rotate_v)) return;  // uniform over the item's warps
  const PartRows pr{n8p, mt.x, mt.y, 2u * static_cast<u32>(b * a.Hkv + g)};
  const int t0 = sub * n / MW, t1 = (sub + 1) * n / MW;
  float M = kNegInf, L = 0.f, o[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = 0.f;
  // One pass, kInFlight partials at a time: every lane loads its slice of each row together with
  // the row's (m, l) (the same address in every lane), so a batch costs one memory round trip; the
  // running maximum is raised partial by partial (warp-uniform).
  for (int base = t0; base < t1; base += kInFlight) {
    VecT v[kInFlight];
    float2 ml[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int t = base + u < t1 ? base + u : t0;  // past the end: reload the first row, unused
      const unsigned long long row = pr.row(t, G, RS) + hd * RS;
      v[u] = __ldcg(reinterpret_cast<const VecT*>(a.part + row + lane * PER));
      ml[u] = __ldcg(reinterpret_cast<const float2*>(a.part + row + D));
    }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      if (base + u >= t1 || !(ml[u].y > 0.f)) continue;
      if (ml[u].x > M) {
        const float sc = M == kNegInf ? 0.f : exp2f(M - ml[u].x);
        L *= sc;
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] *= sc;
        M = ml[u].x;
      }
      const float w = exp2f(ml[u].x - M);
      L = fmaf(w, ml[u].y, L);
      const float* vv = reinterpret_cast<const float*>(&v[u]);
#pragma unroll
      for (int e = 0; e < PER; ++e) o[e] = fmaf(w, vv[e], o[e]);
    }
  }
  if constexpr (MW > 1) {
#pragma unroll
    for (int e = 0; e < PER; ++e) smo[sub][lane * PER + e] = o[e];
    if (lane == 0) {
      smM[sub] = M;
      smL[sub] = L;
    }
    __syncthreads();
    if (sub != 0) return;
    M = kNegInf;
#pragma unroll
    for (int w = 0; w < MW; ++w)
      if (smL[w] > 0.f) M = fmaxf(M, smM[w]);
    L = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = 0.f;
#pragma unroll
    for (int w = 0; w < MW; ++w) {
      const float f = smL[w] > 0.f ? exp2f(smM[w] - M) : 0.f;
      L += f * smL[w];
#pragma unroll
      for (int e = 0; e < PER; ++e) o[e] = fmaf(f, smo[w][lane * PER + e], o[e]);
    }
  }
  float* out = a.out + (static_cast<size_t>(b) * a.Hq + j) * D + lane * PER;
  const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] *= inv;
  if (a.rotate_v) {
    // values were stored as H diag(s) v: o = diag(s) H o_rot / h (lane holds dims PER lane + e)
    const int h = a.h;
#pragma unroll
    for (int st = 1; st < PER; st <<= 1)
      if (st < h)
#pragma unroll
        for (int e = 0; e < PER; ++e)
          if ((e & st) == 0) {
            const float x0 = o[e], x1 = o[e + st];
            o[e] = x0 + x1;
            o[e + st] = x0 - x1;
          }
#pragma unroll
    for (int st = PER; st < D; st <<= 1)
      if (st < h) {
        const int m = st / PER;
        const bool upper = (lane & m) != 0;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          const float x = __shfl_xor_sync(FULL, o[e], m);
          o[e] = upper ? x - o[e] : o[e] + x;
        }
      }
    const float ih = 1.f / static_cast<float>(h);
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int d = lane * PER + e;
      o[e] = __uint_as_float(__float_as_uint(o[e] * ih) ^ (((a.signs[d >> 5] >> (d & 31)) & 1u) << 31));
    }
  }
  if constexpr (PER == 4)
    *reinterpret_cast<float4*>(out) = make_float4(o[0], o[1], o[2], o[3]);
  else
    *reinterpret_cast<float2*>(out) = make_float2(o[0], o[1]);
  if (a.lse && lane == 0) a.lse[static_cast<size_t>(b) * a.Hq + j] = L > 0.f ? (M + log2f(L)) * 0.69314718055994531f : kNegInf;
}

// Launch of the merge kernel as a programmatic dependent of the preceding decode kernel.
template <int D, int G>
cudaError_t launch_merge(const DecodeArgs& a, cudaStream_t st) {
  const int items = a.B * a.Hq;
  // partials of an average (b, g): its share of the split warps, plus the two segment ends
  const long long per = static_cast<long long>(a.W) / (static_cast<long long>(a.B) * a.Hkv) + 2;
  const int mw = per <= kMergeBatch ? 1 : per <= 4 * kMergeBatch ? 4 : per <= 8 * kMergeBatch ? 8 : 16;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(mw > 1 ? items : (items + kMergeThreads / 32 - 1) / (kMergeThreads / 32)));
  cfg.blockDim = dim3(mw > 1 ? 32 * mw : kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (mw) {
    case 1: return cudaLaunchKernelEx(&cfg, merge_int4_kernel<D, G, 1>, a);
    case 4: return cudaLaunchKernelEx(&cfg, merge_int4_kernel<D, G, 4>, a);
    case 8: return cudaLaunchKernelEx(&cfg, merge_int4_kernel<D, G, 8>, a);
    default: return cudaLaunchKernelEx(&cfg, merge_int4_kernel<D, G, 16>, a);
  }
}

template <int D, int G, int QT>
cudaError_t launch_qt(const cudaLaunchConfig_t& cfg, const DecodeArgs& a, std::atomic<uint64_t>* done) {
  // bf16 values: every side tile is visited (masked), so one kernel serves every side-cache size
  if (a.vbf) return launch_variant<D, G, QT, false, true, false>(cfg, a, done[2]);
  if (a.nt8 > kTightSideTiles) return launch_variant<D, G, QT, true, false, false>(cfg, a, done[1]);
  return launch_variant<D, G, QT, false, false, false>(cfg, a, done[0]);
}

template <int D, int G>
cudaError_t launch_dg(const DecodeArgs& a, int ctas, cudaStream_t st) {
  static std::atomic<uint64_t> done[3][3];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (a.q_dtype == KV4_F32) e = launch_qt<D, G, KV4_F32>(cfg, a, done[0]);
  else if (a.q_dtype == KV4_BF16) e = launch_qt<D, G, KV4_BF16>(cfg, a, done[1]);
  else e = launch_qt<D, G, KV4_F16>(cfg, a, done[2]);
  if (e != cudaSuccess) return e;
  return launch_merge<D, G>(a, st);
}

}  // namespace

int decode_warps_per_cta() { return kWarps; }
int decode_ctas_per_sm() { return kCtasPerSm; }

size_t decode_smem_bytes(int D, int G) {
  (void)G;
  return D == 128 ? sizeof(Smem<128, true>) : sizeof(Smem<64, true>);
}

cudaError_t launch_decode_int4(DecodeArgs a, int D, int G, int ctas, cudaStream_t st) {
  a.W = ctas * kWarps;
  note_launches(2);
  if (D == 128) {
    if (G == 4) return launch_dg<128, 4>(a, ctas, st);
    if (G == 2) return launch_dg<128, 2>(a, ctas, st);
    return launch_dg<128, 1>(a, ctas, st);
  }
  if (G == 4) return launch_dg<64, 4>(a, ctas, st);
  if (G == 2) return launch_dg<64, 2>(a, ctas, st);
  return launch_dg<64, 1>(a, ctas, st);
}

}  // namespace kv4
