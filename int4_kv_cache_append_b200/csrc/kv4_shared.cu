// kv4_shared.cu -- kv4_decode_attn_shared: decode attention for batches whose sequences share prefixes.
#include "kv4_decode_kernel.cuh"
#include "kv4_quant.cuh"

namespace kv4 {
namespace {

constexpr int kRB = 64;          // query rows of a prefix segment
constexpr int kTile = 128;       // positions of a prefix unit
constexpr int kPrefixThreads = 256;

// ------------------------------------------------------------------ the prefix schedule
//
// Groups of consecutive batch rows share the pages of their prefix.  A segment is (group, KV head,
// block of kRB query rows); a query row is one query head of one sequence.  Its units are the
// 128-position tiles from the tile of the first position past the sinks to the last whole 16
// positions of the prefix.  The units of all segments form one sequence, thread block c takes
// [c Q, (c + 1) Q) of it and writes one partial (o, m, l) per row of every segment it touches, at
// index c + segment number.

struct Group {
  int b0, n;    // rows of the batch
  int te;       // prefix end, in 16-position tiles
  int tiles;    // units of a segment
  int nrb;      // row blocks
};

template <int G>
__device__ __forceinline__ Group load_group(const DecodeArgs& a, int gr, bool* bad) {
  Group r;
  const int b0 = a.group_start[gr], b1 = a.group_start[gr + 1];
  *bad = b0 < 0 || b1 < b0 || b1 > a.B;
  r.b0 = b0;
  r.n = *bad ? 0 : b1 - b0;
  r.te = clamp_len(a.prefix_len[gr], a.stride * a.P) >> 4;
  const int t0 = a.s >> 4;
  r.tiles = (r.n > 0 && 16 * r.te > a.s) ? (r.te - t0 + kTile / 16 - 1) / (kTile / 16) : 0;
  if (r.tiles == 0) r.te = 0;
  r.nrb = (r.n * G + kRB - 1) / kRB;
  return r;
}

// The schedule as one thread block sees it (shared memory).
struct Plan {
  u32 total, Q;
  u32 unit0, seg0;  // first unit and segment of group `group`
  int group;        // the group of the block's first unit (n_groups: no units)
  int bad;
};

// By warp 0.
template <int G>
__device__ void make_plan(const DecodeArgs& a, int lane, Plan& p) {
  u32 total = 0;
  bool bad = false;
  for (int base = 0; base < a.n_groups; base += 32) {
    bool b = false;
    u32 u = 0;
    if (base + lane < a.n_groups) {
      const Group g = load_group<G>(a, base + lane, &b);
      u = static_cast<u32>(a.Hkv) * g.nrb * g.tiles;
    }
    bad |= b;
    total += __shfl_sync(FULL, warp_incl_scan(u, lane), 31);
  }
  bad = __any_sync(FULL, bad);
  if (bad) total = 0;  // groups that are not consecutive rows: nothing is shared
  const u32 Q = max(1u, (total + gridDim.x - 1) / gridDim.x);
  const u32 c0 = blockIdx.x * Q;
  u32 units = 0, segs = 0;
  int found = a.n_groups;
  u32 unit0 = 0, seg0 = 0;
  for (int base = 0; base < a.n_groups && found == a.n_groups && c0 < total; base += 32) {
    u32 u = 0, s = 0;
    if (base + lane < a.n_groups) {
      bool b;
      const Group g = load_group<G>(a, base + lane, &b);
      s = g.tiles ? static_cast<u32>(a.Hkv) * g.nrb : 0u;
      u = s * g.tiles;
    }
    const u32 ui = warp_incl_scan(u, lane), si = warp_incl_scan(s, lane);
    const unsigned m = __ballot_sync(FULL, c0 < units + ui);
    if (m) {
      const int l = __ffs(m) - 1;
      found = base + l;
      unit0 = units + __shfl_sync(FULL, ui - u, l);
      seg0 = segs + __shfl_sync(FULL, si - s, l);
    }
    units += __shfl_sync(FULL, ui, 31);
    segs += __shfl_sync(FULL, si, 31);
  }
  if (lane == 0) {
    p.total = total;
    p.Q = Q;
    p.unit0 = unit0;
    p.seg0 = seg0;
    p.group = found;
    p.bad = bad;
    if (bad && blockIdx.x == 0) atomicOr(a.err, KV4_DEVERR_GROUP);
  }
}

// Rows without a prefix partial, and every row's first own tile: spread over the thread blocks.
template <int G>
__device__ void write_rows(const DecodeArgs& a, const Plan& p) {
  auto plain = [&](int b) {
    a.own[b] = 0;
    for (int g = 0; g < a.Hkv; ++g) a.pmeta[b * a.Hkv + g] = make_uint4(0u, 0u, 0u, 0u);
  };
  const int tid = threadIdx.x, nt = blockDim.x;
  const int all = gridDim.x * nt, me = blockIdx.x * nt + tid;
  if (p.bad || a.n_groups == 0) {
    for (int b = me; b < a.B; b += all) plain(b);
    return;
  }
  const int lo = a.group_start[0], hi = a.group_start[a.n_groups];
  for (int b = me; b < a.B; b += all)
    if (b < lo || b >= hi) plain(b);
  for (int gr = blockIdx.x; gr < a.n_groups; gr += gridDim.x) {
    bool bad;
    const Group g = load_group<G>(a, gr, &bad);
    for (int i = tid; i < g.n; i += nt) {
      if (g.tiles == 0) plain(g.b0 + i);
      else a.own[g.b0 + i] = g.te;
    }
  }
}

// ------------------------------------------------------------------ prefix attention

template <int D>
struct SmemPrefix {
  float K[kTile][D + 1];
  float V[kTile][D];
  float q[kRB][D];
  float o[kRB][D];
  float p[kPrefixThreads / 32][kTile];
  float m[kRB], l[kRB];
  int lim[kRB];
  Plan plan;
};

template <int D, int G, int QT>
__global__ void __launch_bounds__(kPrefixThreads) prefix_kernel(const DecodeArgs a) {
  using Gm = Geo<D>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  SmemPrefix<D>& sm = *reinterpret_cast<SmemPrefix<D>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cap = a.stride * a.P;
  pdl_wait();
  if (warp == 0) make_plan<G>(a, lane, sm.plan);
  __syncthreads();
  write_rows<G>(a, sm.plan);
  const u32 Q = sm.plan.Q;
  u32 c = blockIdx.x * Q;
  const u32 c1 = min(c + Q, sm.plan.total);
  int gr = sm.plan.group;
  u32 unit0 = sm.plan.unit0, seg0 = sm.plan.seg0;
  while (c < c1) {
    bool bad;
    const Group grp = load_group<G>(a, gr, &bad);
    const u32 nseg = static_cast<u32>(a.Hkv) * grp.nrb;
    if (grp.tiles == 0 || c >= unit0 + nseg * grp.tiles) {
      if (grp.tiles) {
        unit0 += nseg * grp.tiles;
        seg0 += nseg;
      }
      ++gr;
      continue;
    }
    const u32 sg = (c - unit0) / grp.tiles;
    const u32 us = unit0 + sg * grp.tiles;  // first unit of the segment
    const int g = static_cast<int>(sg / grp.nrb), rb = static_cast<int>(sg % grp.nrb);
    const int rows = min(kRB, grp.n * G - rb * kRB);
    const int bfirst = grp.b0 + rb * (kRB / G);
    const u32 ce = min(c1, us + grp.tiles);
    // queries
    for (int r = warp; r < kRB; r += kPrefixThreads / 32) {
      const int b = bfirst + r / G;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      const bool act = lane < D / 4;
      if (r < rows && act) {
        const size_t q0 = (static_cast<size_t>(b) * a.Hq + static_cast<size_t>(g) * G + r % G) * D + 4 * lane;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = load_q<QT>(a.q, q0 + e);
      }
      flip_signs4(x, lane, a.signs);
      hadamard4(x, lane, a.h);
      if (act) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sm.q[r][4 * lane + e] = x[e] * (a.qscale / a.h);
          sm.o[r][4 * lane + e] = 0.f;
        }
      }
      if (lane == 0) {
        sm.m[r] = kNegInf;
        sm.l[r] = 0.f;
        sm.lim[r] = r < rows ? min(16 * grp.te, max(a.s, clamp_len(a.lens[b], cap) - a.w)) : 0;
      }
    }
    if (c == us) {
      const u32 last = (us + grp.tiles - 1) / Q;
      for (int i = tid; i * G < rows; i += kPrefixThreads)
        a.pmeta[(bfirst + i) * a.Hkv + g] = make_uint4(blockIdx.x + seg0 + sg, last - blockIdx.x + 1, i * G, 0u);
    }
    __syncthreads();
    for (; c < ce; ++c) {
      const int t0 = (a.s >> 4) + static_cast<int>(c - us) * (kTile / 16);  // first 16-position tile
      for (int i = tid; i < kTile * D; i += kPrefixThreads) {
        const int pos = i / D, d = i % D, ti = t0 + (pos >> 4), r = pos & 15;
        float k = 0.f, v = 0.f;
        if (ti < grp.te) {
          int lp, tin;
          tile_page(a, ti, &lp, &tin);
          const int page = a.page_table[static_cast<size_t>(grp.b0) * a.stride + lp];
          if (page >= 0 && page < a.max_pages) {
            uint8_t* tile = const_cast<uint8_t*>(a.pool) + static_cast<size_t>(page) * a.page_bytes +
                            (static_cast<size_t>(g) * (a.P / 16) + tin) * Gm::T4B;
            const uint32_t kp = *reinterpret_cast<const uint32_t*>(tile + 16 * D + 4 * r);
            const uint32_t vp = *reinterpret_cast<const uint32_t*>(tile + 16 * D + 64 + 4 * r);
            const uint32_t kw = k4_words<D>(tile, r & 7, d >> 2)[d & 1] >> (16 * ((d >> 2) & 1) + 4 * (r >> 3) + 8 * ((d >> 1) & 1));
            k = fmaf(half_lo(kp), static_cast<float>(kw & 15u), half_hi(kp));
            v = fmaf(half_lo(vp), static_cast<float>((*v4_chunk<D>(tile, r, d >> 2) >> (4 * (d & 3))) & 15), half_hi(vp));
          } else if (d == 0 && r == 0) {
            atomicOr(a.err, KV4_DEVERR_PAGE_RANGE);
          }
        }
        sm.K[pos][d] = k;
        sm.V[pos][d] = v;
      }
      __syncthreads();
      for (int r = warp; r < rows; r += kPrefixThreads / 32) {
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        for (int d = 0; d < D; ++d) {
          const float qv = sm.q[r][d];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = fmaf(qv, sm.K[lane + 32 * i][d], x[i]);
        }
        float mx = kNegInf;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int pos = 16 * t0 + lane + 32 * i;
          if (pos < a.s || pos >= sm.lim[r]) x[i] = kNegInf;
          mx = fmaxf(mx, x[i]);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
        const float mo = sm.m[r], mn = fmaxf(mo, mx);
        if (mn == kNegInf) continue;
        const float alpha = mo == kNegInf ? 0.f : exp2f(mo - mn);
        float ls = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float pv = exp2f(x[i] - mn);
          sm.p[warp][lane + 32 * i] = pv;
          ls += pv;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) ls += __shfl_xor_sync(FULL, ls, o);
        __syncwarp();
        for (int d = lane; d < D; d += 32) {
          float acc = sm.o[r][d] * alpha;
          for (int t = 0; t < kTile; ++t)
            if (sm.p[warp][t] != 0.f) acc = fmaf(sm.p[warp][t], sm.V[t][d], acc);
          sm.o[r][d] = acc;
        }
        if (lane == 0) {
          sm.m[r] = mn;
          sm.l[r] = sm.l[r] * alpha + ls;
        }
        __syncwarp();
      }
      __syncthreads();
    }
    float* part = a.ppart + static_cast<size_t>(blockIdx.x + seg0 + sg) * kRB * kPartRow<D>;
    for (int i = tid; i < rows * D; i += kPrefixThreads) part[(i / D) * kPartRow<D> + i % D] = sm.o[i / D][i % D];
    for (int r = tid; r < rows; r += kPrefixThreads) {
      part[r * kPartRow<D> + D] = sm.m[r];
      part[r * kPartRow<D> + D + 1] = sm.l[r];
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ merge of prefix and own partials

template <int DT>
__device__ __forceinline__ void store_out(void* out, size_t i, float x) {
  if constexpr (DT == KV4_F32) reinterpret_cast<float*>(out)[i] = x;
  else if constexpr (DT == KV4_BF16) reinterpret_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(x);
  else reinterpret_cast<__half*>(out)[i] = __float2half_rn(x);
}

// One warp per (sequence, query head).
template <int D, int G, int DT>
__global__ void __launch_bounds__(128) merge_shared_kernel(const DecodeArgs a) {
  constexpr int PER = D / 32, RS = kPartRow<D>;
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= a.B * a.Hq) return;
  const int b = item / a.Hq, j = item - b * a.Hq, g = j / G, hd = j - g * G;
  pdl_wait();
  const uint4 mt = *reinterpret_cast<const uint4*>(a.meta + 4 * (b * a.Hkv + g));
  const uint4 pm = a.pmeta[b * a.Hkv + g];
  {
    const unsigned long long rows = static_cast<unsigned long long>(a.W) + 2ull * a.B * a.Hkv;
    const unsigned long long sid8 = 2ull * (b * a.Hkv + g);
    const bool bad8 = mt.z && static_cast<unsigned long long>(mt.x) + mt.z + sid8 > rows;
    const bool bad4 = mt.w && static_cast<unsigned long long>(mt.y) + mt.w + sid8 + 1ull > rows;
    if (bad8 || bad4 || mt.z > rows || mt.w > rows) {
      if (lane == 0) atomicOr(a.err, KV4_DEVERR_RECORD);
      return;
    }
  }
  const int n8p = static_cast<int>(mt.z), nown = static_cast<int>(mt.z + mt.w), n = nown + static_cast<int>(pm.y);
  const PartRows pr{n8p, mt.x, mt.y, 2u * static_cast<u32>(b * a.Hkv + g)};
  float M = kNegInf, L = 0.f, o[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = 0.f;
  for (int t = 0; t < n; ++t) {
    const float* row = t < nown ? a.part + pr.row(t, G, RS) + hd * RS
                                : a.ppart + (static_cast<size_t>(pm.x + (t - nown)) * kRB + pm.z + hd) * RS;
    const float m = row[D], l = row[D + 1];
    if (!(l > 0.f)) continue;
    const float mn = fmaxf(M, m), f0 = M == kNegInf ? 0.f : exp2f(M - mn), f1 = exp2f(m - mn);
    L = L * f0 + l * f1;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = o[e] * f0 + f1 * row[lane * PER + e];
    M = mn;
  }
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
  const size_t o0 = (static_cast<size_t>(b) * a.Hq + j) * D + lane * PER;
#pragma unroll
  for (int e = 0; e < PER; ++e) store_out<DT>(a.out, o0 + e, o[e]);
  if (a.lse && lane == 0) a.lse[static_cast<size_t>(b) * a.Hq + j] = L > 0.f ? (M + log2f(L)) * 0.69314718055994531f : kNegInf;
}

template <int D, int G, int QT>
cudaError_t launch_all(const DecodeArgs& a, int ctas, cudaStream_t st) {
  static std::atomic<uint64_t> done_prefix, done_decode[2];
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int smem = static_cast<int>(sizeof(SmemPrefix<D>));
  cudaError_t e = ensure_smem_limit(prefix_kernel<D, G, QT>, smem, done_prefix);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(a.PW));
  cfg.blockDim = dim3(kPrefixThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  e = cudaLaunchKernelEx(&cfg, prefix_kernel<D, G, QT>, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kWarps * 32);
  e = a.nt8 > kTightSideTiles ? launch_variant<D, G, QT, true, false, true>(cfg, a, done_decode[1])
                              : launch_variant<D, G, QT, false, false, true>(cfg, a, done_decode[0]);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>((a.B * a.Hq + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  if (a.out_dtype == KV4_F32) return cudaLaunchKernelEx(&cfg, merge_shared_kernel<D, G, KV4_F32>, a);
  if (a.out_dtype == KV4_BF16) return cudaLaunchKernelEx(&cfg, merge_shared_kernel<D, G, KV4_BF16>, a);
  return cudaLaunchKernelEx(&cfg, merge_shared_kernel<D, G, KV4_F16>, a);
}

template <int D, int G>
cudaError_t launch_types(const DecodeArgs& a, int ctas, cudaStream_t st) {
  if (a.q_dtype == KV4_F32) return launch_all<D, G, KV4_F32>(a, ctas, st);
  if (a.q_dtype == KV4_BF16) return launch_all<D, G, KV4_BF16>(a, ctas, st);
  return launch_all<D, G, KV4_F16>(a, ctas, st);
}

}  // namespace

int shared_row_block() { return kRB; }

cudaError_t launch_decode_shared(DecodeArgs a, int D, int G, int ctas, cudaStream_t st) {
  a.W = ctas * kWarps;
  note_launches(3);
  if (D == 128) {
    if (G == 4) return launch_types<128, 4>(a, ctas, st);
    if (G == 2) return launch_types<128, 2>(a, ctas, st);
    return launch_types<128, 1>(a, ctas, st);
  }
  if (G == 4) return launch_types<64, 4>(a, ctas, st);
  if (G == 2) return launch_types<64, 2>(a, ctas, st);
  return launch_types<64, 1>(a, ctas, st);
}

}  // namespace kv4
