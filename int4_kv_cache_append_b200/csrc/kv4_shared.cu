// kv4_shared.cu -- kv4_decode_attn_shared: decode attention for batches whose sequences share prefixes.
//
// The prefix of a group is one attention of many query rows (sequences x query heads of a KV head)
// over the same keys, so it runs on the tensor cores: positions are the 128 rows of the MMA, query
// rows its columns.  Per 128-position unit of one KV head
//   S^T [position][row]  = codes of K [128][D]  x  Q^T [D][rows]
//   logit                = s_t S + z_t sum(q)        (scale and zero after the reduction, fp32)
//   P                    = exp2(logit - m_row)       (fp16)
//   O^T [dim][row]      += V^T [D][128]         x  P [128][rows]
// The codes go from the packed page tile straight into TMEM as the A operands: a key code is the
// fp16 subnormal c 2^-24 (one mask, exact), a value is dequantised to fp16 (z + s c, one rounding).
// Keeping A in TMEM leaves shared memory to the packed tiles, Q and P; with the positions as the
// MMA's rows its cost follows the number of query rows, and s_t and z_t are one thread's constants.
//
// A thread block is 26 warps: four softmax warpgroups (16 of the 64 columns each, a thread per
// position), a warpgroup unpacking keys, one unpacking values, a warp of bulk copies and a warp
// that issues the MMAs; K, V, S and P have two buffers, the packed tiles four.  The running maximum
// of a row is set 4 (log2) below its largest logit and raised only when one exceeds it by more than
// 15 (P then stays inside fp16): the first unit of a segment sets it, later ones seldom rescale O.
//
// What bounds it: 16 prompts of up to 8 K positions with up to 16 answers each, 32 + 8 heads of 128,
// take 147 us (one by one the prefix kernel 111, own positions 39, merge 11) for 217 MB that have to be
// read, 33 us at copy speed; one prompt of 16 K with 128 answers 143 us for 35 GFLOP.  A unit of 64
// rows takes a CTA about 3200 cycles: the tensor pipe is 16% active, 58% of the issue slots are taken,
// and a warp issues every eleventh cycle, its waits being the fixed latencies of the softmax chain
// (TMEM load, two packed FMAs, exp2, conversion, store) and the hand-overs between roles: all 16 softmax
// warps work on the same unit at the same time.  A group of more than 64 query rows unpacks its pages once
// for every 64.  It pays for groups of 16 rows from about 256 K attended positions in all, of 4 from a
// million; else kv4_decode_attn is faster, since rows that share pages find them in L2 (64 rows over 8 K
// positions each, as groups of 2, 4, 16 and 64: 194, 122, 87, 87 us here, 116 there).  Eight
// softmax warps of 32 columns, with more registers each, took 165 us where sixteen of 16 took 157.
#include "kv4_decode_kernel.cuh"
#include "kv4_quant.cuh"
#include "kv4_tcgen05.cuh"

namespace kv4 {
namespace {

constexpr int kRB = 64;          // query rows of a prefix segment: the MMA's columns
constexpr int kTile = 128;       // positions of a prefix unit: the MMA's rows
constexpr int kRaw = 4;          // buffers of packed tiles

// The loops' rare branches: their code goes out of the way of the straight path, whose instruction
// fetch a taken branch would interrupt.
__device__ __forceinline__ bool unlikely(bool x) { return __builtin_expect(x, 0); }

// ------------------------------------------------------------------ the prefix schedule
//
// Groups of consecutive batch rows share the pages of their prefix; a single row shares nothing and is left
// to the split-K kernel (64 of them over 4 K positions each: 207 us here, 70 there).  A segment is (group, KV head,
// block of kRB query rows); a query row is one query head of one sequence.  Its units are the
// 128-position tiles from the tile of the first position past the sinks to the end of the prefix's last
// whole page (what lies past it is in each sequence's own page).  The units of all segments form one sequence, thread block c takes
// [c Q, (c + 1) Q) of it and writes one partial (o, m, l) per row of every segment it touches, at
// index c + segment number.

struct Group {
  int b0, n;    // rows of the batch
  int te;       // end of the prefix's whole pages, in 16-position tiles
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
  const int tpp = a.P >> 4, tl = clamp_len(a.prefix_len[gr], a.stride * a.P) >> 4;
  r.te = a.tp_shift >= 0 ? tl >> a.tp_shift << a.tp_shift : tl / tpp * tpp;
  const int t0 = a.s >> 4;
  r.tiles = (r.n > 1 && 16 * r.te > a.s) ? (r.te - t0 + kTile / 16 - 1) / (kTile / 16) : 0;
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

// Rows without a prefix partial, and every row's first own tile: spread over the thread blocks, one
// warp of each.
template <int G>
__device__ void write_rows(const DecodeArgs& a, const Plan& p, int lane) {
  auto plain = [&](int b) {
    a.own[b] = 0;
    for (int g = 0; g < a.Hkv; ++g) a.pmeta[b * a.Hkv + g] = make_uint4(0u, 0u, 0u, 0u);
  };
  const int all = gridDim.x * 32, me = blockIdx.x * 32 + lane;
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
    for (int i = lane; i < g.n; i += 32) {
      if (g.tiles == 0) plain(g.b0 + i);
      else a.own[g.b0 + i] = g.te;
    }
  }
}

// ------------------------------------------------------------------ prefix attention

constexpr int kSoftGroups = 4;   // softmax warpgroups: group g takes the 8-column chunks g and g + 4
constexpr int kChunks = kRB / 8 / kSoftGroups;
constexpr int kSoftWarps = 4 * kSoftGroups, kKeyWarp0 = kSoftWarps, kValWarp0 = kKeyWarp0 + 4, kCopyWarp = kValWarp0 + 4,
              kMmaWarp = kCopyWarp + 1, kSoftThreads = 32 * kSoftWarps;
constexpr int kPrefixThreads = 32 * (kMmaWarp + 1);
constexpr float kUnset = -1e30f;   // running maximum of a row that has seen no position
// A raised running maximum is set kLift (log2) below the largest logit, so probabilities start at 2^kLift and
// what fp16 takes as zero is below 2^(-25 - kLift) of the largest: the 10^5 positions that a thread block
// may take lose 2^-12 of it at most, less than the roundings (from 1 on they lost 2^-8, which the sums
// counted and the products did not).  A logit kGrow above raises it again: probabilities end at 2^15.
// With 4 a logit may grow by 2^11 before that, as it could with 0 (no difference in time); with 6 and 8
// the rescaling cost 1% and 2 to 4% (128 answers to one prompt of 16 K: 158.8, 160.6, 164.9 us).
constexpr float kLift = 4.f;
constexpr float kGrow = 15.f;
constexpr float kGrowLarge = 11.f;  // with values taken times 1/16: probabilities are then times 16
constexpr float kQShift = 64.f;    // queries enter fp16 times this: typical ones are then near one

// The units of this thread block, segment by segment: every warp walks them on its own.  The state
// lives in shared memory (it is read once a segment; the loops over units need the registers).
struct Segment {
  u32 at, end, unit0, seg0;  // next and last unit of the block; first unit and segment of group gr
  int gr;
  int te, b0;                // the group's prefix end (16-position tiles) and first row
  int g, rows, bfirst;       // KV head, query rows, first sequence
  int p0;                    // first position
  u32 n;                     // units
  u32 slot, blocks;          // partial index; thread blocks from this one on (0: not the segment's first)
};

template <int D>
struct SmemPrefix {
  uint8_t raw[kRaw][8 * Geo<D>::T4B];
  __half P[2][kRB * kTile];   // [row / 8][position][row % 8]: MN-major core matrices
  __half Q[kRB * D];          // [k / 8][row][k % 8]: K-major core matrices
  float4 cst[kRB / 2];        // rows 2j, 2j + 1: sum(q), sum(q), -m, -m
  alignas(8) float mul[kRB];             // rows whose query had to be scaled down to fit fp16: the factor back
  alignas(16) float alpha[kRB];
  float red[kSoftGroups][4][kRB / kSoftGroups];
  float2 ksz[kRaw][kTile];    // key scale (times the codes' and queries' powers of two) and zero
  alignas(16) uint32_t odd[kRaw][4];  // per key warp (two tiles): bit 0 values beyond fp16, bits 1, 2 a tile was not copied
  int lim[kRB];               // end of the row's INT4 positions in the prefix
  int edge;                   // smallest lim of the rows
  int scaled;                 // some row has mul != 1
  uint32_t ok[kRaw];          // tiles of the buffer that were copied
  uint64_t raw_full[kRaw], raw_empty[kRaw];
  uint64_t k_ready[2], v_ready[2], qk_done[2], p_ready[2], pv_done[2];
  uint64_t q_ready;
  uint64_t drained;           // the MMA warp's last commit
  uint64_t stall;             // never arrived on (kv4_debug_force_wait_timeout)
  uint32_t tmem;
  int abort;
  Plan plan;
  Segment seg[kPrefixThreads / 32];
};

// TMEM columns: keys and values as A operands (two fp16 a column), scores, outputs.
template <int D>
struct Cols {
  static constexpr int K = 0, V = 2 * (D / 2), S = V + 2 * (kTile / 2), O = S + 2 * kRB, All = 512;
  static_assert(O + kRB <= All, "TMEM columns");
};

// The same value in every lane, known as such to the compiler: branches on it need no reconvergence.
template <typename T>
__device__ __forceinline__ T uniform(T x) { return __shfl_sync(FULL, x, 0); }

// Up to N polls of a phase.
template <int N>
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, 0;\n"
      "KV4_POLL_%=:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra KV4_DONE_%=;\n"
      " add.u32 n, n, 1;\n setp.lt.u32 q, n, %3;\n @q bra KV4_POLL_%=;\n"
      "KV4_DONE_%=:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "n"(N)
      : "memory");
  return ok != 0;
}

// A bounded wait that gives up when any warp of the block has.  Then the warps that meet at hardware
// barriers run their loops to the end, each wait costing a few polls, on whatever the buffers hold; the
// copy warp starts no more copies, and the last commit's barrier says when the products are done.  A
// warpgroup waits by one warp, the others at a hardware barrier: polls by every warp were half of the
// issued instructions.
__device__ __forceinline__ void wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* err, uint64_t limit_ns) {
  const uint32_t at = smem_u32(bar);
  if (unlikely(!poll<4>(at, parity))) {
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t it = 0;; ++it) {
      if (*abort || poll<64>(at, parity)) return;
      const uint64_t t = global_timer_ns();
      if (it == 0) t0 = t;
      if (t - t0 > limit_ns || it >= kWaitLimitPolls / 64) {
        *abort = 1;
        atomicOr(err, KV4_DEVERR_WAIT_LIMIT);
        return;
      }
    }
  }
}

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) arrive(bar);
}

// One of the softmax warpgroups in step, with the OR of a predicate.
__device__ __forceinline__ bool group_or(int id, bool x) {
  uint32_t r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 q, %1, 0;\n barrier.cta.red.or.pred p, %2, 128, q;\n selp.b32 %0, 1, 0, p;\n}\n"
               : "=r"(r)
               : "r"(static_cast<uint32_t>(x)), "r"(id)
               : "memory");
  return r != 0;
}
__device__ __forceinline__ void soft_sync() { asm volatile("barrier.cta.sync 5, %0;" ::"n"(kSoftThreads) : "memory"); }
__device__ __forceinline__ void group_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }

__device__ __forceinline__ void walk_start(Segment& s, const Plan& p, int lane) {
  if (lane == 0) {
    s.at = blockIdx.x * p.Q;
    s.end = min(blockIdx.x * p.Q + p.Q, p.total);
    s.unit0 = p.unit0;
    s.seg0 = p.seg0;
    s.gr = p.group;
  }
  __syncwarp();
}

template <int G>
__device__ __forceinline__ bool walk_next(const DecodeArgs& a, const Plan& p, Segment& s, int lane) {
  u32 c = s.at, unit0 = s.unit0, seg0 = s.seg0;
  int gr = s.gr;
  __syncwarp();
  while (c < s.end) {
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
    const u32 sg = (c - unit0) / grp.tiles, us = unit0 + sg * grp.tiles, ce = min(s.end, us + grp.tiles);
    const int rb = static_cast<int>(sg % grp.nrb);
    if (lane == 0) {
      s.at = ce;
      s.unit0 = unit0;
      s.seg0 = seg0;
      s.gr = gr;
      s.te = grp.te;
      s.b0 = grp.b0;
      s.g = static_cast<int>(sg / grp.nrb);
      s.rows = min(kRB, grp.n * G - rb * kRB);
      s.bfirst = grp.b0 + rb * (kRB / G);
      s.p0 = 16 * (a.s >> 4) + static_cast<int>(c - us) * kTile;
      s.n = ce - c;
      s.slot = blockIdx.x + seg0 + sg;
      s.blocks = c == us ? (us + grp.tiles - 1) / p.Q - blockIdx.x + 1 : 0;
    }
    __syncwarp();
    return true;
  }
  return false;
}

// End of the positions that some row of the segment attends; those past it may be unwritten.
template <int G>
__device__ __forceinline__ int attended_end(const DecodeArgs& a, const Segment& s, int cap, int lane) {
  int hi = 0;
  for (int r = lane; r * G < s.rows; r += 32) hi = max(hi, clamp_len(a.lens[s.bfirst + r], cap) - a.w);
#pragma unroll
  for (int o = 16; o; o >>= 1) hi = max(hi, __shfl_xor_sync(FULL, hi, o));
  return min(hi, 16 * s.te);
}

// Row of the A operand's k order that dimension d takes (the order in which unpack_keys meets it).
template <int D>
__device__ __forceinline__ int key_order(int d) {
  constexpr int NU = D / 64;
  const int group = d >> 3, u = group >> 1, j = 2 * (group & 1) + (d & 1), pair = (d >> 1) & 1, hi = (d >> 2) & 1;
  const int i = 8 * (u % NU) + 2 * j + pair;
  return 2 * (4 * i + u / NU) + hi;
}

// Key codes of two tiles (this warp's 32 TMEM lanes) to fp16 subnormals: thread t reads pair-row t / 4
// (rows t / 4 in the low nibbles, t / 4 + 8 in the high ones, kept as 16 c), 16 NU bytes of it; the
// 8 lanes of a shared-memory phase read 8 different 16-byte units.
template <int D>
__device__ __forceinline__ void unpack_keys(const uint8_t* raw, uint32_t tmem, int w, int lane) {
  constexpr int NU = D / 64;
  const int pr = lane >> 2, q = lane & 3;
#pragma unroll 1
  for (int t = 0; t < 2; ++t) {
    const uint8_t* row = raw + (2 * w + t) * Geo<D>::T4B + pr * D;
#pragma unroll
    for (int ul = 0; ul < NU; ++ul) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + 16 * ((NU * q + ul) ^ (D >= 128 ? (pr & 1) : 0)));
      const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
      uint32_t r[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = wd[j], hi = wd[j] >> 8;
        r[4 * j + 0] = lo & 0x000F000Fu;
        r[4 * j + 1] = lo & 0x00F000F0u;
        r[4 * j + 2] = hi & 0x000F000Fu;
        r[4 * j + 3] = hi & 0x00F000F0u;
      }
      tc::st_16x128b_x8(tmem + (static_cast<uint32_t>(32 * w + 16 * t) << 16) + 32 * ul, r);
    }
  }
}

// A position whose largest value z + 15 s is beyond fp16 (z and s are fp16, so it is below 16 times its
// range): the unit's values are then taken times 1/16 and its probabilities times 16.  The warps
// that unpack and the ones that form P find it each from the same bytes.
__device__ __forceinline__ bool value_large(uint32_t sz) { return fmaf(15.f, half_lo(sz), half_hi(sz)) > 65504.f; }

// Values of the unit to fp16, transposed: thread t takes quad Q = 8 w + t / 4 (4 dims) and the row
// pairs 4 i + t % 4 of the unit; dim 4 Q + k goes to TMEM lane 32 w + 8 k + t / 4, row pair p to
// column p.  Rows outside [lo, hi) may hold anything: their scale and zero are taken as 0.  With
// `large` the values are taken times 1/16 (see value_large).
template <int D>
__device__ __forceinline__ void unpack_values(const uint8_t* raw, uint32_t tmem, int w, int lane, uint32_t ok, int lo, int hi, bool large) {
  using Gm = Geo<D>;
  const int a = lane >> 2, q = lane & 3, Q = 8 * w + a;
  const uint8_t* vw = raw + 8 * D + ((Q / Gm::WPC) * 4 + q) * Gm::CH + 4 * (Q % Gm::WPC);
  const uint8_t* pp = raw + 16 * D + 64 + 8 * q;
  const bool part = ok != 0xFFu || lo > 0 || hi < kTile;
  const __half2 sixteenth = __float2half2_rn(0.0625f);
  // the unit's instructions are few: the warps of all roles run from one instruction cache
#pragma unroll 1
  for (int blk = 0; blk < 4; ++blk) {  // 16 columns: 2 tiles
    uint32_t r[2][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int T = 2 * blk + (i >> 1), half = i & 1;
      const uint32_t x = *reinterpret_cast<const uint32_t*>(vw + T * Gm::T4B + half * 32 * Gm::CH);
      uint2 sz = *reinterpret_cast<const uint2*>(pp + T * Gm::T4B + half * 32);
      if (unlikely(part)) {
        const int p0 = 16 * T + 8 * half + 2 * q, h = ((ok >> T) & 1u) ? hi : 0;
        if (p0 < lo || p0 >= h) sz.x = 0u;
        if (p0 + 1 < lo || p0 + 1 >= h) sz.y = 0u;
      }
      const uint32_t s2 = prmt(sz.x, sz.y, 0x5410u), z2 = prmt(sz.x, sz.y, 0x7632u);
      __half2 s = *reinterpret_cast<const __half2*>(&s2), z = *reinterpret_cast<const __half2*>(&z2);
      if (unlikely(large)) {
        s = __hmul2(s, sixteenth);
        z = __hmul2(z, sixteenth);
      }
      const uint32_t x8 = x >> 8;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // 1024 + c or 1024 + 16 c, the exact code c, then one rounding of z + s c
        const uint32_t src = k < 2 ? x : x8;
        uint32_t h;
        if (k & 1) asm("lop3.b32 %0, %1, 0x00F000F0, 0x64006400, 0xea;" : "=r"(h) : "r"(src));
        else asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xea;" : "=r"(h) : "r"(src));
        const __half2 m = *reinterpret_cast<const __half2*>(&h);
        const __half2 n = (k & 1) ? __hfma2(m, sixteenth, __float2half2_rn(-64.f)) : __hadd2(m, __float2half2_rn(-1024.f));
        const __half2 v = __hfma2(n, s, z);
        r[k >> 1][2 * i + (k & 1)] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    tc::st_16x128b_x4(tmem + (static_cast<uint32_t>(32 * w) << 16) + 16 * blk, r[0]);
    tc::st_16x128b_x4(tmem + (static_cast<uint32_t>(32 * w + 16) << 16) + 16 * blk, r[1]);
  }
}

// What a softmax warp needs to find its unit.
struct SoftUnit {
  uint32_t tm;              // TMEM address of this warp's lanes
  int wg, w4, lane, nch;    // softmax group, warp in it, lane, the group's 8-column chunks
  int p0;                   // first position of the unit
  u32 i;                    // number of the unit
  bool first, raise;        // first unit of the segment; the running maxima have to be raised
};

// A unit off the straight path, for one warp of a softmax group (all four take it together): positions
// that some row does not attend, scaled queries, values taken times 1/16, and running maxima to be
// raised (outputs are rescaled in TMEM, after the MMAs that are adding to them).  Reads the scores,
// writes the unit's probabilities over what the straight path may have left there, and adds them to
// the positions' sums l.
// Kept out of the loop: the loops of all roles run side by side from one instruction cache.
template <int D>
__device__ __noinline__ void soft_unit_slow(SmemPrefix<D>& sm, const SoftUnit u, int sinks, float* l, uint32_t* err, uint64_t limit_ns) {
  using C = Cols<D>;
  const int st = static_cast<int>(u.i % kRaw), bf = static_cast<int>(u.i & 1);
  const int pos = 32 * u.w4 + u.lane, at = u.p0 + pos, id = 1 + u.wg;
  const float2 sz = sm.ksz[st][pos];
  const uint32_t scores = u.tm + C::S + kRB * bf;
  const bool dead = ((sm.odd[st][u.w4] >> (1 + (u.lane >> 4))) & 1u) || at < sinks;
  const bool large = ((sm.odd[st][0] | sm.odd[st][1] | sm.odd[st][2] | sm.odd[st][3]) & 1u) != 0u;
  auto logit = [&](int n, uint32_t s) {
    const float x = sm.mul[n] * fmaf(sz.x, __uint_as_float(s), sz.y * reinterpret_cast<const float*>(&sm.cst[n >> 1])[n & 1]);
    return dead || at >= sm.lim[n] ? kNegInf : x;
  };
  auto neg_max = [&](int n) -> float& { return reinterpret_cast<float*>(&sm.cst[n >> 1])[2 + (n & 1)]; };
  bool raise = u.raise;
  if (!raise) {
    float top = kNegInf;
#pragma unroll 1
    for (int k = 0; k < u.nch; ++k) {
      const int c0 = 8 * (u.wg + kSoftGroups * k);
      uint32_t r[8];
      tc::ld8(scores + c0, r);
      tc::wait_ld(r);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, logit(c0 + j, r[j]) + neg_max(c0 + j));
    }
    raise = group_or(id, top > (large ? kGrowLarge : kGrow));
  }
  if (raise) {
    // column maxima over the 128 positions
#pragma unroll 1
    for (int k = 0; k < u.nch; ++k) {
      const int c0 = 8 * (u.wg + kSoftGroups * k);
      uint32_t r[8];
      tc::ld8(scores + c0, r);
      tc::wait_ld(r);
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = logit(c0 + j, r[j]);
#pragma unroll
      for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = fmaxf(x[j], __shfl_xor_sync(FULL, x[j], o));
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (u.lane == j) sm.red[u.wg][u.w4][8 * k + j] = x[j];
    }
    group_sync(id);
    if (u.w4 == 0 && u.lane < 8 * u.nch) {
      const int n = 8 * (u.wg + kSoftGroups * (u.lane >> 3)) + (u.lane & 7);
      const float m0 = -neg_max(n);
      const float m1 = fmaxf(fmaxf(sm.red[u.wg][0][u.lane], sm.red[u.wg][1][u.lane]), fmaxf(sm.red[u.wg][2][u.lane], sm.red[u.wg][3][u.lane])) - kLift;
      const bool up = m1 > m0;
      sm.alpha[n] = !up ? 1.f : m0 == kUnset ? 0.f : exp2_fast(m0 - m1);
      if (up) neg_max(n) = -m1;
    }
    group_sync(id);
    if (!u.first) {
      wait_bar(&sm.pv_done[(u.i - 1) & 1], ((u.i - 1) >> 1) & 1u, &sm.abort, err, limit_ns);
      tc::fence_after();
#pragma unroll 1
      for (int k = 0; k < u.nch; ++k) {
        const int c0 = 8 * (u.wg + kSoftGroups * k);
        uint32_t r[8];
        tc::ld8(u.tm + C::O + c0, r);
        tc::wait_ld(r);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          r[j] = __float_as_uint(__uint_as_float(r[j]) * sm.alpha[c0 + j]);
          l[8 * k + j] *= sm.alpha[c0 + j];
        }
        tc::st8(u.tm + C::O + c0, r);
      }
      tc::wait_st();
    }
  }
#pragma unroll 1
  for (int k = 0; k < u.nch; ++k) {
    const int c0 = 8 * (u.wg + kSoftGroups * k);
    uint32_t r[8], pk[4];
    tc::ld8(scores + c0, r);
    tc::wait_ld(r);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x0 = exp2_fast(logit(c0 + 2 * j, r[2 * j]) + neg_max(c0 + 2 * j));
      const float x1 = exp2_fast(logit(c0 + 2 * j + 1, r[2 * j + 1]) + neg_max(c0 + 2 * j + 1));
      l[8 * k + 2 * j] += x0;
      l[8 * k + 2 * j + 1] += x1;
      __half2 t = __floats2half2_rn(x0, x1);
      if (large) t = __hmul2(t, __float2half2_rn(16.f));  // the unit's values were taken times 1/16
      pk[j] = *reinterpret_cast<const uint32_t*>(&t);
    }
    *reinterpret_cast<uint4*>(&sm.P[bf][c0 * kTile + pos * 8]) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
  }
}

template <int D, int G, int QT>
__global__ void __launch_bounds__(kPrefixThreads, 1) prefix_kernel(const __grid_constant__ DecodeArgs a) {
  using Gm = Geo<D>;
  using C = Cols<D>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  SmemPrefix<D>& sm = *reinterpret_cast<SmemPrefix<D>*>(smem_raw);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int cap = a.stride * a.P;
  volatile int* abort = &sm.abort;
  pdl_wait();
  if (warp == 0) make_plan<G>(a, lane, sm.plan);
  if (tid == 32) {
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&sm.raw_full[i], 1);
      mbar_init(&sm.raw_empty[i], 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.k_ready[i], 4);
      mbar_init(&sm.v_ready[i], 4);
      mbar_init(&sm.qk_done[i], 1);
      mbar_init(&sm.p_ready[i], kSoftWarps);
      mbar_init(&sm.pv_done[i], 1);
    }
    mbar_init(&sm.q_ready, kSoftWarps);
    mbar_init(&sm.drained, 1);
    mbar_init(&sm.stall, 1);
    fence_mbar_init();
    sm.abort = 0;
  }
  if (warp == kMmaWarp) tc::alloc(&sm.tmem, C::All);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tm = uniform(sm.tmem);
  auto wait = [&](uint64_t* bar, u32 n) { wait_bar(bar, n & 1u, abort, a.err, a.wait_ns); };  // the n-th completion (0-based)

  Segment& s = sm.seg[warp];
  walk_start(s, sm.plan, lane);
  u32 i = 0;  // units so far

  if (warp < kSoftWarps) {
    // ------------------------------------------------------------------ softmax
    const int wg = warp >> 2, w4 = warp & 3, pos = 32 * w4 + lane, id = 1 + wg;
    const uint32_t quad = static_cast<uint32_t>(32 * w4) << 16;
    if (a.stall_test) wait(&sm.stall, 0);
    while (walk_next<G>(a, sm.plan, s, lane)) {
      // the segment's queries, rotated, in log2 units: 8 rows a warp
      if (tid == 0) {
        sm.edge = 0x7fffffff;
        sm.scaled = 0;
      }
      soft_sync();
      // all of a warp's loads are in flight before the first is used
      constexpr int NR = kRB / kSoftWarps;
      const bool act = lane < D / 4;
      float x[NR][4];
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        const int r = warp + k * kSoftWarps;
        x[k][0] = x[k][1] = x[k][2] = x[k][3] = 0.f;
        if (r < s.rows && act) {
          const size_t q0 = (static_cast<size_t>(s.bfirst + r / G) * a.Hq + static_cast<size_t>(s.g) * G + r % G) * D + 4 * lane;
#pragma unroll
          for (int e = 0; e < 4; ++e) x[k][e] = load_q<QT>(a.q, q0 + e);
        }
      }
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        const int r = warp + k * kSoftWarps;
        float big = 0.f, sum = 0.f, f = 1.f;
        if (r < s.rows) {
          flip_signs4(x[k], lane, a.signs);
          hadamard4(x[k], lane, a.h);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[k][e] *= a.qscale * kQShift / a.h;
            big = fmaxf(big, fabsf(x[k][e]));
          }
#pragma unroll
          for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(FULL, big, o));
          if (big > 32768.f) {  // beyond fp16: down by a power of two (2^100 at most), undone on the logits
            const int ex = min(((__float_as_int(big) >> 23) & 0xff) - 127 - 14, 100);
            f = __int_as_float((127 + ex) << 23);
            const float down = __int_as_float((127 - ex) << 23);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[k][e] *= down;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half hx = __float2half_rn(x[k][e]);
          sum += __half2float(hx);
          const int ko = key_order<D>(4 * lane + e);
          if (act) sm.Q[(ko >> 3) * (kRB * 8) + r * 8 + (ko & 7)] = hx;
        }
        if (r < s.rows) {
#pragma unroll
          for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
        }
        if (lane == 0) {
          float* c = reinterpret_cast<float*>(&sm.cst[r >> 1]);
          c[r & 1] = sum * (1.f / kQShift);
          c[2 + (r & 1)] = r < s.rows ? -kUnset : 0.f;
          sm.mul[r] = f;
          if (f != 1.f) sm.scaled = 1;
        }
      }
      if (tid < kRB) {
        const int lim = tid < s.rows ? min(16 * s.te, max(a.s, clamp_len(a.lens[s.bfirst + tid / G], cap) - a.w)) : 0;
        sm.lim[tid] = lim;
        if (tid < s.rows) atomicMin(&sm.edge, lim);
      }
      if (s.blocks)
        for (int k = tid; k * G < s.rows; k += kSoftThreads) a.pmeta[(s.bfirst + k) * a.Hkv + s.g] = make_uint4(s.slot, s.blocks, k * G, 0u);
      fence_proxy_async_smem();
      soft_sync();
      warp_arrive(&sm.q_ready, lane);
      // a scaled query takes every unit of the segment off the straight path, a row block without rows none
      const int lim_min = uniform(sm.scaled ? -1 : sm.edge), sinks = a.s;
      const int nch = uniform((((s.rows + 15) >> 4) * 2 - wg + kSoftGroups - 1) / kSoftGroups);  // this group's chunks: 0, 1 or 2
      uint64_t l2[4 * kChunks];  // this position's share of the rows' sums, two rows a register pair
#pragma unroll
      for (int j = 0; j < 4 * kChunks; ++j) l2[j] = 0ull;
      const u32 i0 = i, i1 = i + uniform(s.n);
#pragma unroll 1
      for (int p0 = uniform(s.p0); i != i1; ++i, p0 += kTile) {
        const int st = static_cast<int>(i % kRaw), bf = static_cast<int>(i & 1);
        // the unit's scores; products are issued in order, so the P buffer's last ones are done too
        if (w4 == 0) wait(&sm.qk_done[bf], i >> 1);
        group_sync(id);
        tc::fence_after();
        // off the straight path: positions that some row does not attend, scaled queries, large values
        const uint4 fl = *reinterpret_cast<const uint4*>(sm.odd[st]);
        const bool odd = uniform(fl.x | fl.y | fl.z | fl.w) != 0u || p0 < sinks || p0 + kTile > lim_min || i == i0;
        bool slow = odd;
        if (!odd) {
          const float2 sz = sm.ksz[st][pos];
          const uint64_t ks2 = pack2(sz.x, sz.x), kz2 = pack2(sz.y, sz.y);
          const uint32_t scores = tm + quad + C::S + kRB * bf + 8 * wg;
          const float4* cst = &sm.cst[4 * wg];
          __half* pb = &sm.P[bf][wg * (kTile * 8) + pos * 8];
          float top = kNegInf;
          uint64_t x2[4 * kChunks];
          uint32_t r[8 * kChunks];
#pragma unroll
          for (int k = 0; k < kChunks; ++k)
            if (k < nch) tc::ld8(scores + 8 * kSoftGroups * k, r + 8 * k);
          tc::wait_ld(r);
#pragma unroll
          for (int k = 0; k < kChunks; ++k) {
            if (k >= nch) break;
            uint32_t pk[4];
#pragma unroll
            for (int j = 4 * k; j < 4 * k + 4; ++j) {
              // logits minus the running maximum, two rows at once
              const float4 cc = cst[4 * kSoftGroups * k + j - 4 * k];
              const uint64_t sv = pack2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
              const uint64_t x = fma2(ks2, sv, fma2(kz2, pack2(cc.x, cc.y), pack2(cc.z, cc.w)));
              float e0, e1;
              unpack2(x, e0, e1);
              top = tc::max3(top, e0, e1);
              const float x0 = exp2_fast(e0), x1 = exp2_fast(e1);
              x2[j] = pack2(x0, x1);
              asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(pk[j - 4 * k]) : "f"(x1), "f"(x0));
            }
            *reinterpret_cast<uint4*>(pb + k * (kSoftGroups * kTile * 8)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
          slow = uniform(static_cast<int>(group_or(id, top > kGrow))) != 0;  // then the unit is done again
          if (!slow) {
#pragma unroll
            for (int k = 0; k < kChunks; ++k) {
              if (k >= nch) break;
#pragma unroll
              for (int j = 4 * k; j < 4 * k + 4; ++j) l2[j] = add2(l2[j], x2[j]);
            }
          }
        }
        if (unlikely(slow)) {
          float l[8 * kChunks];
#pragma unroll
          for (int j = 0; j < 4 * kChunks; ++j) unpack2(l2[j], l[2 * j], l[2 * j + 1]);
          soft_unit_slow<D>(sm, SoftUnit{tm + quad, wg, w4, lane, nch, p0, i, i == i0, !odd || i == i0}, sinks, l, a.err, a.wait_ns);
#pragma unroll
          for (int j = 0; j < 4 * kChunks; ++j) l2[j] = pack2(l[2 * j], l[2 * j + 1]);
        }
        fence_proxy_async_smem();
        tc::fence_before();
        warp_arrive(&sm.p_ready[bf], lane);
      }

      // the segment's partial: O^T lane 8 k + a of this warp is dim 32 w4 + 4 a + k
      if (w4 == 0) wait(&sm.pv_done[(i - 1) & 1], (i - 1) >> 1);
      group_sync(id);
      tc::fence_after();
      float* part = a.ppart + static_cast<size_t>(s.slot) * kRB * kPartRow<D>;
      const int dim = 32 * w4 + 4 * (lane & 7) + (lane >> 3), rows = s.rows;
#pragma unroll 1
      for (int k = 0; k < nch; ++k) {
        const int c0 = 8 * (wg + kSoftGroups * k);
        uint32_t o[8];
        tc::ld8(tm + quad + C::O + c0, o);
        tc::wait_ld(o);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c0 + j < rows && dim < D) part[(c0 + j) * kPartRow<D> + dim] = __uint_as_float(o[j]);
      }
      // sums over the 128 positions: lanes j and j + 16 of each warp end with this group's column j
      float l[8 * kChunks];
#pragma unroll
      for (int j = 0; j < 4 * kChunks; ++j) unpack2(l2[j], l[2 * j], l[2 * j + 1]);
      static_assert(8 * kChunks == 16, "two halves of a warp");
#pragma unroll
      for (int j = 0; j < 16; ++j) l[j] += __shfl_xor_sync(FULL, l[j], 16);
#pragma unroll
      for (int o = 8; o; o >>= 1)
#pragma unroll
        for (int j = 0; j < o; ++j) {
          const bool up = (lane & o) != 0;
          const float got = __shfl_xor_sync(FULL, up ? l[j] : l[j + o], o);
          l[j] = (up ? l[j + o] : l[j]) + got;
        }
      if (lane < 16) sm.red[wg][w4][lane] = l[0];
      group_sync(id);
      const int n = 8 * (wg + kSoftGroups * (lane >> 3)) + (lane & 7);
      if (w4 == 0 && lane < 8 * nch && n < rows) {
        const float m = -(reinterpret_cast<const float*>(&sm.cst[n >> 1])[2 + (n & 1)]);
        *reinterpret_cast<float2*>(part + n * kPartRow<D> + D) =
            make_float2(m, (sm.red[wg][0][lane] + sm.red[wg][1][lane]) + (sm.red[wg][2][lane] + sm.red[wg][3][lane]));
      }
      tc::fence_before();
      soft_sync();
    }
  } else if (warp < kValWarp0) {
    // ------------------------------------------------------------------ keys
    const int w = warp - kKeyWarp0;
    const int pos = 32 * w + lane;
    // codes are c 2^-24 (rows 8-15 of a tile: 16 c 2^-24), queries times kQShift
    const float unit = (pos & 8) ? 1048576.f / kQShift : 16777216.f / kQShift;
    while (walk_next<G>(a, sm.plan, s, lane)) {
      const int hi = attended_end<G>(a, s, cap, lane);
      const u32 i1 = i + uniform(s.n);
#pragma unroll 1
      for (int at = uniform(s.p0) + pos; i != i1; ++i, at += kTile) {
        const int st = static_cast<int>(i % kRaw), bf = static_cast<int>(i & 1);
        if (w == 0) {
          wait(&sm.raw_full[st], i / kRaw);
          if (i >= 2) wait(&sm.qk_done[bf], (i >> 1) - 1);
        }
        group_sync(6);
        tc::fence_after();
        const uint8_t* tile = sm.raw[st] + (pos >> 4) * Gm::T4B + 16 * D + 4 * (pos & 15);
        const uint32_t kp = *reinterpret_cast<const uint32_t*>(tile), vp = *reinterpret_cast<const uint32_t*>(tile + 64);
        unpack_keys<D>(sm.raw[st], tm + C::K + (D / 2) * bf, w, lane);
        sm.ksz[st][pos] = make_float2(half_lo(kp) * unit, half_hi(kp));
        const bool large = ((sm.ok[st] >> (pos >> 4)) & 1u) && at >= a.s && at < hi && value_large(vp);
        const uint32_t any = __ballot_sync(FULL, large);
        if (lane == 0) sm.odd[st][w] = (any != 0u) | (((sm.ok[st] >> (2 * w)) & 3u) ^ 3u) << 1;
        warp_arrive(&sm.raw_empty[st], lane);
        tc::wait_st();
        tc::fence_before();
        warp_arrive(&sm.k_ready[bf], lane);
      }
    }
  } else if (warp < kCopyWarp) {
    // ------------------------------------------------------------------ values
    const int w = warp - kValWarp0;
    while (walk_next<G>(a, sm.plan, s, lane)) {
      const int hi = attended_end<G>(a, s, cap, lane);
      const u32 i1 = i + uniform(s.n);
#pragma unroll 1
      for (int p0 = uniform(s.p0); i != i1; ++i, p0 += kTile) {
        const int st = static_cast<int>(i % kRaw), bf = static_cast<int>(i & 1);
        if (w == 0) {
          wait(&sm.raw_full[st], i / kRaw);
          if (i >= 2) wait(&sm.pv_done[bf], (i >> 1) - 1);
        }
        group_sync(7);
        tc::fence_after();
        const uint32_t ok = uniform(sm.ok[st]);
        if (32 * w < D) {
          const uint4 vp = *reinterpret_cast<const uint4*>(sm.raw[st] + (lane >> 2) * Gm::T4B + 16 * D + 64 + 16 * (lane & 3));
          const uint32_t v4[4] = {vp.x, vp.y, vp.z, vp.w};
          bool large = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = p0 + 4 * lane + e;
            large |= ((ok >> (lane >> 2)) & 1u) && at >= a.s && at < hi && value_large(v4[e]);
          }
          unpack_values<D>(sm.raw[st], tm + C::V + (kTile / 2) * bf, w, lane, ok, a.s - p0, hi - p0, __any_sync(FULL, large));
        }
        warp_arrive(&sm.raw_empty[st], lane);
        tc::wait_st();
        tc::fence_before();
        warp_arrive(&sm.v_ready[bf], lane);
      }
    }
  } else if (warp == kCopyWarp) {
    // ------------------------------------------------------------------ copies
    // After an abort none is started: a buffer's barrier may still wait for the bytes of its last ones, and
    // "empty" no longer means that it has been read.  i counts the units whose copies were started.
    bool stop = false;
    while (!stop && walk_next<G>(a, sm.plan, s, lane)) {
      const int te = s.te;
      const int32_t* row = a.page_table + static_cast<size_t>(s.b0) * a.stride;
      const uint8_t* head = a.pool + static_cast<size_t>(s.g) * (a.P / 16) * Gm::T4B;
      auto page_of = [&](int ti) {  // page of a 16-position tile; the next unit's is read one unit ahead
        int lp, tin;
        tile_page(a, ti, &lp, &tin);
        return lane < 8 && ti < te ? row[lp] : 0;
      };
      int ti = (s.p0 >> 4) + lane, page = page_of(ti);
      const u32 i1 = i + uniform(s.n);
#pragma unroll 1
      for (; i != i1; ++i, ti += 8) {
        const int st = static_cast<int>(i % kRaw);
        const int next = i + 1 != i1 ? page_of(ti + 8) : 0;
        if (i >= kRaw) wait(&sm.raw_empty[st], i / kRaw - 1);
        stop = __any_sync(FULL, *abort);
        if (stop) break;
        const bool in = lane < 8 && ti < te, good = in && page >= 0 && page < a.max_pages;
        if (in && !good) atomicOr(a.err, KV4_DEVERR_PAGE_RANGE);
        const uint32_t ok = __ballot_sync(FULL, good);
        if (lane == 0) {
          sm.ok[st] = ok;
          mbar_arrive_expect_tx(&sm.raw_full[st], __popc(ok) * Gm::T4B);
        }
        __syncwarp();
        if (good) {
          int lp, tin;
          tile_page(a, ti, &lp, &tin);
          bulk_g2s(sm.raw[st] + lane * Gm::T4B,
                   head + static_cast<size_t>(page) * a.page_bytes + static_cast<size_t>(tin) * Gm::T4B, Gm::T4B, &sm.raw_full[st]);
        }
        page = next;
      }
    }
    // no copy outlives the block
    for (u32 k = i > kRaw ? i - kRaw : 0; k < i; ++k) mbar_wait_bounded(&sm.raw_full[k % kRaw], (k / kRaw) & 1u, a.err, kWaitLimitNs);
    write_rows<G>(a, sm.plan, lane);
  } else {
    // ------------------------------------------------------------------ matrix products
    // the descriptors' low bits are the address in units of 16 bytes: steps are added to them
    const uint64_t q_desc = tc::smem_desc(smem_u32(sm.Q), kRB * 16, 128), p_desc = tc::smem_desc(smem_u32(sm.P), 128, kTile * 16);
    u32 seg = 0;
    const bool leader = lane == 0;
    while (walk_next<G>(a, sm.plan, s, lane)) {
      const u32 i0 = i, i1 = i + uniform(s.n);
      const uint32_t nmma = static_cast<uint32_t>((uniform(s.rows) + 15) & ~15);
      const uint32_t id_s = tc::idesc_f16(kTile, nmma, false), id_o = tc::idesc_f16(kTile, nmma, true);
      wait(&sm.q_ready, seg++);
      // scores of unit i, then the products of the unit before; all lanes wait, one issues
#pragma unroll 1
      for (; i != i1 + 1; ++i) {
        if (i != i1) {
          const int bf = static_cast<int>(i & 1);
          wait(&sm.k_ready[bf], i >> 1);
          tc::fence_after();
          const uint32_t ak = tm + C::K + (D / 2) * bf, ds = tm + C::S + kRB * bf;
#pragma unroll
          for (int x = 0; x < D / 16; ++x) tc::mma_ts(ds, ak + 8 * x, q_desc + x * (2 * kRB * 16 / 16), id_s, x > 0, leader);
          tc::commit(&sm.qk_done[bf], leader);
        }
        if (i != i0) {
          const u32 k = i - 1;
          const int bf = static_cast<int>(k & 1);
          wait(&sm.p_ready[bf], k >> 1);
          wait(&sm.v_ready[bf], k >> 1);
          tc::fence_after();
          const uint64_t b = p_desc + bf * (kRB * kTile * 2 / 16);
          const uint32_t av = tm + C::V + (kTile / 2) * bf;
#pragma unroll
          for (int x = 0; x < kTile / 16; ++x) tc::mma_ts(tm + C::O, av + 8 * x, b + x * (256 / 16), id_o, k != i0 || x > 0, leader);
          tc::commit(&sm.pv_done[bf], leader);
        }
      }
      i = i1;
    }
    // all products are done before TMEM is freed, however the loop ended (after an abort, waits that are not
    // awaited leave the parities of qk_done and pv_done meaningless)
    if (i) {
      tc::commit(&sm.drained, leader);
      if (leader) mbar_wait_bounded(&sm.drained, 0u, a.err, kWaitLimitNs);
    }
    __syncwarp();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::dealloc(tm, C::All);
}

// ------------------------------------------------------------------ merge of prefix and own partials

// One warp per (sequence, query head).  The rows of kMergeRows partials are read together: a batch is
// one memory round trip (one by one, the merge of 128 sequences took 13 us).
constexpr int kMergeRows = 8;
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
  using VecT = typename std::conditional<PER == 4, float4, float2>::type;
  for (int t0 = 0; t0 < n; t0 += kMergeRows) {
    VecT v[kMergeRows];
    float2 ml[kMergeRows];
#pragma unroll
    for (int u = 0; u < kMergeRows; ++u) {
      const int t = min(t0 + u, n - 1);
      const float* row = t < nown ? a.part + pr.row(t, G, RS) + hd * RS
                                  : a.ppart + (static_cast<size_t>(pm.x + (t - nown)) * kRB + pm.z + hd) * RS;
      v[u] = __ldcg(reinterpret_cast<const VecT*>(row) + lane);
      ml[u] = __ldcg(reinterpret_cast<const float2*>(row + D));
    }
    float mb = M;
#pragma unroll
    for (int u = 0; u < kMergeRows; ++u)
      if (t0 + u < n && ml[u].y > 0.f) mb = fmaxf(mb, ml[u].x);
    if (mb == kNegInf) continue;  // nothing attended so far
    const float f0 = M == kNegInf ? 0.f : exp2f(M - mb);
    L *= f0;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] *= f0;
#pragma unroll
    for (int u = 0; u < kMergeRows; ++u) {
      const float w = (t0 + u < n && ml[u].y > 0.f) ? exp2f(ml[u].x - mb) : 0.f;
      if (w > 0.f) {
        const float* x = reinterpret_cast<const float*>(&v[u]);
        L = fmaf(w, ml[u].y, L);
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] = fmaf(w, x[e], o[e]);
      }
    }
    M = mb;
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
  if constexpr (DT == KV4_F32) {
    float* out = a.out + o0;
    if constexpr (PER == 4) *reinterpret_cast<float4*>(out) = make_float4(o[0], o[1], o[2], o[3]);
    else *reinterpret_cast<float2*>(out) = make_float2(o[0], o[1]);
  } else {
    uint32_t h[PER / 2];
#pragma unroll
    for (int e = 0; e < PER / 2; ++e) {
      if constexpr (DT == KV4_BF16) {
        h[e] = pack_bf2(__float2bfloat16_rn(o[2 * e]), __float2bfloat16_rn(o[2 * e + 1]));
      } else {
        const __half2 t = __floats2half2_rn(o[2 * e], o[2 * e + 1]);
        h[e] = *reinterpret_cast<const uint32_t*>(&t);
      }
    }
    uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + o0;
    if constexpr (PER == 4) *reinterpret_cast<uint2*>(out) = make_uint2(h[0], h[1]);
    else *reinterpret_cast<uint32_t*>(out) = h[0];
  }
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
